// Rows of bf16 or fp32 values read and written in slots of eight consecutive
// elements, and sums over a wave.  Used by the operators around the layer,
// whose rows may have any length and start at any element: the slots need
// element alignment only (gfx950 takes 16-byte global accesses at any
// address), and the last slot of a row may be partial.
#pragma once
#include "common.h"

namespace moe {

constexpr int kSlot = 8;  // elements per slot: 16 bytes of bf16, 32 of fp32

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));

// One slot as loaded: a thread keeps several in flight before it unpacks them.
template <bool F32>
struct Slot;
template <>
struct Slot<false> {
  u32x4 w;
};
template <>
struct Slot<true> {
  u32x4 w, w2;
};

// 16 bytes at an element's address.
template <bool NT>
__device__ __forceinline__ u32x4 get16(const float* p) {
  const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(p);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}
template <bool NT>
__device__ __forceinline__ u32x4 get16(const bf16_t* p) {
  const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}
template <bool NT>
__device__ __forceinline__ void put16(float* p, u32x4 v) {
  u32x4_a4* q = reinterpret_cast<u32x4_a4*>(p);
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}
template <bool NT>
__device__ __forceinline__ void put16(bf16_t* p, u32x4 v) {
  u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

// Elements [0, left) of the slot at element `e` of p; the others read as 0.
// TAIL false: the row is whole slots, so left is at least 8 or not positive.
// NT: whole slots with the streaming hint, for data that is not read again.
// A partial slot is read and written in pieces of four, two and one elements
// (one access per bit of left), which the value is shifted together from.
template <bool F32, bool TAIL = true, bool NT = false>
__device__ __forceinline__ Slot<F32> load_slot(const void* p, int64_t e, int left) {
  Slot<F32> s = {};
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + e;
    if (left >= kSlot) {
      s.w = get16<NT>(q);
      s.w2 = get16<NT>(q + 4);
    } else if constexpr (TAIL) {
      if (left > 0) {
        const bool has4 = left & 4, has2 = left & 2;
        u32x4 four = {};
        u32x2 two = {};
        uint32_t one = 0;
        if (has4) four = *reinterpret_cast<const u32x4_a4*>(q);
        if (has2) two = *reinterpret_cast<const u32x2_a4*>(q + (left & 4));
        if (left & 1) one = __float_as_uint(q[left - 1]);
        const u32x4 rest = has2 ? u32x4{two[0], two[1], one, 0} : u32x4{one, 0, 0, 0};
        s.w = has4 ? four : rest;
        s.w2 = has4 ? rest : u32x4{0, 0, 0, 0};
      }
    }
  } else {
    const bf16_t* q = static_cast<const bf16_t*>(p) + e;
    if (left >= kSlot) {
      s.w = get16<NT>(q);
    } else if constexpr (TAIL) {
      if (left > 0) {
        const bool has4 = left & 4, has2 = left & 2;
        u32x2 four = {};
        uint32_t two = 0, one = 0;
        if (has4) four = *reinterpret_cast<const u32x2_a2*>(q);
        if (has2) two = *reinterpret_cast<const u32_a2*>(q + (left & 4));
        if (left & 1) one = q[left - 1];
        const u32x2 rest = has2 ? u32x2{two, one} : u32x2{one, 0};
        s.w = has4 ? u32x4{four[0], four[1], rest[0], rest[1]} : u32x4{rest[0], rest[1], 0, 0};
      }
    }
  }
  return s;
}

template <bool F32>
__device__ __forceinline__ void unpack_slot(const Slot<F32>& s, float (&v)[kSlot]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      v[i] = __uint_as_float(s.w[i]);
      v[i + 4] = __uint_as_float(s.w2[i]);
    } else {
      v[2 * i] = __uint_as_float(s.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(s.w[i] & 0xFFFF0000u);
    }
  }
}

// bf16: rounded to nearest even, the one rounding of the value.
template <bool F32>
__device__ __forceinline__ Slot<F32> pack_slot(const float (&v)[kSlot]) {
  Slot<F32> s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      s.w[i] = __float_as_uint(v[i]);
      s.w2[i] = __float_as_uint(v[i + 4]);
    } else {
      s.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
  return s;
}

// Writes elements [0, left) of the slot.
template <bool F32, bool TAIL = true, bool NT = false>
__device__ __forceinline__ void store_slot(void* p, int64_t e, int left, const Slot<F32>& s) {
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + e;
    if (left >= kSlot) {
      put16<NT>(q, s.w);
      put16<NT>(q + 4, s.w2);
    } else if constexpr (TAIL) {
      if (left > 0) {
        const u32x4 rest = (left & 4) ? s.w2 : s.w;
        if (left & 4) *reinterpret_cast<u32x4_a4*>(q) = s.w;
        if (left & 2) *reinterpret_cast<u32x2_a4*>(q + (left & 4)) = u32x2{rest[0], rest[1]};
        if (left & 1) q[left - 1] = __uint_as_float((left & 2) ? rest[2] : rest[0]);
      }
    }
  } else {
    bf16_t* q = static_cast<bf16_t*>(p) + e;
    if (left >= kSlot) {
      put16<NT>(q, s.w);
    } else if constexpr (TAIL) {
      if (left > 0) {
        const uint32_t r0 = (left & 4) ? s.w[2] : s.w[0], r1 = (left & 4) ? s.w[3] : s.w[1];
        if (left & 4) *reinterpret_cast<u32x2_a2*>(q) = u32x2{s.w[0], s.w[1]};
        if (left & 2) *reinterpret_cast<u32_a2*>(q + (left & 4)) = r0;
        if (left & 1) q[left - 1] = (bf16_t)((left & 2) ? r1 : r0);
      }
    }
  }
}

// Sum over the 64 lanes of a wave, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = half_sum32(v);
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__host__ __device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace moe
