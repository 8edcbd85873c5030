// Rows of bf16 or fp32 values read and written in slots of eight or four
// consecutive elements, and sums over a wave.  Used by the operators around the layer,
// whose rows may have any length and start at any element: the slots need
// element alignment only (gfx950 takes 16-byte global accesses at any
// address), and the last slot of a row may be partial.
#pragma once
#include "common.h"

namespace moe {

constexpr int kSlot = 8;  // elements per slot where a kernel does not say otherwise

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));

// Vectors at an element's address, NT with the streaming hint, for data that
// is not read again.
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
__device__ __forceinline__ u32x2 get8(const bf16_t* p) {
  const u32x2_a2* q = reinterpret_cast<const u32x2_a2*>(p);
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
template <bool NT>
__device__ __forceinline__ void put8(bf16_t* p, u32x2 v) {
  u32x2_a2* q = reinterpret_cast<u32x2_a2*>(p);
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

// N consecutive elements (8 or 4) as loaded: a thread keeps several such
// slots in flight before it unpacks them.
template <bool F32, int N = kSlot>
struct Slot {
  uint32_t w[F32 ? N : N / 2];
};

// Elements [0, left) of the slot at element `e` of p; the others read as 0.
// TAIL false: the row is whole slots, so left is at least N or not positive.
// A partial slot is read and written in pieces of four, two and one elements
// (one access per bit of left), which the value is shifted together from.
template <bool F32, bool TAIL = true, bool NT = false, int N = kSlot>
__device__ __forceinline__ Slot<F32, N> load_slot(const void* p, int64_t e, int left) {
  Slot<F32, N> s = {};
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + e;
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const u32x4 v = get16<NT>(q + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) s.w[i + k] = v[k];
      }
    } else if constexpr (TAIL) {
      if (left > 0) {
        const bool has4 = N == 8 && (left & 4), has2 = left & 2;
        u32x4 four = {};
        u32x2 two = {};
        uint32_t one = 0;
        if (has4) four = *reinterpret_cast<const u32x4_a4*>(q);
        if (has2) two = *reinterpret_cast<const u32x2_a4*>(q + (left & 4));
        if (left & 1) one = __float_as_uint(q[left - 1]);
        const u32x4 rest = has2 ? u32x4{two[0], two[1], one, 0} : u32x4{one, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s.w[k] = has4 ? four[k] : rest[k];
          if constexpr (N == 8) s.w[4 + k] = has4 ? rest[k] : 0;
        }
      }
    }
  } else {
    const bf16_t* q = static_cast<const bf16_t*>(p) + e;
    if (left >= N) {
      if constexpr (N == 8) {
        const u32x4 v = get16<NT>(q);
#pragma unroll
        for (int k = 0; k < 4; ++k) s.w[k] = v[k];
      } else {
        const u32x2 v = get8<NT>(q);
        s.w[0] = v[0];
        s.w[1] = v[1];
      }
    } else if constexpr (TAIL) {
      if (left > 0) {
        const bool has4 = N == 8 && (left & 4), has2 = left & 2;
        u32x2 four = {};
        uint32_t two = 0, one = 0;
        if (has4) four = *reinterpret_cast<const u32x2_a2*>(q);
        if (has2) two = *reinterpret_cast<const u32_a2*>(q + (left & 4));
        if (left & 1) one = q[left - 1];
        const u32x2 rest = has2 ? u32x2{two, one} : u32x2{one, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          s.w[k] = has4 ? four[k] : rest[k];
          if constexpr (N == 8) s.w[2 + k] = has4 ? rest[k] : 0;
        }
      }
    }
  }
  return s;
}

template <bool F32, int N>
__device__ __forceinline__ void unpack_slot(const Slot<F32, N>& s, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (F32)
      v[i] = __uint_as_float(s.w[i]);
    else
      v[i] = __uint_as_float(i % 2 ? s.w[i / 2] & 0xFFFF0000u : s.w[i / 2] << 16);
  }
}

// bf16: rounded to nearest even, the one rounding of the value.
template <bool F32, int N>
__device__ __forceinline__ Slot<F32, N> pack_slot(const float (&v)[N]) {
  Slot<F32, N> s;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (F32)
      s.w[i] = __float_as_uint(v[i]);
    else if (i % 2 == 0)
      s.w[i / 2] = pack_bf16x2(v[i], v[i + 1]);
  }
  return s;
}

// Writes elements [0, left) of the slot.
template <bool F32, bool TAIL = true, bool NT = false, int N = kSlot>
__device__ __forceinline__ void store_slot(void* p, int64_t e, int left, const Slot<F32, N>& s) {
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + e;
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) put16<NT>(q + i, u32x4{s.w[i], s.w[i + 1], s.w[i + 2], s.w[i + 3]});
    } else if constexpr (TAIL) {
      if (left > 0) {
        const bool has4 = N == 8 && (left & 4);
        uint32_t rest[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) rest[k] = has4 ? s.w[(4 + k) % N] : s.w[k];
        if (has4) *reinterpret_cast<u32x4_a4*>(q) = u32x4{s.w[0], s.w[1], s.w[2], s.w[3]};
        if (left & 2) *reinterpret_cast<u32x2_a4*>(q + (left & 4)) = u32x2{rest[0], rest[1]};
        if (left & 1) q[left - 1] = __uint_as_float((left & 2) ? rest[2] : rest[0]);
      }
    }
  } else {
    bf16_t* q = static_cast<bf16_t*>(p) + e;
    if (left >= N) {
      if constexpr (N == 8)
        put16<NT>(q, u32x4{s.w[0], s.w[1], s.w[2], s.w[3]});
      else
        put8<NT>(q, u32x2{s.w[0], s.w[1]});
    } else if constexpr (TAIL) {
      if (left > 0) {
        const bool has4 = N == 8 && (left & 4);
        const uint32_t r0 = has4 ? s.w[2 % (N / 2)] : s.w[0], r1 = has4 ? s.w[3 % (N / 2)] : s.w[1];
        if (has4) *reinterpret_cast<u32x2_a2*>(q) = u32x2{s.w[0], s.w[1]};
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
