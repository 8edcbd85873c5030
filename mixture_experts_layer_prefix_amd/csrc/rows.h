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

// Elements [0, left) of the slot at element `e` of p; the others read as 0.
// TAIL false: the row is whole slots, so left is at least 8 or not positive.
template <bool F32, bool TAIL = true>
__device__ __forceinline__ Slot<F32> load_slot(const void* p, int64_t e, int left) {
  Slot<F32> s = {};
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + e;
    if (left >= kSlot) {
      s.w = *reinterpret_cast<const u32x4_a4*>(q);
      s.w2 = *reinterpret_cast<const u32x4_a4*>(q + 4);
    } else if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < left) s.w[i] = __float_as_uint(q[i]);
        if (i + 4 < left) s.w2[i] = __float_as_uint(q[i + 4]);
      }
    }
  } else {
    const bf16_t* q = static_cast<const bf16_t*>(p) + e;
    if (left >= kSlot) {
      s.w = *reinterpret_cast<const u32x4_a2*>(q);
    } else if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v = 0;
        if (2 * i < left) v = q[2 * i];
        if (2 * i + 1 < left) v |= (uint32_t)q[2 * i + 1] << 16;
        s.w[i] = v;
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
template <bool F32, bool TAIL = true>
__device__ __forceinline__ void store_slot(void* p, int64_t e, int left, const Slot<F32>& s) {
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + e;
    if (left >= kSlot) {
      *reinterpret_cast<u32x4_a4*>(q) = s.w;
      *reinterpret_cast<u32x4_a4*>(q + 4) = s.w2;
    } else if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < left) q[i] = __uint_as_float(s.w[i]);
        if (i + 4 < left) q[i + 4] = __uint_as_float(s.w2[i]);
      }
    }
  } else {
    bf16_t* q = static_cast<bf16_t*>(p) + e;
    if (left >= kSlot) {
      *reinterpret_cast<u32x4_a2*>(q) = s.w;
    } else if constexpr (TAIL) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (2 * i < left) q[2 * i] = (bf16_t)s.w[i];
        if (2 * i + 1 < left) q[2 * i + 1] = (bf16_t)(s.w[i] >> 16);
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
