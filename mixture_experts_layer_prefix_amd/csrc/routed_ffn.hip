// The routed experts of a few tokens on weights in 4 bits.  For token t with
// E4M3 activations x_t (a scale per 32 channels) and routes j to experts e:
//   G = x_t Wg[e]^T, U = x_t Wu[e]^T, h = MX(SiLU(G) * U)    (E4M3, a scale per 32)
//   y_t = y_add_t + sum_j w_tj h Wd[e]^T
// A route whose id is outside [0, E) adds nothing.
//
// A decoded token reads every weight of its experts for one product each, so
// the weights' bytes bound the time.  The weights stay in 4 bits up to the
// matrix cores: v_mfma_scale_f32_16x16x128_f8f6f4 takes E2M1 weights and E4M3
// activations with their block scales as they lie in memory, sixteen weight
// rows against sixteen tokens.
#include "mxfp4.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kWaves = 4;

// Lane l = 16 g + r of the operation feeds weight row r with K[32g, 32g+32)
// and its scale, and token r with K[16g, 16g+16), K[64+16g, 64+16g+16) and the
// scale of block g.  Accumulator element i of the lane is weight row 4g + i,
// token r.
__device__ __forceinline__ f32x4 mma(u32x4 w, uint32_t ws, u32x4 lo, u32x4 hi, uint32_t xs, f32x4 acc) {
  const i32x8 a{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8 b{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 0, 0, (int)ws, 0, (int)xs);
}

struct Tile {
  const uint8_t* codes;   // the lane's codes in slab 0
  const uint8_t* scale;   // the scale word of the lane's row in slab 0
};

// NT tiles of sixteen rows of a chunk of an expert's tokens.
template <int NT>
__global__ void __launch_bounds__(256) gate_up_kernel(RoutedFfn p, const int32_t* __restrict__ offsets,
                                                      const int32_t* __restrict__ row_token,
                                                      uint8_t* __restrict__ h, uint8_t* __restrict__ h_scale) {
  __shared__ f32x4 part[kWaves][4 * NT][64];
  const int e = blockIdx.y, c0 = blockIdx.x * 32;
  const int first = offsets[e], end = offsets[e + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int slabs = p.d / 128;
  const int64_t ld = p.d / 2, step = (int64_t)p.E * p.I * 4;
  const uint8_t *wq[4], *ws[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int64_t row = (int64_t)e * p.I + c0 + (m & 1) * 16 + r;
    wq[m] = (m < 2 ? p.w.q_gate : p.w.q_up) + row * ld + 16 * g;
    ws[m] = (m < 2 ? p.w.q_gate_scale : p.w.q_up_scale) + row * 4;
  }
  for (int n0 = first; n0 < end; n0 += 16 * NT) {
    const uint8_t *xq[NT], *xs[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = n0 + 16 * n + r;
      const int64_t t = row_token[row < end ? row : n0];
      xq[n] = p.x + t * p.d + 16 * g;
      xs[n] = p.x_scale + t * (p.d / 32) + g;
    }
    f32x4 acc[4][NT] = {};
    for (int s = wave; s < slabs; s += kWaves) {
      u32x4 w[4];
      uint32_t sc[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        w[m] = *reinterpret_cast<const u32x4*>(wq[m] + s * 64);
        sc[m] = *reinterpret_cast<const uint32_t*>(ws[m] + s * step) >> (8 * g);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4 lo = *reinterpret_cast<const u32x4*>(xq[n] + s * 128);
        const u32x4 hi = *reinterpret_cast<const u32x4*>(xq[n] + s * 128 + 64);
        const uint32_t xsc = xs[n][s * 4];
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[m][n] = mma(w[m], sc[m], lo, hi, xsc, acc[m][n]);
      }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) part[wave][n * 4 + m][lane] = acc[m][n];
    __syncthreads();
    for (int n = wave; n < NT; n += kWaves) {
      f32x4 v[4] = {};
      for (int q = 0; q < kWaves; ++q)
#pragma unroll
        for (int m = 0; m < 4; ++m) v[m] += part[q][n * 4 + m][lane];
      float z[8];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[i] = silu_f32(v[i / 4][i % 4]) * v[2 + i / 4][i % 4];
        mx = max(mx, __float_as_uint(z[i]) & 0x7FFFFFFFu);
      }
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
      const int be = mx_block_exp_bits(mx);
      const float inv = mx_inv_scale(be);
      const int64_t row = n0 + 16 * n + r;
      if (row < end) {
        uint8_t* out = h + row * p.I + c0 + 4 * g;
        *reinterpret_cast<uint32_t*>(out) = e4m3x4_rne_sat(z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv);
        *reinterpret_cast<uint32_t*>(out + 16) = e4m3x4_rne_sat(z[4] * inv, z[5] * inv, z[6] * inv, z[7] * inv);
        if (g == 0) h_scale[row * (p.I / 32) + c0 / 32] = (uint8_t)(be + 127);
      }
    }
    __syncthreads();
  }
}

// Each wave takes sixteen rows of the down projection and all of K.
template <int NT>
__global__ void __launch_bounds__(256) down_kernel(RoutedFfn p, const int32_t* __restrict__ offsets,
                                                   const uint8_t* __restrict__ h, const uint8_t* __restrict__ h_scale,
                                                   float* __restrict__ o) {
  const int e = blockIdx.y, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int c0 = (blockIdx.x * kWaves + (threadIdx.x >> 6)) * 16;
  const int first = offsets[e], end = offsets[e + 1], slabs = p.I / 128;
  const int64_t wrow = (int64_t)e * p.d + c0 + r, step = (int64_t)p.E * p.d * 4;
  const uint8_t* wq = p.w.q_down + wrow * (p.I / 2) + 16 * g;
  const uint8_t* ws = p.w.q_down_scale + wrow * 4;
  for (int n0 = first; n0 < end; n0 += 16 * NT) {
    const uint8_t *xq[NT], *xs[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int64_t row = min(n0 + 16 * n + r, end - 1);
      xq[n] = h + row * p.I + 16 * g;
      xs[n] = h_scale + row * (p.I / 32) + g;
    }
    f32x4 acc[NT] = {};
#pragma unroll 4
    for (int s = 0; s < slabs; ++s) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(wq + s * 64);
      const uint32_t sc = *reinterpret_cast<const uint32_t*>(ws + s * step) >> (8 * g);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4 lo = *reinterpret_cast<const u32x4*>(xq[n] + s * 128);
        const u32x4 hi = *reinterpret_cast<const u32x4*>(xq[n] + s * 128 + 64);
        acc[n] = mma(w, sc, lo, hi, xs[n][s * 4], acc[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int64_t row = n0 + 16 * n + r;
      if (row < end) *reinterpret_cast<f32x4*>(o + row * p.d + c0 + 4 * g) = acc[n];
    }
  }
}

// y[t] = y_add[t] + sum_j w_j o[row_j] over the present routes in slot order.
__global__ void __launch_bounds__(256) weighted_sum_kernel(RoutedFfn p, const int32_t* __restrict__ token_row,
                                                           const float* __restrict__ o) {
  const int per = (p.d + 1023) / 1024;  // workgroup steps of a token
  for (int64_t b = blockIdx.x; b < p.T * per; b += gridDim.x) {
    const int64_t t = b / per;
    const int c = ((int)(b - t * per) * 256 + (int)threadIdx.x) * 4;
    if (c >= p.d) continue;
    f32x4 acc = {};
    for (int j = 0; j < p.k; ++j) {
      const int64_t row = token_row[t * p.k + j];
      if (row < 0) continue;
      const float g = p.topk_w[t * p.k + j];
      const f32x4 v = *reinterpret_cast<const f32x4*>(o + row * p.d + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(g, v[i], acc[i]);
    }
    if (p.y_add) {
      float v[4];
      unpack_slot(load_slot<false, false, false, 4>(p.y_add, t * p.d + c, 4), v);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += v[i];
    }
    const float out[4] = {acc[0], acc[1], acc[2], acc[3]};
    store_slot<false, false, false, 4>(p.y, t * p.d + c, 4, pack_slot<false>(out));
  }
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct Scratch {
  int32_t *counts, *offsets, *row_token, *token_row;
  void* sort;
  uint8_t *h, *h_scale;
  float* o;
  size_t bytes;
};
Scratch carve(char* base, int64_t T, int d, int E, int k, int I) {
  const int64_t R = T * k;
  Scratch s;
  size_t at = 0;
  auto take = [&](size_t n) {
    char* p = base + at;
    at += up(n);
    return static_cast<void*>(p);
  };
  s.counts = static_cast<int32_t*>(take(E * 4));
  s.offsets = static_cast<int32_t*>(take((E + 1) * 4));
  s.row_token = static_cast<int32_t*>(take(R * 4));
  s.token_row = static_cast<int32_t*>(take(R * 4));
  s.sort = take(sort_scratch_bytes(T, k, E));
  s.h = static_cast<uint8_t*>(take(R * I));
  s.h_scale = static_cast<uint8_t*>(take(R * (I / 32)));
  s.o = static_cast<float*>(take(R * d * 4));
  s.bytes = at;
  return s;
}

}  // namespace

size_t routed_ffn_scratch_bytes(int64_t T, int d, int E, int k, int I) {
  return carve(nullptr, T, d, E, k, I).bytes;
}

hipError_t launch_routed_ffn(const RoutedFfn& p, void* scratch, hipStream_t s) {
  const Scratch b = carve(static_cast<char*>(scratch), p.T, p.d, p.E, p.k, p.I);
  const hipError_t e = launch_sort(false, p.topk_idx, nullptr, p.T, p.d, p.E, p.k, b.counts, b.offsets, b.row_token,
                                   b.token_row, nullptr, b.sort, s);
  if (e != hipSuccess) return e;
  gate_up_kernel<1><<<dim3(p.I / 32, p.E), 256, 0, s>>>(p, b.offsets, b.row_token, b.h, b.h_scale);
  down_kernel<1><<<dim3(p.d / 64, p.E), 256, 0, s>>>(p, b.offsets, b.h, b.h_scale, b.o);
  const int64_t steps = p.T * ceil_div(p.d, 1024);
  weighted_sum_kernel<<<(unsigned)(steps < 65536 ? steps : 65536), 256, 0, s>>>(p, b.token_row, b.o);
  return hipGetLastError();
}

}  // namespace moe
