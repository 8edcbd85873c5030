// The matrix-core operations under the grouped GEMMs and the router GEMM,
// one per tile, so that the instructions' own arithmetic, which every GEMM
// here inherits, can be measured and tested on the device.
//
// MXFP8 (Mixture-of-Kittens blog post, "Other features / MXFP8 support": the
// routed experts' GEMMs take E4M3 operands with one E8M0 scale per 32
// elements along K, OCP MX v1.0): one v_mfma_scale_f32_32x32x64_f8f6f4 per
// 32x32x64 tile, placed as csrc/gemm_mxfp8.hip places it: lane l = 32 g + r
// feeds row r of A (and of B) with K[16g, 16g+16) in its low 16 bytes and
// K[32+16g, 32+16g+16) in its high 16 bytes, and the scale of row r's K
// block g.
//
// MXFP4 by E4M3 (the routed experts of csrc/routed_ffn.hip): one
// v_mfma_scale_f32_16x16x128_f8f6f4 per 16x16x128 tile, placed as there: lane
// l = 16 g + r feeds weight row r with K[32g, 32g+32) and its scale, and token r
// with K[16g, 16g+16) in its low 16 bytes, K[64+16g, 64+16g+16) in its high ones
// and the scale of block g.  Accumulator element v of the lane is weight row
// 4g + v, token r.
//
// bf16 (the grouped GEMMs and the router logits of csrc/gemm_bf16.hip): one
// v_mfma_f32_32x32x16_bf16 per 32x32x16 tile; lane l = 32 g + r feeds row r
// with K[8g, 8g+8).
//
// In the 32x32 forms, accumulator element v of lane l is row 4g + 8(v/4) + v%4, column
// r of the 32x32 result.
//
// Beside them the address check of loads through a buffer address, on which
// csrc/routed_ffn.hip relies to end its reads.
#include "common.h"

namespace moe {
namespace {

__global__ __launch_bounds__(64) void mx_mma_tiles_kernel(const uint8_t* __restrict__ a,
                                                          const uint8_t* __restrict__ a_scale,
                                                          const uint8_t* __restrict__ b,
                                                          const uint8_t* __restrict__ b_scale,
                                                          const float* __restrict__ c, float* __restrict__ d) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x, r = lane & 31, g = lane >> 5;
  const uint8_t* ar = a + (t * 32 + r) * 64;
  const uint8_t* br = b + (t * 32 + r) * 64;
  const u32x4 alo = *reinterpret_cast<const u32x4*>(ar + 16 * g);
  const u32x4 ahi = *reinterpret_cast<const u32x4*>(ar + 32 + 16 * g);
  const u32x4 blo = *reinterpret_cast<const u32x4*>(br + 16 * g);
  const u32x4 bhi = *reinterpret_cast<const u32x4*>(br + 32 + 16 * g);
  const i32x8 fa{(int)alo[0], (int)alo[1], (int)alo[2], (int)alo[3], (int)ahi[0], (int)ahi[1], (int)ahi[2], (int)ahi[3]};
  const i32x8 fb{(int)blo[0], (int)blo[1], (int)blo[2], (int)blo[3], (int)bhi[0], (int)bhi[1], (int)bhi[2], (int)bhi[3]};
  const float* ct = c + t * 1024 + (4 * g) * 32 + r;
  float* dt = d + t * 1024 + (4 * g) * 32 + r;
  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = ct[(8 * (v >> 2) + (v & 3)) * 32];
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa, fb, acc, 0, 0, 0, a_scale[(t * 32 + r) * 2 + g], 0,
                                                        b_scale[(t * 32 + r) * 2 + g]);
#pragma unroll
  for (int v = 0; v < 16; ++v) dt[(8 * (v >> 2) + (v & 3)) * 32] = acc[v];
}

__global__ __launch_bounds__(64) void mxfp4_mma_tiles_kernel(const uint8_t* __restrict__ w,
                                                             const uint8_t* __restrict__ w_scale,
                                                             const uint8_t* __restrict__ x,
                                                             const uint8_t* __restrict__ x_scale,
                                                             const float* __restrict__ c, float* __restrict__ d) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const uint8_t* xr = x + (t * 16 + r) * 128;
  const u32x4 a = *reinterpret_cast<const u32x4*>(w + (t * 16 + r) * 64 + 16 * g);
  const u32x4 lo = *reinterpret_cast<const u32x4*>(xr + 16 * g);
  const u32x4 hi = *reinterpret_cast<const u32x4*>(xr + 64 + 16 * g);
  const i32x8 fa{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 fb{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  const float* ct = c + t * 256 + (4 * g) * 16 + r;
  float* dt = d + t * 256 + (4 * g) * 16 + r;
  f32x4 acc;
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = ct[v * 16];
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa, fb, acc, 4, 0, 0, w_scale[(t * 16 + r) * 4 + g], 0,
                                                         x_scale[(t * 16 + r) * 4 + g]);
#pragma unroll
  for (int v = 0; v < 4; ++v) dt[v * 16] = acc[v];
}

__global__ __launch_bounds__(64) void bf16_mma_tiles_kernel(const bf16_t* __restrict__ a,
                                                            const bf16_t* __restrict__ b,
                                                            const float* __restrict__ c, float* __restrict__ d) {
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x, r = lane & 31, g = lane >> 5;
  const bf16x8 fa = *reinterpret_cast<const bf16x8*>(a + (t * 32 + r) * 16 + 8 * g);
  const bf16x8 fb = *reinterpret_cast<const bf16x8*>(b + (t * 32 + r) * 16 + 8 * g);
  const float* ct = c + t * 1024 + (4 * g) * 32 + r;
  float* dt = d + t * 1024 + (4 * g) * 32 + r;
  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = ct[(8 * (v >> 2) + (v & 3)) * 32];
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
#pragma unroll
  for (int v = 0; v < 16; ++v) dt[(8 * (v >> 2) + (v & 3)) * 32] = acc[v];
}

// Lane l of all lanes reads 16 bytes at `scalar` + `first` + 16 l of a buffer of
// `length` bytes in each form that the kernels use: into a register, directly to
// LDS, and of 4 bytes into a register and to LDS.
__global__ __launch_bounds__(64) void buffer_reads_kernel(const uint8_t* src, uint32_t length, uint32_t scalar,
                                                          uint32_t first, int64_t lanes, uint32_t* __restrict__ dst) {
  __shared__ u32x4 wide[64];
  __shared__ uint32_t word[64];
  const int64_t l = (int64_t)blockIdx.x * 64 + threadIdx.x;
  const uint32_t at = first + 16 * (uint32_t)l;
  const __amdgpu_buffer_rsrc_t rsrc =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(src), 0, (int)length, 0x00027000);
  lds_dma<16>(rsrc, wide, at, scalar);
  lds_dma<4>(rsrc, word, at, scalar);
  const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, scalar, 0);
  const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at, scalar, 0);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  *reinterpret_cast<u32x4*>(dst + 4 * l) = v;
  *reinterpret_cast<u32x4*>(dst + 4 * (lanes + l)) = wide[threadIdx.x];
  dst[8 * lanes + l] = w;
  dst[9 * lanes + l] = word[threadIdx.x];
}

}  // namespace

hipError_t launch_buffer_reads(const uint8_t* src, uint32_t length, uint32_t scalar, uint32_t first, int64_t lanes,
                               uint32_t* dst, hipStream_t s) {
  buffer_reads_kernel<<<(unsigned)(lanes / 64), 64, 0, s>>>(src, length, scalar, first, lanes, dst);
  return hipGetLastError();
}

hipError_t launch_bf16_mma_tiles(const bf16_t* a, const bf16_t* b, const float* c, float* d, int64_t n,
                                 hipStream_t s) {
  if (n < 0 || n > INT32_MAX) return hipErrorInvalidValue;
  if (n == 0) return hipSuccess;
  bf16_mma_tiles_kernel<<<(unsigned)n, 64, 0, s>>>(a, b, c, d);
  return hipGetLastError();
}

hipError_t launch_mxfp4_mma_tiles(const uint8_t* w, const uint8_t* w_scale, const uint8_t* x, const uint8_t* x_scale,
                                  const float* c, float* d, int64_t n, hipStream_t s) {
  if (n < 0 || n > INT32_MAX) return hipErrorInvalidValue;
  if (n == 0) return hipSuccess;
  mxfp4_mma_tiles_kernel<<<(unsigned)n, 64, 0, s>>>(w, w_scale, x, x_scale, c, d);
  return hipGetLastError();
}

hipError_t launch_mx_mma_tiles(const uint8_t* a, const uint8_t* a_scale, const uint8_t* b, const uint8_t* b_scale,
                               const float* c, float* d, int64_t n, hipStream_t s) {
  if (n < 0 || n > INT32_MAX) return hipErrorInvalidValue;
  if (n == 0) return hipSuccess;
  mx_mma_tiles_kernel<<<(unsigned)n, 64, 0, s>>>(a, a_scale, b, b_scale, c, d);
  return hipGetLastError();
}

}  // namespace moe
