// Weights in 4 bits: E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) with one E8M0 scale per 32 elements of a row (OCP MX v1.0).  The
// block exponent is the smallest e with max|v| / 2^e <= 6 (the finest
// power-of-two scale that clips nothing, the rule of the E4M3 quantizers),
// clamped to [-127, 127]; an element is v / 2^e rounded to nearest even, sign
// kept.  v / 2^e is exact, so there is one rounding.
//
// Both directions touch every byte once and are bound by memory: 65,536 x
// 7,168 to 4 bits in 215 us (5.5 TB/s), back in 173 (6.9 TB/s).  Sixteen
// lanes take the 128 columns of a slab, eight each, so that a row's four
// scales form a word in one exchange inside the lanes' row, and sixteen rows
// write 64 consecutive bytes of the slab-major scales.  Sixteen columns a
// thread, so that a wave's codes fill whole cache lines, took 235 and 485 us:
// the reads and writes of bf16 then fill half a line each.
#include "mxfp4.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kRows = 16;   // rows of a workgroup of 256 threads
constexpr int kSlabs = 4;   // slabs of 128 columns a thread has in flight

// From the bits of a block's largest magnitude.  floor(log2) - 2 places it in
// [4, 8); a mantissa above 1.5 would land past 6.
__device__ __forceinline__ int mx4_block_exp_bits(uint32_t abits) {
  const int e = (int)(abits >> 23) - 129 + ((abits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return max(e, -127);
}

__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(const bf16_t* __restrict__ src, int64_t rows, int cols,
                                                             uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scale) {
  const int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / 16;
  const int c = threadIdx.x % 16, s0 = blockIdx.y * kSlabs, slabs = cols / 128;
  const bool on = r < rows;
  const bf16_t* from = src + r * cols + c * 8;
  Slot<false, 8> in[kSlabs];
#pragma unroll
  for (int i = 0; i < kSlabs; ++i)
    if (on && s0 + i < slabs) in[i] = load_slot<false, false, true, 8>(from, (s0 + i) * 128, 8);
#pragma unroll
  for (int i = 0; i < kSlabs; ++i) {
    if (s0 + i >= slabs) break;
    float v[8];
    unpack_slot(in[i], v);
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
    m = max(m, dpp_u32<0xB1>(m));
    m = max(m, dpp_u32<0x4E>(m));
    const int e = mx4_block_exp_bits(m);
    const float inv = mx_inv_scale(e);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= inv;
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0], v[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
    uint32_t b = (uint32_t)(e + 127) << (8 * (c / 4));
    b |= dpp_u32<0x141>(b);  // the other block of eight lanes, then the other eight lanes
    b |= dpp_u32<0x140>(b);
    if (!on) continue;
    *reinterpret_cast<uint32_t*>(codes + r * (cols / 2) + (s0 + i) * 64 + c * 4) = w;
    if (c == 0) *reinterpret_cast<uint32_t*>(scale + ((s0 + i) * rows + r) * 4) = b;
  }
}

__global__ void __launch_bounds__(256) dequantize_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scale, int64_t rows,
                                                               int cols, bf16_t* __restrict__ dst) {
  const int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / 16;
  const int c = threadIdx.x % 16, s0 = blockIdx.y * kSlabs, slabs = cols / 128;
  if (r >= rows) return;
  uint32_t w[kSlabs] = {}, b[kSlabs] = {};
#pragma unroll
  for (int i = 0; i < kSlabs; ++i) {
    if (s0 + i < slabs) {
      w[i] = *reinterpret_cast<const uint32_t*>(codes + r * (cols / 2) + (s0 + i) * 64 + c * 4);
      b[i] = *reinterpret_cast<const uint32_t*>(scale + ((s0 + i) * rows + r) * 4);
    }
  }
#pragma unroll
  for (int i = 0; i < kSlabs; ++i) {
    if (s0 + i >= slabs) break;
    // a scale of code 0 is 2^-127, below fp32's normal numbers
    const uint32_t code = (b[i] >> (8 * (c / 4))) & 0xFFu;
    const float f = __uint_as_float(code ? code << 23 : 1u << 22);
    Slot<false, 8> out;
    const auto put = [&](int q, auto v) { out.w[q] = __builtin_bit_cast(uint32_t, v); };
    put(0, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 0));
    put(1, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 1));
    put(2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 2));
    put(3, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], f, 3));
    store_slot<false, false, true, 8>(dst + r * cols + c * 8, (s0 + i) * 128, 8, out);
  }
}

dim3 slab_grid(int64_t rows, int64_t cols) {
  return dim3((unsigned)ceil_div(rows, kRows), (unsigned)ceil_div(cols / 128, kSlabs));
}

}  // namespace

hipError_t launch_quantize_mxfp4(const bf16_t* src, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scale,
                                 hipStream_t s) {
  quantize_mxfp4_kernel<<<slab_grid(rows, cols), 256, 0, s>>>(src, rows, (int)cols, codes, scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scale, int64_t rows, int64_t cols, bf16_t* dst,
                                   hipStream_t s) {
  dequantize_mxfp4_kernel<<<slab_grid(rows, cols), 256, 0, s>>>(codes, scale, rows, (int)cols, dst);
  return hipGetLastError();
}

}  // namespace moe
