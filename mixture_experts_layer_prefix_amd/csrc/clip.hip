// The global norm of many gradient tensors and their clipping:
//   norm = sqrt(sum_i sum g_i^2),  out_i = g_i min(1, max_norm / (norm + 1e-6)).
// The squares are taken and summed in fp64 (an fp32 gradient's square may
// leave fp32's range, and a long fp32 sum loses bits), in an order fixed by
// the tensors' sizes; the norm is rounded to fp32 once and the factor follows
// from that fp32 norm, so a norm computed apart gives the same bits.
//
// Tensors are cut into chunks of kChunk elements, chunks dealt round-robin to
// at most kClipGroups workgroups; the table of a launch's tensors travels in
// its kernel arguments, so a call keeps nothing on the device.  Two kernels:
// partial sums per workgroup, then the scaling, whose workgroups each add the
// partial sums up again (a launch of its own for that would cost more).
// Bound by memory: one read for the norm, one read and one write to scale.
// 604 MB of bf16: 100 + 193 us (6.0 and 6.3 TB/s) in place or into other
// buffers; 600 tensors of odd sizes, 205 MB, eight launches: 124 us.  There a
// table has 1,340 to 2,680 chunks, so the busiest workgroup takes two or three
// where the average is 1.3 to 2.6: the turns are filled 61 to 82%.
#include <type_traits>

#include "clip.h"
#include "rows.h"

namespace moe {

namespace {

// A wave's copy of a table's `first`, a few entries per lane, from which the
// entry of a chunk follows without a chain of loads: the number of entries
// that start at or before it, less one.
template <class Table>
struct EntryIndex {
  static constexpr int kPer = (Table::kEntries + 63) / 64;
  uint32_t first[kPer];
  __device__ explicit EntryIndex(const Table& t) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 64 + (threadIdx.x & 63);
      first[i] = e < t.n ? t.first[e] : 0xFFFFFFFFu;
    }
  }
  __device__ int find(uint32_t chunk) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) n += __popcll(__ballot(first[i] <= chunk));
    return n - 1;
  }
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum over a 256-thread workgroup, the same bits in every thread.
__device__ __forceinline__ double group_sum_f64(double v, double* lds) {
  v = wave_sum_f64(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

constexpr int kBatch = 4;  // 16-byte loads a thread has in flight

// Calls f(element, elements, values) for this thread's share of the chunk's n
// elements from e0: 16-byte pieces (eight bf16 or four fp32 values), kBatch
// at a time, then the elements that are left one by one.  STREAM: with the
// hint that they are not read again.  604 MB of gradients take 295 us with it
// on the scaling's reads and writes only, 298 also on the first reads, 323
// on the writes only, 347 nowhere; 201 MB of them 93, 97, 93 and 107.
template <bool F32, bool STREAM, class F>
__device__ __forceinline__ void for_pieces(const void* src, int64_t e0, int n, F f) {
  constexpr int kPiece = F32 ? 4 : 8, kStep = 256 * kPiece;
  typedef typename std::conditional<F32, float, bf16_t>::type E;
  const E* p = static_cast<const E*>(src) + e0;
  int c = threadIdx.x * kPiece;
  for (; c + (kBatch - 1) * kStep + kPiece <= n; c += kBatch * kStep) {
    u32x4 w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) w[i] = get16<STREAM>(p + c + i * kStep);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) f(c + i * kStep, kPiece, w[i]);
  }
  for (; c < n; c += kStep) {
    if (c + kPiece <= n) {
      f(c, kPiece, get16<STREAM>(p + c));
    } else {
      for (; c < n; ++c) {
        uint32_t v;
        if constexpr (F32)
          v = __float_as_uint(p[c]);
        else
          v = p[c];
        f(c, 1, u32x4{v, 0, 0, 0});
      }
    }
  }
}

// The values of a 16-byte piece.
template <bool F32>
__device__ __forceinline__ void piece_values(u32x4 w, float (&v)[F32 ? 4 : 8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ double chunk_squares(const void* p, int64_t e0, int64_t numel) {
  double s = 0.0;
  for_pieces<F32, false>(p, e0, (int)min((int64_t)kChunk, numel - e0), [&](int, int, u32x4 w) {
    float v[F32 ? 4 : 8];
    piece_values<F32>(w, v);  // zeros behind a single element
#pragma unroll
    for (float x : v) s = fma((double)x, (double)x, s);
  });
  return s;
}

__global__ void __launch_bounds__(256) squares_kernel(NormTable t, double* __restrict__ part) {
  __shared__ double lds[4];
  const EntryIndex<NormTable> index(t);
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int i = index.find(c);
    const int64_t e0 = (int64_t)(c - t.first[i]) * kChunk;
    const uint32_t m = t.numel[i];
    s += (m & kF32Entry) ? chunk_squares<true>(t.src[i], e0, m & ~kF32Entry)
                         : chunk_squares<false>(t.src[i], e0, m);
  }
  s = group_sum_f64(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// norm from the partial sums, thread t adding t, t + 256, ... first.
__device__ __forceinline__ float norm_of(const double* part, int64_t n, double* lds) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 256) s += part[i];
  return (float)sqrt(group_sum_f64(s, lds));
}

__global__ void __launch_bounds__(256) norm_kernel(const double* __restrict__ part, int64_t n, float* norm) {
  __shared__ double lds[4];
  const float v = norm_of(part, n, lds);
  if (threadIdx.x == 0) *norm = v;
}

// The factor: 1 unless the norm exceeds max_norm; a NaN norm gives NaN.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  const float f = max_norm / (norm + 1e-6f);
  return f > 1.0f ? 1.0f : f;
}

template <bool F32>
__device__ __forceinline__ void scale_chunk(const void* src, void* dst, int64_t e0, int64_t numel, float f) {
  typedef typename std::conditional<F32, float, bf16_t>::type E;
  E* out = static_cast<E*>(dst) + e0;
  for_pieces<F32, true>(src, e0, (int)min((int64_t)kChunk, numel - e0), [&](int c, int n, u32x4 w) {
    float v[F32 ? 4 : 8];
    piece_values<F32>(w, v);
#pragma unroll
    for (float& x : v) x *= f;
    if constexpr (F32) {
      if (n == 4)
        put16<true>(out + c, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                   __float_as_uint(v[3])});
      else
        out[c] = v[0];
    } else {
      if (n == 8)
        put16<true>(out + c, u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                   pack_bf16x2(v[6], v[7])});
      else
        out[c] = f32_to_bf16(v[0]);
    }
  });
}

// part null: the norm is *norm_in.
__global__ void __launch_bounds__(256) scale_kernel(ClipTable t, const double* __restrict__ part, int64_t nparts,
                                                    const float* norm_in, float* norm_out, float max_norm) {
  __shared__ double lds[4];
  const float norm = part ? norm_of(part, nparts, lds) : *norm_in;
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  const float f = clip_factor(norm, max_norm);
  const EntryIndex<ClipTable> index(t);
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int i = index.find(c);
    if (f == 1.0f && t.src[i] == t.dst[i]) continue;  // in place and nothing to clip: the bits are there
    const int64_t e0 = (int64_t)(c - t.first[i]) * kChunk;
    const uint32_t m = t.numel[i];
    if (m & kF32Entry)
      scale_chunk<true>(t.src[i], t.dst[i], e0, m & ~kF32Entry, f);
    else
      scale_chunk<false>(t.src[i], t.dst[i], e0, m, f);
  }
}

unsigned groups_of(uint32_t chunks) { return chunks < (uint32_t)kClipGroups ? chunks : (uint32_t)kClipGroups; }

// Feeds the tensors to `emit(table)` in tables of at most N entries: tensors
// above kEntryMax elements take several entries, empty ones none.
template <class Table, class Fill, class Emit>
hipError_t for_tables(int n, const int64_t* numel, const int32_t* types, Fill fill, Emit emit) {
  Table t;
  t.n = 0;
  t.first[0] = 0;
  for (int i = 0; i < n; ++i) {
    const bool f32 = types[i] == MOE_F32;
    for (int64_t e = 0; e < numel[i]; e += kEntryMax) {
      if (t.n == Table::kEntries) {
        if (hipError_t err = emit(t); err != hipSuccess) return err;
        t.n = 0;
      }
      const int64_t m = numel[i] - e < kEntryMax ? numel[i] - e : kEntryMax;
      fill(t, t.n, i, e * (f32 ? 4 : 2));
      t.numel[t.n] = (uint32_t)m | (f32 ? kF32Entry : 0);
      t.first[t.n + 1] = t.first[t.n] + (uint32_t)ceil_div(m, kChunk);
      ++t.n;
    }
  }
  return t.n ? emit(t) : hipSuccess;
}

int64_t entries_of(int n, const int64_t* numel) {
  int64_t e = 0;
  for (int i = 0; i < n; ++i) e += ceil_div(numel[i], kEntryMax);
  return e;
}

// Partial sums of every table, one after another; *nparts is their number.
hipError_t launch_squares(int n, const void* const* grads, const int64_t* numel, const int32_t* types, double* part,
                          int64_t* nparts, hipStream_t s) {
  *nparts = 0;
  return for_tables<NormTable>(
      n, numel, types,
      [&](NormTable& t, int at, int i, int64_t byte) { t.src[at] = static_cast<const char*>(grads[i]) + byte; },
      [&](const NormTable& t) {
        const unsigned g = groups_of(t.first[t.n]);
        squares_kernel<<<g, 256, 0, s>>>(t, part + *nparts);
        *nparts += g;
        return hipGetLastError();
      });
}

}  // namespace

size_t grad_norm_scratch_bytes(int n, const int64_t* numel) {
  return (size_t)(ceil_div(entries_of(n, numel), NormTable::kEntries) * kClipGroups + 1) * sizeof(double);
}

hipError_t launch_grad_norm(int n, const void* const* grads, const int64_t* numel, const int32_t* types, float* norm,
                            void* scratch, hipStream_t s) {
  double* part = static_cast<double*>(scratch);
  int64_t nparts;
  if (hipError_t err = launch_squares(n, grads, numel, types, part, &nparts, s); err != hipSuccess) return err;
  norm_kernel<<<1, 256, 0, s>>>(part, nparts, norm);
  return hipGetLastError();
}

hipError_t launch_clip_grads(int n, const void* const* grads, void* const* out, const int64_t* numel,
                             const int32_t* types, float max_norm, const float* norm_in, float* norm, void* scratch,
                             hipStream_t s) {
  double* part = nullptr;
  int64_t nparts = 0;
  if (!norm_in) {
    // At most kClipGroups partial sums, in one table or several: the scaling
    // workgroups add them up themselves.  More, or none at all (no elements):
    // one workgroup does.
    part = static_cast<double*>(scratch);
    if (hipError_t err = launch_squares(n, grads, numel, types, part, &nparts, s); err != hipSuccess) return err;
    if (nparts == 0 || nparts > kClipGroups) {
      norm_kernel<<<1, 256, 0, s>>>(part, nparts, norm);
      if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
      part = nullptr;
      norm_in = norm;
    }
  }
  float* norm_out = part ? norm : nullptr;
  return for_tables<ClipTable>(
      n, numel, types,
      [&](ClipTable& t, int at, int i, int64_t byte) {
        t.src[at] = static_cast<const char*>(grads[i]) + byte;
        t.dst[at] = static_cast<char*>(out[i]) + byte;
      },
      [&](const ClipTable& t) {
        scale_kernel<<<groups_of(t.first[t.n]), 256, 0, s>>>(t, part, nparts, norm_in, norm_out, max_norm);
        return hipGetLastError();
      });
}

}  // namespace moe
