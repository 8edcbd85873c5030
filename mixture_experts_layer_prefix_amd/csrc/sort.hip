// Tokens sorted by expert and back, with the gradients of both, for routes
// that may be absent (an expert id outside [0, E): a padding token, a dropped
// route, an expert of another rank) and rows of any length.
//
// Route r = t * k + j goes to expert e = topk_idx[t][j].  Its row is
// offsets[e] plus the number of present routes of e with a smaller r, so an
// expert's rows follow in (token, slot) order; absent routes get row -1.
//   sort             x_perm[row] = x[t]
//   sort backward    dx[t] = sum_j dx_perm[row_j] (+ dx_add[t])
//   unsort           y[t] = sum_j w_j o_perm[row_j] (+ y_add[t])
//   unsort backward  do_perm[row_j] = w_j dy[t], dw_j = <dy[t], o_perm[row_j]>
// with j over the present routes in slot order, fp32 sums and one rounding.
// Every one of them is a single pass over the rows, bound by memory: a
// workgroup takes a token (several where one wave is enough for the row), a
// thread a 16-byte slot of it, and the token's row numbers are scalars.  On
// new inputs, bf16: sort of 8,192 x 7,168 with k = 8, an eighth of the tokens
// absent, 197 us (4.8 TB/s, 14 us of it the schedule); unsort of 16,384 x
// 6,144 with one route in eight present 95 to 103 us (about 6 TB/s); unsort
// backward of 8,192 x 4,096 with k = 8 209 us (5.5 TB/s).  A copy reaches 5.0
// TB/s.  The sort also takes rows of E4M3 codes with their scale rows (8,192 x
// 7,168, k = 8, an eighth of the tokens absent: 92 us, 5.3 TB/s).
#include <type_traits>

#include "rows.h"

namespace moe {

namespace {

// Elements of a 16-byte slot: the lanes of a wave then read and write whole
// cache lines with one instruction, as streaming wants them.
template <bool F32>
constexpr int kPer = F32 ? 4 : 8;
template <bool F32>
using Slot16 = Slot<F32, kPer<F32>>;
template <bool F32, bool TAIL, bool STREAM = false>
__device__ __forceinline__ Slot16<F32> load16(const void* p, int64_t e, int left) {
  return load_slot<F32, TAIL, STREAM, kPer<F32>>(p, e, left);
}
template <bool F32, bool TAIL, bool STREAM = false>
__device__ __forceinline__ void store16(void* p, int64_t e, int left, const Slot16<F32>& s) {
  store_slot<F32, TAIL, STREAM, kPer<F32>>(p, e, left, s);
}

constexpr int kSortRoutes = 256;  // routes per schedule workgroup, one per thread

// The schedule in three launches, for any number of routes (65,536: 15 us):
// routes per expert of each workgroup's 256 routes, expert-major; prefixes per
// expert; the rows.
__global__ void __launch_bounds__(kSortRoutes) sort_count_kernel(const int32_t* __restrict__ idx, int64_t R, int E,
                                                                 int32_t* __restrict__ block_counts) {
  __shared__ int32_t h[1024];
  for (int e = threadIdx.x; e < E; e += kSortRoutes) h[e] = 0;
  __syncthreads();
  const int64_t r = (int64_t)blockIdx.x * kSortRoutes + threadIdx.x;
  const int e = r < R ? idx[r] : -1;
  if ((unsigned)e < (unsigned)E) atomicAdd(&h[e], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kSortRoutes) block_counts[(int64_t)i * gridDim.x + blockIdx.x] = h[i];
}

// Exclusive prefix over the threads of a workgroup (lds: one int per wave);
// *total its sum.
__device__ __forceinline__ int scan_threads(int v, int* lds, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 63) lds[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    if (w < wave) before += lds[w];
    all += lds[w];
  }
  *total = all;
  return before + inc - v;
}

// One workgroup per expert: its column of block counts becomes prefixes.
__global__ void __launch_bounds__(256) sort_scan_kernel(int32_t* __restrict__ block_counts, int nb,
                                                        int32_t* __restrict__ counts) {
  __shared__ int lds[4];
  int32_t* col = block_counts + (int64_t)blockIdx.x * nb;
  const int per = (nb + 255) / 256;
  const int b0 = min((int)threadIdx.x * per, nb), b1 = min(b0 + per, nb);
  int sum = 0, total;
  for (int b = b0; b < b1; ++b) sum += col[b];
  int run = scan_threads(sum, lds, &total);
  for (int b = b0; b < b1; ++b) {
    const int c = col[b];
    col[b] = run;
    run += c;
  }
  if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// Lanes of the wave that hold the same id (ids below 1024; lanes with a
// negative id get an empty mask): one ballot per bit of the id.
__device__ __forceinline__ uint64_t same_id_lanes(int e) {
  uint64_t m = __ballot(e >= 0);
#pragma unroll
  for (int bit = 0; bit < 10; ++bit) {
    const uint64_t b = __ballot((e >> bit) & 1);
    m &= ((e >> bit) & 1) ? b : ~b;
  }
  return e >= 0 ? m : 0;
}

__global__ void __launch_bounds__(kSortRoutes) sort_rank_kernel(const int32_t* __restrict__ idx, int64_t R, int E, int k,
                                                                const int32_t* __restrict__ block_base,
                                                                const int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ row_token,
                                                                int32_t* __restrict__ token_row) {
  __shared__ int32_t cursor[1024];
  __shared__ int lds[4];
  // offsets: four consecutive experts per thread
  const int e0 = threadIdx.x * 4;
  int c[4], sum = 0, total;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    c[q] = e0 + q < E ? counts[e0 + q] : 0;
    sum += c[q];
  }
  int run = scan_threads(sum, lds, &total);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (e0 + q < E) {
      cursor[e0 + q] = run + block_base[(int64_t)(e0 + q) * gridDim.x + blockIdx.x];
      if (blockIdx.x == 0) offsets[e0 + q] = run;
    }
    run += c[q];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = total;
  const int64_t r = (int64_t)blockIdx.x * kSortRoutes + threadIdx.x;
  int e = r < R ? idx[r] : -1;
  if ((unsigned)e >= (unsigned)E) e = -1;
  const uint64_t same = same_id_lanes(e);
  const int lane = threadIdx.x & 63;
  const int rank = __popcll(same & ((1ull << lane) - 1));
  // the four waves take their rows in turn
  int row = -1;
  for (int w = 0; w < kSortRoutes / 64; ++w) {
    __syncthreads();
    if ((threadIdx.x >> 6) == w && e >= 0) {
      row = cursor[e] + rank;
      if ((same >> lane) == 1) cursor[e] += __popcll(same);  // the id's last lane; the wave has read
    }
  }
  if (r < R) {
    token_row[r] = row;
    if (row >= 0) row_token[row] = (int32_t)(r / k);
  }
}

// The schedule in one launch where the ids are few enough for every workgroup
// to read them all: workgroup b counts, per expert, the routes before its
// kSortRoutes own ones and the routes from there on.  Their sum is the
// expert's count, and the first count what its own ranks start from.
__global__ void __launch_bounds__(1024) sort_wide_kernel(const int32_t* __restrict__ idx, int R, int E, int k,
                                                                int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ row_token,
                                                                int32_t* __restrict__ token_row) {
  __shared__ int32_t before[1024], after[1024];  // before becomes the experts' next rows
  __shared__ int lds[16];
  const int tid = threadIdx.x, lane = tid & 63, r0 = blockIdx.x * kSortRoutes;
  before[tid] = 0;
  after[tid] = 0;
  __syncthreads();
  auto count = [&](int r, int e) {
    if ((unsigned)e < (unsigned)E) atomicAdd(r < r0 ? &before[e] : &after[e], 1);
  };
  int r = tid * 4;
#pragma unroll 4
  for (; r + 4 <= R; r += 1024 * 4) {
    const u32x4 e = get16<false>(reinterpret_cast<const float*>(idx + r));
#pragma unroll
    for (int i = 0; i < 4; ++i) count(r + i, (int)e[i]);
  }
  for (int i = 0; i < 4; ++i)
    if (r + i < R) count(r + i, idx[r + i]);
  __syncthreads();
  const int all = before[tid] + after[tid];  // of expert tid
  int total;
  const int first = scan_threads(all, lds, &total);
  before[tid] += first;
  if (blockIdx.x == 0 && tid < E) {
    counts[tid] = all;
    offsets[tid] = first;
    if (tid == 0) offsets[E] = total;
  }
  r = r0 + tid;
  const bool mine = tid < kSortRoutes && r < R;
  int e = mine ? idx[r] : -1;
  if ((unsigned)e >= (unsigned)E) e = -1;
  const uint64_t same = same_id_lanes(e);
  const int rank = __popcll(same & ((1ull << lane) - 1));
  int row = -1;
  for (int w = 0; w < kSortRoutes / 64; ++w) {
    __syncthreads();
    if ((tid >> 6) == w && e >= 0) {
      row = before[e] + rank;
      if ((same >> lane) == 1) before[e] += __popcll(same);
    }
  }
  if (mine) {
    token_row[r] = row;
    if (row >= 0) row_token[row] = r / k;
  }
}

__global__ void __launch_bounds__(256) sort_empty_kernel(int32_t* counts, int32_t* offsets, int E) {
  for (int e = threadIdx.x; e <= E; e += 256) {
    if (e < E) counts[e] = 0;
    offsets[e] = 0;
  }
}

// Absent routes have row -1; no row past the buffer is touched either.
__device__ __forceinline__ bool row_here(int64_t row, int64_t R) { return (uint64_t)row < (uint64_t)R; }

// A row kernel's workgroup: `th` threads (whole waves) per token, several
// tokens where one wave is enough.
struct RowShape {
  dim3 grid, block;
};
RowShape row_shape(bool f32, int64_t T, int d, int most = 1024) {
  const int64_t slots = ceil_div(d, f32 ? 4 : 8), per = ceil_div(slots, most);  // per thread
  const int th = (int)ceil_div(ceil_div(slots, per), 64) * 64;
  const int tok = th >= 256 ? 1 : 256 / th;
  return {dim3((unsigned)ceil_div(T, tok)), dim3((unsigned)th, (unsigned)tok)};
}

// Scale rows of MX tokens, n bytes each: read and written as words where the
// rows are whole words (d a multiple of 128), else as bytes.
struct ScaleRows {
  const uint8_t* from;
  uint8_t* to;
  int n;
};
// The token's scale bytes go to the rows row(0), ..., row(k - 1) that are there.
template <class Row>
__device__ __forceinline__ void copy_scales(const ScaleRows& s, int64_t t, int k, Row row) {
  auto copy = [&](auto unit) {
    typedef decltype(unit) W;
    const int n = s.n / (int)sizeof(W);
    const W* from = reinterpret_cast<const W*>(s.from) + t * n;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const W v = from[i];
      for (int j = 0; j < k; ++j) {
        const int64_t r = row(j);
        if (r >= 0) reinterpret_cast<W*>(s.to)[r * n + i] = v;
      }
    }
  };
  if (s.n % 4 == 0)
    copy(uint32_t());
  else
    copy(uint8_t());
}

// The whole sort in one launch for a few routes, at the cost of every
// workgroup reading all the ids: workgroup t < T finds the rows of token t's
// routes by counting the routes that come before them (an expert below, or
// the same expert and a smaller route) and copies the token; workgroup T
// makes the counts and offsets.  At least 256 threads.
template <bool F32, bool TAIL, bool MX>
__global__ void __launch_bounds__(1024) sort_few_kernel(const int32_t* __restrict__ idx, const void* __restrict__ x,
                                                        int T, int d, int E, int k, int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ offsets,
                                                        int32_t* __restrict__ row_token,
                                                        int32_t* __restrict__ token_row, void* __restrict__ xp,
                                                        ScaleRows scales) {
  __shared__ int32_t h[1024];
  __shared__ int32_t part[16][16];
  __shared__ int lds[16];
  const int R = T * k, t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if (t == T) {
    for (int e = threadIdx.x; e < 1024; e += blockDim.x) h[e] = 0;
    __syncthreads();
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
      const int e = idx[r];
      if ((unsigned)e < (unsigned)E) atomicAdd(&h[e], 1);
    }
    __syncthreads();
    const int e0 = threadIdx.x * 4;  // the first 256 threads hold the experts
    int c[4] = {}, sum = 0, total;
    if (e0 < 1024) {
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += c[q] = h[e0 + q];
    }
    int run = scan_threads(sum, lds, &total);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (e0 + q < E) {
        counts[e0 + q] = c[q];
        offsets[e0 + q] = run;
      }
      run += c[q];
    }
    if (threadIdx.x == 0) offsets[E] = total;
    return;
  }
  const int r0 = t * k;
  int c = threadIdx.x * kPer<F32>;  // the token's first slots are under way while the rows are found
  Slot16<F32> s = {};
  if (xp) s = load16<F32, TAIL>(x, (int64_t)t * d + c, d - c);
  int before[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) before[j] = 0;
  for (int base = 0; base < R; base += blockDim.x) {
    const int r = base + threadIdx.x;
    int e = r < R ? idx[r] : -1;
    if ((unsigned)e >= (unsigned)E) e = E;  // absent: behind every expert
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (j < k) {
        const int ej = idx[r0 + j];
        before[j] += __popcll(__ballot(e < ej || (e == ej && r < r0 + j)));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (lane == j) part[wave][j] = before[j];
  __syncthreads();
  if ((int)threadIdx.x < k) {
    const int e = idx[r0 + threadIdx.x];
    int row = -1;
    if ((unsigned)e < (unsigned)E) {
      row = 0;
      for (int w = 0; w < waves; ++w) row += part[w][threadIdx.x];
      row_token[row] = t;
    }
    token_row[r0 + threadIdx.x] = row;
    h[threadIdx.x] = row;
  }
  if (!xp) return;
  __syncthreads();
  if constexpr (MX) copy_scales(scales, t, k, [&](int j) { return h[j]; });
  while (c < d) {
    for (int j = 0; j < k; ++j) {
      const int row = __builtin_amdgcn_readfirstlane(h[j]);
      if (row >= 0) store16<F32, TAIL>(xp, (int64_t)row * d + c, d - c, s);
    }
    c += blockDim.x * kPer<F32>;
    if (c < d) s = load16<F32, TAIL>(x, (int64_t)t * d + c, d - c);
  }
}

constexpr int kRoutes = 8;  // routes whose rows a thread has in flight

// MX: rows of codes with their scales.  STREAM: written with the hint that they
// are not read soon.
template <bool F32, bool TAIL, bool MX, bool STREAM>
__global__ void __launch_bounds__(1024) sort_rows_kernel(const void* __restrict__ x,
                                                         const int32_t* __restrict__ token_row, void* __restrict__ xp,
                                                         int64_t T, int k, int d, ScaleRows scales) {
  const int64_t t = uniform_i64((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= T) return;
  if constexpr (MX) {
    copy_scales(scales, t, k, [&](int j) {
      const int64_t row = token_row[t * k + j];
      return row_here(row, T * k) ? row : -1;
    });
  }
  for (int c = threadIdx.x * kPer<F32>; c < d; c += blockDim.x * kPer<F32>) {
    const Slot16<F32> s = load16<F32, TAIL>(x, t * d + c, d - c);
    for (int j = 0; j < k; ++j) {
      const int64_t row = token_row[t * k + j];
      if (row_here(row, T * k)) store16<F32, TAIL, STREAM>(xp, row * d + c, d - c, s);
    }
  }
}

// The rows of up to eight present routes are in flight before the first is
// added (one after another: 166 us where this takes 101).
// y[t] = sum_j w_j rows[row_j] + add[t]; w NULL: every weight 1, add NULL: 0.
// add may be y: a slot is read before the thread that read it writes it.
// STREAM: reads with the hint that they are not read again.
template <bool F32, bool TAIL, bool STREAM>
__global__ void __launch_bounds__(1024) unsort_kernel(const void* __restrict__ rows,
                                                      const int32_t* __restrict__ token_row,
                                                      const float* __restrict__ w, const void* add, void* y, int64_t T,
                                                      int k, int d) {
  const int64_t t = uniform_i64((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= T) return;
  const int32_t* tr = token_row + t * k;
  for (int c = threadIdx.x * kPer<F32>; c < d; c += blockDim.x * kPer<F32>) {
    float acc[kPer<F32>] = {}, v[kPer<F32>];
    Slot16<F32> a;
    if (add) a = load16<F32, TAIL, STREAM>(add, t * d + c, d - c);
    for (int j0 = 0; j0 < k; j0 += kRoutes) {
      Slot16<F32> s[kRoutes];
      bool here[kRoutes];
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        const int64_t row = j0 + j < k ? tr[j0 + j] : -1;
        here[j] = row_here(row, T * k);
        if (here[j]) s[j] = load16<F32, TAIL, STREAM>(rows, row * d + c, d - c);
      }
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        if (!here[j]) continue;
        const float g = w ? w[t * k + j0 + j] : 1.0f;
        unpack_slot(s[j], v);
#pragma unroll
        for (int i = 0; i < kPer<F32>; ++i) acc[i] = fmaf(g, v[i], acc[i]);
      }
    }
    if (add) {
      unpack_slot(a, v);
#pragma unroll
      for (int i = 0; i < kPer<F32>; ++i) acc[i] += v[i];
    }
    store16<F32, TAIL, true>(y, t * d + c, d - c, pack_slot<F32>(acc));
  }
}

// dy's slot is read once for all routes, o's rows stream through and so do the
// gradient's (8,192 x 4,096, k = 8: 231 us without the hint on the writes,
// 209).  A kernel that reads those rows next pays for it: with the sort's
// backward after it 312 us, 299 without the hint; 1,024 x 7,168 81 and 74.
// Weights (dov) and rows of o (dw) are read only for the output they serve.
template <bool F32, bool TAIL>
__global__ void __launch_bounds__(1024) unsort_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ o,
                                                          const int32_t* __restrict__ token_row,
                                                          const float* __restrict__ w, void* __restrict__ dov,
                                                          float* __restrict__ dw, int64_t T, int k, int d) {
  __shared__ float part[16][16];
  const int64_t t = uniform_i64((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  const int waves = blockDim.x / 64, lane = threadIdx.x & 63;
  float(*sums)[16] = part + threadIdx.y * waves;  // a row per wave of the token
  if (t >= T) k = 0;                              // the workgroup's last tokens may be missing
  const int32_t* tr = token_row + t * k;
  const int64_t R = T * k;
  for (int j0 = 0; j0 < k; j0 += kRoutes) {
    float dot[kRoutes] = {};
    for (int c = threadIdx.x * kPer<F32>; c < d; c += blockDim.x * kPer<F32>) {
      float a[kPer<F32>], b[kPer<F32>];
      const Slot16<F32> q = load16<F32, TAIL>(dy, t * d + c, d - c);
      Slot16<F32> s[kRoutes];
      int64_t row[kRoutes];
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        row[j] = j0 + j < k ? tr[j0 + j] : -1;
        if (dw && row_here(row[j], R)) s[j] = load16<F32, TAIL, true>(o, row[j] * d + c, d - c);
      }
      unpack_slot(q, a);
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        if (!row_here(row[j], R)) continue;
        if (dw) {
          unpack_slot(s[j], b);
#pragma unroll
          for (int i = 0; i < kPer<F32>; ++i) dot[j] = fmaf(a[i], b[i], dot[j]);
        }
        if (dov) {
          const float g = w[t * k + j0 + j];
#pragma unroll
          for (int i = 0; i < kPer<F32>; ++i) b[i] = g * a[i];
          store16<F32, TAIL, true>(dov, row[j] * d + c, d - c, pack_slot<F32>(b));
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int j = 0; j < kRoutes; ++j) {
      dot[j] = wave_sum(dot[j]);  // 0 for an absent route
      if (waves > 1 && lane == 0) sums[threadIdx.x >> 6][j0 + j] = dot[j];
      if (waves == 1 && lane == 0 && j0 + j < k) dw[t * k + j0 + j] = dot[j];
    }
  }
  if (!dw || waves == 1) return;
  __syncthreads();
  if ((int)threadIdx.x < k) {
    float v = 0.0f;
    for (int i = 0; i < waves; ++i) v += sums[i][threadIdx.x];
    dw[t * k + threadIdx.x] = v;
  }
}

// Rows that the last cache level (256 MB) holds little of are read with the
// streaming hint; smaller ones are likely to be in it, having just been
// written.  The rule is on the buffer's T * k rows: which of them are present
// is known on the device only.  A present eighth is not slower for it: 59 MB of
// a 470 MB buffer 32.3 us, 33.6 without the hint; 117 MB of 940 MB 62.0, 63.3.
bool beyond_caches(bool f32, int64_t rows, int d) { return rows * d * (f32 ? 4 : 2) > (384ll << 20); }

// The instance of a kernel for an element type, a row length and a hint:
// pick(F32, TAIL, STREAM) with std::bool_constant arguments.
template <class Pick>
auto row_kernel(bool f32, int d, bool stream, Pick pick) {
  constexpr std::true_type yes;
  constexpr std::false_type no;
  const bool tail = d % (f32 ? 4 : 8) != 0;
  if (f32) {
    if (stream) return tail ? pick(yes, yes, yes) : pick(yes, no, yes);
    return tail ? pick(yes, yes, no) : pick(yes, no, no);
  }
  if (stream) return tail ? pick(no, yes, yes) : pick(no, no, yes);
  return tail ? pick(no, yes, no) : pick(no, no, no);
}

}  // namespace

// Which schedule.  Device times in us of whole calls, one after another
// (k = 8; 1 expert: k = 1).  With the rows of 512 or 7,168 channels, 256
// experts:
//   routes                512        2,048      4,096
//   few                   4.4 / 5.8  8.2 / 11   13.4 / 20.9
//   wide                  6.4 / 8.2  6.8 / 11   7.2 / 16.5
//   count, scan, rank     10 / 12    11 / 15    12 / 21
// The schedule alone (no rows):
//   routes                512   2,048   4,096   16,384   32,768   65,536
//   few, 8 or more        3.8   7.4     12.4
//     1                   3.4   8.7     21.2
//   wide, 1,024 experts   4.0   4.2     4.4     5.5      6.8      9.8
//     256                 3.9   4.2     4.5     5.6      6.9      9.6
//     8                   4.0   4.2     4.6     7.0      10.3     16.7
//     1                   4.1   5.4     7.2     17.7     31.5     59.3
//   three, 1,024 experts  9.0   9.9     10.1    11.0     12.1     14.2
//     256                 8.1   8.5     8.8     9.5      10.1     10.9
//     8                   7.5   7.7     8.1     8.4      8.5      8.7
//     1                   6.8   7.5     7.5     7.6      7.7      7.9
// The limits suit 64 experts and more with the rows copied (65,536 routes of
// 256 experts with rows of 7,168: wide 200, three launches 197).  They are not
// the best for 16,384 to 32,768 routes of very few experts, whose LDS counters
// collide (wide, where three launches are up to 24 us faster).
constexpr int64_t kFewRoutes = 2048, kFewAlone = 512, kWideLimit = 32768;

size_t sort_scratch_bytes(int64_t T, int k, int E) {
  return (size_t)ceil_div(T * k, kSortRoutes) * (size_t)E * sizeof(int32_t);
}

namespace {

hipError_t sort_rows(bool f32, const int32_t* topk_idx, const void* x, int64_t T, int d, int E, int k, int32_t* counts,
                     int32_t* offsets, int32_t* row_token, int32_t* token_row, void* x_perm, const ScaleRows& scales,
                     void* scratch, hipStream_t s) {
  if (T == 0) {
    sort_empty_kernel<<<1, 256, 0, s>>>(counts, offsets, E);
    return hipGetLastError();
  }
  const int64_t R = T * k;
  if (R <= (x_perm ? kFewRoutes : kFewAlone)) {
    const int slots = (int)ceil_div(d, f32 ? 4 : 8);
    const int th = slots <= 256 ? 256 : slots >= 1024 ? 1024 : (slots + 63) / 64 * 64;
    auto kernel = row_kernel(f32, d, false, [](auto F32, auto TAIL, auto) {
      return sort_few_kernel<F32.value, TAIL.value, false>;
    });
    if (scales.n) kernel = sort_few_kernel<false, false, true>;
    kernel<<<(unsigned)T + 1, th, 0, s>>>(topk_idx, x, (int)T, d, E, k, counts, offsets, row_token, token_row, x_perm,
                                          scales);
    return hipGetLastError();
  }
  if (R <= kWideLimit) {
    sort_wide_kernel<<<(unsigned)ceil_div(R, kSortRoutes), 1024, 0, s>>>(topk_idx, (int)R, E, k, counts, offsets,
                                                                         row_token, token_row);
  } else {
    const unsigned nb = (unsigned)ceil_div(R, kSortRoutes);
    int32_t* bc = static_cast<int32_t*>(scratch);
    sort_count_kernel<<<nb, kSortRoutes, 0, s>>>(topk_idx, R, E, bc);
    sort_scan_kernel<<<(unsigned)E, 256, 0, s>>>(bc, (int)nb, counts);
    sort_rank_kernel<<<nb, kSortRoutes, 0, s>>>(topk_idx, R, E, k, bc, counts, offsets, row_token, token_row);
  }
  if (x_perm) {
    const RowShape g = row_shape(f32, T, d, 512);  // 8,192 x 7,168, k = 8: 183 us; with up to 1,024 threads 187
    // Streaming the writes gains nothing here (8,192 x 7,168, k = 8: 196 to 197
    // us either way) and costs up to 10% where the rows fit the last cache level.
    auto kernel = row_kernel(f32, d, false, [](auto F32, auto TAIL, auto) {
      return sort_rows_kernel<F32.value, TAIL.value, false, false>;
    });
    // Codes are half as many bytes a row, and streaming them gains: 8,192 x
    // 7,168, k = 8: 130 us, streaming 108, with a kernel that reads the rows next
    // 281 and 284; 2,048: 37, 31 and 74, 71; 1,024: 18, 18 and 37, 38.
    if (scales.n)
      kernel = T * k * d * 2 > (96ll << 20) ? sort_rows_kernel<false, false, true, true>
                                            : sort_rows_kernel<false, false, true, false>;
    kernel<<<g.grid, g.block, 0, s>>>(x, token_row, x_perm, T, k, d, scales);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sort(bool f32, const int32_t* topk_idx, const void* x, int64_t T, int d, int E, int k,
                       int32_t* counts, int32_t* offsets, int32_t* row_token, int32_t* token_row, void* x_perm,
                       void* scratch, hipStream_t s) {
  return sort_rows(f32, topk_idx, x, T, d, E, k, counts, offsets, row_token, token_row, x_perm, ScaleRows{}, scratch,
                   s);
}

// A row of d codes is copied as d / 2 elements of two bytes.
hipError_t launch_sort_mx(const int32_t* topk_idx, const uint8_t* x, const uint8_t* x_scale, int64_t T, int d, int E,
                          int k, int32_t* counts, int32_t* offsets, int32_t* row_token, int32_t* token_row,
                          uint8_t* x_perm, uint8_t* x_perm_scale, void* scratch, hipStream_t s) {
  return sort_rows(false, topk_idx, x, T, d / 2, E, k, counts, offsets, row_token, token_row, x_perm,
                   ScaleRows{x_scale, x_perm_scale, d / 32}, scratch, s);
}

hipError_t launch_unsort(bool f32, const void* rows, const int32_t* token_row, const float* w, const void* add, void* y,
                         int64_t T, int d, int k, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const RowShape g = row_shape(f32, T, d);
  // 65,536 bf16 rows of 7,168 without an addend: 199 us, streaming 189; of
  // 4,096: 110, 102; of 1,536: 44.4, 40.5 from memory, but 37.7, 41.3 where the
  // last cache level holds them.  The sums are streamed in any case: 206 us
  // for 7,168 without.
  const auto kernel = row_kernel(f32, d, beyond_caches(f32, T * k, d), [](auto F32, auto TAIL, auto STREAM) {
    return unsort_kernel<F32.value, TAIL.value, STREAM.value>;
  });
  kernel<<<g.grid, g.block, 0, s>>>(rows, token_row, w, add, y, T, k, d);
  return hipGetLastError();
}

hipError_t launch_unsort_bwd(bool f32, const void* dy, const void* o_perm, const int32_t* token_row, const float* w,
                             void* do_perm, float* dw, int64_t T, int d, int k, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const RowShape g = row_shape(f32, T, d);
  const auto kernel = row_kernel(f32, d, true, [](auto F32, auto TAIL, auto) {
    return unsort_bwd_kernel<F32.value, TAIL.value>;
  });
  kernel<<<g.grid, g.block, 0, s>>>(dy, o_perm, token_row, w, do_perm, dw, T, k, d);
  return hipGetLastError();
}

}  // namespace moe
