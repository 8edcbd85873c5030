// The norms before and after a residual block, fused with the block's gate
// and the residual scale, and the gradient.  For token t with residual x,
// block output y, and r(v) = 1 / sqrt(mean(v^2) + eps):
//   n  = y r(y) w_post                 (post_norm; else n = y)
//   x' = alpha x + beta gate_g n       (g = t / gate_every; no y: x' = x)
//   a  = x' r(x') w_pre                (the next block's input)
// a is taken from x' before x' is rounded to the residual's type.
//
// Backward, for dx' and da, with xh = x' r_pre, yh = y r_post, u = da w_pre:
//   dz = dx' + r_pre (u - xh mean(u xh)),  dx = alpha dz,  dw_pre = sum_t da xh
//   e = beta dz,  dgate_g = sum_{t in g} e n,  dn = e gate
//   dw_post = sum_t dn yh,  v = dn w_post,  dy = r_post (v - yh mean(v yh))
// mean(v yh) splits into sums that need no second pass over the row: with
// c = beta gate w_post,
//   mean(v yh) = mean(c yh (dx' + r_pre u)) - mean(u xh) mean(c yh r_pre xh),
// so one exchange per row carries all three sums.
//
// fp32 throughout; outputs are rounded once.  Both directions read and write
// every row once and are bound by memory.  A slot is 16 bytes of the residual,
// so that one instruction of a wave covers whole cache lines: fp32 in slots of
// 32 bytes, each access filling half of its lines, took 106 us for 8,192 x
// 4,096 forward, in 16 bytes 83.  The forward's outputs are always written
// with the streaming hint.  8,192 x 7,168 bf16 on new inputs: 88 us, 93
// without; two such steps, the second reading the first's outputs: 177 and
// 186.  Where the caches hold the outputs the reader pays for it: two steps of
// 2,048 rows 52 and 51 us, of 1,024 rows 29.0 and 27.8; of 1 and 64 no change.
#include <type_traits>

#include "block_norm.h"
#include "rows.h"

namespace moe {

namespace {

// Channels of a thread's slot: 16 bytes of bf16, or of fp32 where the residual
// is fp32 (the activations' slots are then 8 bytes where they are bf16).
template <bool RF32>
constexpr int kPer = RF32 ? 4 : 8;

// Sums of NV values over the `waves` waves of a team in wave order, for all
// teams of the workgroup at once; exchanges alternate between the halves of
// `lds`, so that one barrier each is enough.  One wave: no exchange.
template <int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float (*lds)[16][NV], int waves, int& phase) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  const int first = threadIdx.y * waves;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) lds[phase][first + (threadIdx.x >> 6)][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = 0.0f;
  for (int w = 0; w < waves; ++w) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += lds[phase][first + w][i];
  }
  phase ^= 1;
}

__device__ __forceinline__ float rms_inverse(float sum, int d, float eps) { return 1.0f / sqrtf(sum / d + eps); }

// A slot of an fp32 vector, ones where the vector is missing.
template <bool TAIL, int N>
__device__ __forceinline__ void load_vec(const float* v, int64_t e, int left, float (&out)[N]) {
  if (v) {
    unpack_slot(load_slot<true, TAIL, false, N>(v, e, left), out);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = 1.0f;
  }
}

// Teams of blockDim.x threads (whole waves), blockDim.y of them in a
// workgroup, VPT slots of a row per thread.  Team b takes the rows b, b + n,
// ... of n teams, all teams of a workgroup in step, so that one barrier
// serves them.  w_pre and c = beta gate w_post stay in the threads' registers
// (MANY, several gate rows: c without the gate, whose row is read each time):
// read anew for every row they would be 12 bytes a channel from L2 beside the
// row's 8 bytes from memory (126 us for 8,192 x 7,168 bf16; so 93, and 88 with
// the writes streamed: 5.3 TB/s).  TAIL: d is not a multiple of the slot.
template <bool AF32, bool RF32, int VPT, bool MANY, bool TAIL>
__global__ void __launch_bounds__(1024, VPT * kPer<RF32> <= 8 ? 8 : 4) block_norm_kernel(BlockNorm p) {
  constexpr int N = kPer<RF32>;
  __shared__ float lds[2][16][1];
  const int waves = blockDim.x / 64, d = p.d;
  const int64_t teams = (int64_t)gridDim.x * blockDim.y;
  int phase = 0;
  auto column = [&](int q) { return (q * (int)blockDim.x + (int)threadIdx.x) * N; };
  float w_pre[VPT][N], c[VPT][N];
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    const int e = column(q), left = d - e;
    float v[N];
    load_vec<TAIL>(p.w_pre, e, left, w_pre[q]);
    load_vec<TAIL>(p.w_post, e, left, c[q]);
    load_vec<TAIL>(MANY ? nullptr : p.gate, e, left, v);
#pragma unroll
    for (int i = 0; i < N; ++i) c[q][i] *= p.beta * v[i];
  }
  const int64_t first = (int64_t)blockIdx.x * blockDim.y;
  for (int64_t t0 = first; t0 < p.T; t0 += teams) {
    const int64_t t = uniform_i64(t0 + threadIdx.y);
    const bool on = t < p.T;
    float z[VPT][N], v[N], sum[1] = {0.0f}, r = 1.0f;
    Slot<RF32, N> xs[VPT];
    if (on) {
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int left = d - column(q);
        const int64_t e = t * d + column(q);
        xs[q] = load_slot<RF32, TAIL, false, N>(p.x, e, left);
        if (p.y) {
          unpack_slot(load_slot<AF32, TAIL, false, N>(p.y, e, left), z[q]);
#pragma unroll
          for (int i = 0; i < N; ++i) sum[0] = fmaf(z[q][i], z[q][i], sum[0]);
        }
      }
    }
    if (p.post_norm) {
      team_sum<1>(sum, lds, waves, phase);
      r = rms_inverse(sum[0], d, p.eps);
      if (on && p.r_post && threadIdx.x == 0) p.r_post[t] = r;
    }
    sum[0] = 0.0f;
    if (on) {
      const int64_t g = MANY ? (uint32_t)t / (uint32_t)p.gate_every : 0;  // MANY: fewer than 2^23 tokens
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int left = d - column(q);
        const int64_t e = t * d + column(q);
        if (p.y) {
          if constexpr (MANY) {
            load_vec<TAIL>(p.gate, g * d + column(q), left, v);
#pragma unroll
            for (int i = 0; i < N; ++i) z[q][i] *= v[i];
          }
          unpack_slot(xs[q], v);
#pragma unroll
          for (int i = 0; i < N; ++i) z[q][i] = fmaf(p.alpha, v[i], c[q][i] * (z[q][i] * r));
          store_slot<RF32, TAIL, true, N>(p.x_out, e, left, pack_slot<RF32>(z[q]));
        } else {
          unpack_slot(xs[q], z[q]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) sum[0] = fmaf(z[q][i], z[q][i], sum[0]);
      }
    }
    if (!p.a) continue;
    team_sum<1>(sum, lds, waves, phase);
    if (!on) continue;
    r = rms_inverse(sum[0], d, p.eps);
    if (p.r_pre && threadIdx.x == 0) p.r_pre[t] = r;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[q][i] *= r * w_pre[q][i];
      store_slot<AF32, TAIL, true, N>(p.a, t * d + column(q), d - column(q), pack_slot<AF32>(z[q]));
    }
  }
}

// The raw slots of one row: x', da, dx', y; and its r_pre and r_post.
template <bool AF32, bool RF32, int VPT>
struct BwdRow {
  static constexpr int N = kPer<RF32>;
  float r2, r1;
  Slot<RF32, N> x[VPT], d[VPT];
  Slot<AF32, N> a[VPT], y[VPT];
};

// Workgroups of up to 16 waves, one per compute unit; a workgroup holds
// blockDim.y teams of blockDim.x threads, team b the rows [b per, (b+1) per),
// one at a time.  All teams of a workgroup take the same number of steps, so
// that one barrier serves them.  Each thread owns VPT slots of columns: w_pre
// and c = beta gate w_post stay in its registers, as do the column sums
//   sum_t da xh  and  A = sum_t dz yh,
// from which dgate_g = beta w_post A and dw_post = sum_g beta gate_g A_g.
// Where all tokens share a gate row (or there is none) A is one more column
// sum; with several gate rows, a group inside the team's rows is written
// whole, a group that began in an earlier team goes to row 2b of part_gate
// and one that begins here and goes on to row 2b + 1.  The teams' column sums
// are added over the workgroup and left as its row of part_pre and part_post
// (A where there is one gate row); sum_parts_kernel adds those rows.  16,384 x
// 7,168 bf16 with both norms and a gate: 282 us (5.0 TB/s); with the weights
// read anew and three partial rows for each of 512 teams it was 588.
// MANY: several gate rows.  TAIL: d is not a multiple of the slot.  STREAM:
// rows are read and written with the streaming hint.
template <bool AF32, bool RF32, int VPT, bool MANY, bool TAIL, bool STREAM>
__global__ void __launch_bounds__(1024) block_norm_bwd_kernel(BlockNormBwd p) {
  constexpr int N = kPer<RF32>, Q = N / 4;
  // Up to eight channels a thread the column sums are in registers, and cols
  // is room to add the teams' sums; for sixteen (rows above 8,192 channels)
  // they are in LDS, as [sum][slot][quarter][thread], each thread touching its
  // own only.  All instances of sixteen still spill at 128 registers: 8 to 56
  // of bf16, 22 to 99 with an fp32 residual, 38 to 129 of fp32.  4,096 x 12,288
  // with both norms and a gate: 140, 227 and 343 us (floors 120, 180, 240).
  constexpr bool REG = VPT * N <= 8;
  __shared__ float red[2][16][3];
  __shared__ f32x4 cols[(REG ? 1 : 2 * VPT) * Q * 1024];
  const int b = __builtin_amdgcn_readfirstlane(blockIdx.x * blockDim.y + threadIdx.y);
  const int T = (int)p.T, per = (int)p.per, every = MANY ? (int)p.gate_every : T;
  const int t0 = min(b * per, T), t1 = min(t0 + per, T);
  const int waves = blockDim.x / 64, d = p.d;
  int phase = 0;
  int g = MANY ? t0 / every : 0, g_end = min((g + 1) * every, T);  // the row's gate group and its end
  constexpr bool KEEP = REG || !RF32;  // else w_pre is read anew for each row, for want of registers
  float w_pre[KEEP ? VPT : 1][N], c[VPT][N];
  constexpr int PRE = 0, A = 1, POST = 2;  // the column sums; POST with MANY only
  float acc[REG ? 3 : 1][REG ? VPT : 1][N] = {};
  auto cell = [&](int sum, int q, int h) -> f32x4& { return cols[((sum * VPT + q) * Q + h) * 1024 + threadIdx.x]; };
  if constexpr (!REG) {  // the third sum is in the team's row of part_post
#pragma unroll
    for (int i = 0; i < 2 * VPT * Q; ++i) cell(i / (VPT * Q), i / Q % VPT, i % Q) = f32x4{};
  }
  auto add = [&](int sum, int q, const float (&v)[N]) {
    if constexpr (REG) {
#pragma unroll
      for (int i = 0; i < N; ++i) acc[sum][q][i] += v[i];
    } else {
#pragma unroll
      for (int h = 0; h < Q; ++h) cell(sum, q, h) += f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    }
  };
  auto value = [&](int sum, int q, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (REG)
        v[i] = acc[sum][q][i];
      else
        v[i] = cell(sum, q, i / 4)[i % 4];
    }
  };

  auto column = [&](int q) { return (q * (int)blockDim.x + (int)threadIdx.x) * N; };
  auto load_c = [&] {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      float gt[N];
      load_vec<TAIL>(p.w_post, column(q), d - column(q), c[q]);
      load_vec<TAIL>(p.gate, (int64_t)g * d + column(q), d - column(q), gt);
#pragma unroll
      for (int i = 0; i < N; ++i) c[q][i] *= p.beta * gt[i];
    }
  };
  bool posted = false;
  typedef BwdRow<AF32, RF32, VPT> Row;
  auto load_row = [&](int t, Row& r) {
    r.r2 = p.da ? p.r_pre[t] : 0.0f;
    r.r1 = p.post_norm ? p.r_post[t] : 1.0f;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int left = d - column(q);
      const int64_t e = (int64_t)t * d + column(q);
      r.x[q] = p.da ? load_slot<RF32, TAIL, STREAM, N>(p.x_out, e, left) : Slot<RF32, N>{};
      r.a[q] = p.da ? load_slot<AF32, TAIL, STREAM, N>(p.da, e, left) : Slot<AF32, N>{};
      r.d[q] = p.dx_out ? load_slot<RF32, TAIL, STREAM, N>(p.dx_out, e, left) : Slot<RF32, N>{};
      r.y[q] = p.y ? load_slot<AF32, TAIL, STREAM, N>(p.y, e, left) : Slot<AF32, N>{};
    }
  };
  // One row (t < t1: an idle team only joins the exchange).
  auto step = [&](int t, const Row& r) {
    const bool on = t < t1;
    const float r2 = r.r2, r1 = r.r1;
    float sum[3] = {0.0f, 0.0f, 0.0f};
    float xh[VPT][N], dz[VPT][N], yh[VPT][N];
    if (on) {
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        float a[N];
        unpack_slot(r.x[q], xh[q]);
        unpack_slot(r.a[q], a);
        unpack_slot(r.d[q], dz[q]);
        unpack_slot(r.y[q], yh[q]);
        if constexpr (!KEEP) load_vec<TAIL>(p.w_pre, column(q), d - column(q), w_pre[0]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          xh[q][i] *= r2;
          yh[q][i] *= r1;
          const float u = a[i] * w_pre[KEEP ? q : 0][i];
          sum[0] = fmaf(u, xh[q][i], sum[0]);
          dz[q][i] = fmaf(r2, u, dz[q][i]);
          const float s = c[q][i] * yh[q][i];
          sum[1] = fmaf(s, dz[q][i], sum[1]);
          sum[2] = fmaf(s, xh[q][i], sum[2]);
          a[i] *= xh[q][i];
        }
        add(PRE, q, a);
      }
    }
    team_sum<3>(sum, red, waves, phase);
    if (!on) return;
    const float m2 = r2 * (sum[0] / d), m1 = p.post_norm ? (sum[1] - m2 * sum[2]) / d : 0.0f;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int left = d - column(q);
      const int64_t e = (int64_t)t * d + column(q);
      float out[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dz[q][i] = fmaf(-m2, xh[q][i], dz[q][i]);
        out[i] = p.y ? p.alpha * dz[q][i] : dz[q][i];
      }
      store_slot<RF32, TAIL, STREAM, N>(p.dx, e, left, pack_slot<RF32>(out));
      if (!p.y) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = dz[q][i] * yh[q][i];
      add(A, q, out);
#pragma unroll
      for (int i = 0; i < N; ++i) out[i] = r1 * fmaf(c[q][i], dz[q][i], -m1 * yh[q][i]);
      store_slot<AF32, TAIL, STREAM, N>(p.dy, e, left, pack_slot<AF32>(out));
    }
    if constexpr (!MANY) return;
    const bool ends = t + 1 == g_end;
    if (!ends && t + 1 != t1) return;
    // the gate's group or the team's rows end here: hand A on
    float* out = (int64_t)g * every < t0 ? p.part_gate + 2 * (int64_t)b * p.ldp
                 : !ends                 ? p.part_gate + (2 * (int64_t)b + 1) * p.ldp
                                         : p.dgate + (int64_t)g * d;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      float wp[N], gt[N], sum_a[N];
      load_vec<TAIL>(p.w_post, column(q), d - column(q), wp);
      load_vec<TAIL>(p.gate, (int64_t)g * d + column(q), d - column(q), gt);
      value(A, q, sum_a);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        sum_a[i] *= p.beta;
        wp[i] *= sum_a[i];
        gt[i] *= sum_a[i];
      }
      if (p.dgate) store_slot<true, TAIL, false, N>(out, column(q), d - column(q), pack_slot<true>(wp));
      if constexpr (REG) {
        add(POST, q, gt);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[A][q][i] = 0.0f;
      } else {
#pragma unroll
        for (int h = 0; h < Q; ++h) cell(A, q, h) = f32x4{};
        if (p.dw_post) {  // this team's row (one team a workgroup), this thread's columns
          float* post = p.part_post + blockIdx.x * p.ldp;
          if (posted) {
            unpack_slot(load_slot<true, TAIL, false, N>(post, column(q), d - column(q)), wp);
#pragma unroll
            for (int i = 0; i < N; ++i) gt[i] += wp[i];
          }
          store_slot<true, TAIL, false, N>(post, column(q), d - column(q), pack_slot<true>(gt));
        }
      }
    }
    posted = true;
    if (ends && t + 1 < t1) {
      ++g;
      g_end = min(g_end + every, T);
      load_c();
    }
  };

  Row r = {};
  if (t0 < t1) load_row(t0, r);
  if constexpr (KEEP) {
#pragma unroll
    for (int q = 0; q < VPT; ++q) load_vec<TAIL>(p.w_pre, column(q), d - column(q), w_pre[q]);
  }
  if (t0 < T) load_c();
  for (int t = t0; t < t0 + per; ++t) {
    step(t, r);
    if (t + 1 < t1) load_row(t + 1, r);
  }

  // Column sums over the workgroup's teams, in team order.
  auto leave = [&](int sum, float* part) {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      float v[N];
      value(sum, q, v);
      if (REG && blockDim.y > 1) {
        __syncthreads();
        f32x4* mine = cols + (threadIdx.y * blockDim.x + threadIdx.x) * Q;
#pragma unroll
        for (int h = 0; h < Q; ++h) mine[h] = f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        __syncthreads();
        if (threadIdx.y == 0) {
          for (int k = 1; k < (int)blockDim.y; ++k) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += cols[(k * blockDim.x + threadIdx.x) * Q + i / 4][i % 4];
          }
        }
      }
      if (threadIdx.y == 0) store_slot<true, TAIL, false, N>(part + blockIdx.x * p.ldp, column(q), d - column(q), pack_slot<true>(v));
    }
  };
  if (p.dw_pre) leave(PRE, p.part_pre);
  if constexpr (MANY) {
    if (REG && p.dw_post) leave(POST, p.part_post);
  } else if (p.dw_post || p.dgate) {
    leave(A, p.part_post);
  }
}

// Sums of partial rows, kSumCols columns per workgroup.  Eight threads share
// four columns each, the other 32 ways of the workgroup take the n rows
// row(0), row(1), ... of src in turn; the 32 sums are then added in order and
// given to put(column, sum).
constexpr int kSumCols = 32;
template <class RowOf, class Put>
__device__ __forceinline__ void sum_rows(const BlockNormBwd& p, const float* src, int n, RowOf row_of, Put put) {
  __shared__ float lds[32][kSumCols];
  const int col = threadIdx.x & 7, sub = threadIdx.x >> 3;
  const int c = blockIdx.x * kSumCols + col * 4;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < p.ldp) {
#pragma unroll 4
    for (int i = sub; i < n; i += 32) s += *reinterpret_cast<const f32x4*>(src + (int64_t)row_of(i) * p.ldp + c);
  }
  __syncthreads();  // the sums before have been read
  *reinterpret_cast<f32x4*>(&lds[sub][col * 4]) = s;
  __syncthreads();
  const int out = blockIdx.x * kSumCols + threadIdx.x;
  if (threadIdx.x >= kSumCols || out >= p.d) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += lds[i][threadIdx.x];
  put(out, v);
}

// blockIdx.y 0 sums dw_pre; 1 dw_post and, with one gate row, dgate; the rest
// share the gate groups that span teams: the candidates are the groups or,
// where those are more than the teams, each team's last group.
__global__ void __launch_bounds__(256) sum_parts_kernel(BlockNormBwd p, int teams, int groups, int spans) {
  const bool many = p.gate && p.gate_every < p.T;
  auto same = [](int i) { return i; };
  if (blockIdx.y == 0) {
    if (p.dw_pre) sum_rows(p, p.part_pre, groups, same, [&](int c, float v) { p.dw_pre[c] = v; });
    return;
  }
  if (blockIdx.y == 1) {
    if (many && p.dw_post) sum_rows(p, p.part_post, groups, same, [&](int c, float v) { p.dw_post[c] = v; });
    if (!many && (p.dw_post || p.dgate))
      sum_rows(p, p.part_post, groups, same, [&](int c, float v) {  // v is the column's A
        if (p.dw_post) p.dw_post[c] = v * (p.gate ? p.beta * p.gate[c] : p.beta);
        if (p.dgate) p.dgate[c] = v * (p.w_post ? p.beta * p.w_post[c] : p.beta);
      });
    return;
  }
  const int T = (int)p.T, per = (int)p.per, every = (int)p.gate_every;
  const bool by_team = (T + every - 1) / every > teams;
  for (int i = blockIdx.y - 2; i < spans; i += gridDim.y - 2) {
    const int g = by_team ? (min((i + 1) * per, T) - 1) / every : i;
    const int first = g * every / per, last = (min((g + 1) * every, T) - 1) / per;
    if (first == last || (by_team && first != i)) continue;
    // row 2 first + 1, then rows 2b of the teams b after it
    sum_rows(p, p.part_gate, last - first + 1, [&](int r) { return 2 * (first + r) + (r == 0); },
             [&](int c, float v) { p.dgate[(int64_t)g * p.d + c] = v; });
  }
}

// A row's threads (whole waves), for rows of up to 16,384 channels at most
// 1,024 with as few slots each as that takes; and the rows of a workgroup.
struct TeamShape {
  int vpt, th, tpb;
};
TeamShape team_shape(int d, bool res_f32) {
  const int per = res_f32 ? 4 : 8;
  TeamShape s;
  s.vpt = 1;
  while (d > 1024 * per * s.vpt) s.vpt *= 2;
  s.th = (int)ceil_div(ceil_div(d, per * s.vpt), 64) * 64;
  s.tpb = 1024 / s.th;
  return s;
}

// Calls f with VPT, MANY and TAIL as std::integral_constant values.
template <bool RF32, class F>
void with_shape(int vpt, bool many, bool tail, F f) {
  auto flags = [&](auto v) {
    constexpr std::true_type yes;
    constexpr std::false_type no;
    if (many)
      tail ? f(v, yes, yes) : f(v, yes, no);
    else
      tail ? f(v, no, yes) : f(v, no, no);
  };
  if (vpt == 1) return flags(std::integral_constant<int, 1>());
  if (vpt == 2) return flags(std::integral_constant<int, 2>());
  if constexpr (RF32) flags(std::integral_constant<int, 4>());
}

template <bool AF32, bool RF32>
void launch_fwd(const BlockNorm& p, hipStream_t s) {
  constexpr int64_t kGroups = 512;  // two workgroups of 16 waves per compute unit
  const TeamShape t = team_shape(p.d, RF32);
  const int64_t groups = ceil_div(p.T, t.tpb);
  with_shape<RF32>(t.vpt, p.gate && p.gate_every < p.T, p.d % kPer<RF32> != 0, [&](auto V, auto MANY, auto TAIL) {
    block_norm_kernel<AF32, RF32, V.value, MANY.value, TAIL.value>
        <<<dim3((unsigned)(groups < kGroups ? groups : kGroups)), dim3(t.th, t.tpb), 0, s>>>(p);
  });
}

// The backward's workgroups: up to 16 waves, one workgroup per compute unit.
struct BwdShape {
  TeamShape t;
  int64_t per, teams, groups;  // rows of a team, teams, workgroups
};
BwdShape bwd_shape(int64_t T, int d, bool res_f32) {
  constexpr int64_t kGroups = 256;
  BwdShape s;
  s.t = team_shape(d, res_f32);
  s.per = T ? ceil_div(T, kGroups * s.t.tpb) : 1;
  s.teams = ceil_div(T, s.per);
  s.groups = ceil_div(s.teams, s.t.tpb);
  return s;
}

template <bool AF32, bool RF32>
void launch_bwd(const BlockNormBwd& p, const BwdShape& b, hipStream_t s) {
  with_shape<RF32>(b.t.vpt, p.gate && p.gate_every < p.T, p.d % kPer<RF32> != 0, [&](auto V, auto MANY, auto TAIL) {
    // Rows that the last cache level (256 MB) cannot hold stream, where they
    // are whole slots: 16,384 x 7,168 bf16 286 us, else 298; 8,192 x 4,096 with
    // an fp32 residual 127, else 131; 1,531 x 2,047 (56 MB) 27.6, else 23.4.
    auto go = [&](auto kernel) { kernel<<<dim3((unsigned)b.groups), dim3(b.t.th, b.t.tpb), 0, s>>>(p); };
    if (!TAIL.value && p.T * p.d * 3 * ((AF32 ? 4 : 2) + (RF32 ? 4 : 2)) > (256ll << 20))
      go(block_norm_bwd_kernel<AF32, RF32, V.value, MANY.value, false, true>);
    else
      go(block_norm_bwd_kernel<AF32, RF32, V.value, MANY.value, TAIL.value, false>);
  });
}

}  // namespace

size_t block_norm_scratch_bytes(int64_t T, int d) {
  size_t rows = 0;
  for (bool res_f32 : {false, true}) {  // either residual type
    const BwdShape b = bwd_shape(T, d, res_f32);
    const size_t n = (size_t)(2 * b.groups + 2 * b.teams);
    rows = n > rows ? n : rows;
  }
  return rows * (size_t)(ceil_div(d, 8) * 8) * sizeof(float);
}

hipError_t launch_block_norm(bool act_f32, bool res_f32, const BlockNorm& p, hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  if (act_f32)
    launch_fwd<true, true>(p, s);
  else if (res_f32)
    launch_fwd<false, true>(p, s);
  else
    launch_fwd<false, false>(p, s);
  return hipGetLastError();
}

hipError_t launch_block_norm_bwd(bool act_f32, bool res_f32, BlockNormBwd p, void* scratch, hipStream_t s) {
  const BwdShape b = bwd_shape(p.T, p.d, act_f32 || res_f32);
  p.ldp = ceil_div(p.d, 8) * 8;
  p.per = b.per;
  if (p.T == 0) p.gate = p.w_post = p.dgate = nullptr;  // the gate has no rows, and zero sums need no factor
  p.part_pre = static_cast<float*>(scratch);
  p.part_post = p.part_pre + b.groups * p.ldp;
  p.part_gate = p.part_post + b.groups * p.ldp;
  if (p.T == 0)
    ;  // no rows: the sums below are zero
  else if (act_f32)
    launch_bwd<true, true>(p, b, s);
  else if (res_f32)
    launch_bwd<false, true>(p, b, s);
  else
    launch_bwd<false, false>(p, b, s);
  // teams begin at multiples of per: no group spans two where the gate's period divides it
  int64_t spans = 0;
  if (p.dgate && p.gate_every < p.T && p.per % p.gate_every) {
    spans = ceil_div(p.T, p.gate_every);
    if (spans > b.teams) spans = b.teams;
  }
  if (p.dw_pre || p.dw_post || p.dgate) {
    const dim3 grid((unsigned)ceil_div(p.ldp, kSumCols), 2 + (unsigned)(spans < 256 ? spans : 256));
    sum_parts_kernel<<<grid, 256, 0, s>>>(p, (int)b.teams, (int)b.groups, (int)spans);
  }
  return hipGetLastError();
}

}  // namespace moe
