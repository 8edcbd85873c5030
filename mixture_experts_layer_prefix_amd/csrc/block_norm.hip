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
// every row once and are bound by memory.
#include "block_norm.h"
#include "rows.h"

namespace moe {

namespace {

// Sums of NV values over the `waves` waves of a workgroup (blockDim.y == 1)
// in wave order; each exchange alternates between the halves of `lds`, so
// that one barrier per exchange is enough.  One wave: no exchange.
template <int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float (*lds)[16][NV], int waves, int& phase) {
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) lds[phase][threadIdx.x >> 6][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = 0.0f;
  for (int w = 0; w < waves; ++w) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += lds[phase][w][i];
  }
  phase ^= 1;
}

__device__ __forceinline__ float rms_inverse(float sum, int d, float eps) { return 1.0f / sqrtf(sum / d + eps); }

// One row per team of blockDim.x threads (whole waves); VPT slots per thread.
template <bool AF32, bool RF32, int VPT>
__global__ void __launch_bounds__(1024) block_norm_kernel(BlockNorm p) {
  __shared__ float lds[2][16][1];
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= p.T) return;  // several teams only where each is one wave: no barrier below
  const int waves = blockDim.x / 64;
  int phase = 0;
  float z[VPT][kSlot], v[kSlot], sum[1] = {0.0f};
  Slot<RF32> xs[VPT];
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    const int c = (q * blockDim.x + threadIdx.x) * kSlot;
    if (p.x) xs[q] = load_slot<RF32>(p.x, t * p.d + c, p.d - c);
    if (p.y) {
      unpack_slot<AF32>(load_slot<AF32>(p.y, t * p.d + c, p.d - c), z[q]);
#pragma unroll
      for (int i = 0; i < kSlot; ++i) sum[0] = fmaf(z[q][i], z[q][i], sum[0]);
    }
  }
  float r = 1.0f;
  if (p.post_norm) {
    team_sum<1>(sum, lds, waves, phase);
    r = rms_inverse(sum[0], p.d, p.eps);
    if (p.r_post && threadIdx.x == 0) p.r_post[t] = r;
  }
  sum[0] = 0.0f;
  const int64_t g = p.gate ? t / p.gate_every : 0;
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    const int c = (q * blockDim.x + threadIdx.x) * kSlot;
    if (p.y) {
      if (p.post_norm) {
#pragma unroll
        for (int i = 0; i < kSlot; ++i) z[q][i] *= r;
        if (p.w_post) {
          unpack_slot<true>(load_slot<true>(p.w_post, c, p.d - c), v);
#pragma unroll
          for (int i = 0; i < kSlot; ++i) z[q][i] *= v[i];
        }
      }
      if (p.gate) {
        unpack_slot<true>(load_slot<true>(p.gate, g * p.d + c, p.d - c), v);
#pragma unroll
        for (int i = 0; i < kSlot; ++i) z[q][i] *= v[i];
      }
      unpack_slot<RF32>(xs[q], v);
#pragma unroll
      for (int i = 0; i < kSlot; ++i) z[q][i] = fmaf(p.alpha, v[i], p.beta * z[q][i]);
      store_slot<RF32>(p.x_out, t * p.d + c, p.d - c, pack_slot<RF32>(z[q]));
    } else {
      unpack_slot<RF32>(xs[q], z[q]);
    }
#pragma unroll
    for (int i = 0; i < kSlot; ++i) sum[0] = fmaf(z[q][i], z[q][i], sum[0]);
  }
  if (!p.a) return;
  team_sum<1>(sum, lds, waves, phase);
  r = rms_inverse(sum[0], p.d, p.eps);
  if (p.r_pre && threadIdx.x == 0) p.r_pre[t] = r;
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    const int c = (q * blockDim.x + threadIdx.x) * kSlot;
#pragma unroll
    for (int i = 0; i < kSlot; ++i) z[q][i] *= r;
    if (p.w_pre) {
      unpack_slot<true>(load_slot<true>(p.w_pre, c, p.d - c), v);
#pragma unroll
      for (int i = 0; i < kSlot; ++i) z[q][i] *= v[i];
    }
    store_slot<AF32>(p.a, t * p.d + c, p.d - c, pack_slot<AF32>(z[q]));
  }
}

// Team b owns the rows [b * per, (b + 1) * per).  The gradients of the
// weights are summed over the team's rows in registers and left as row b of
// part_pre and part_post.  dgate of a group inside the team's rows is whole;
// a group that began in an earlier team goes to row 2b of part_gate, one that
// began here and goes on to row 2b + 1.  sum_parts_kernel adds the rows.
template <bool AF32, bool RF32, int VPT>
__global__ void __launch_bounds__(1024) block_norm_bwd_kernel(BlockNormBwd p) {
  __shared__ float lds[2][16][3];
  const int64_t b = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t t0 = b * p.per, t1 = min(t0 + p.per, p.T);
  if (t0 >= p.T) return;  // several teams only where each is one wave: no barrier below
  const int waves = blockDim.x / 64, d = p.d;
  int phase = 0;
  float acc_pre[VPT][kSlot] = {}, acc_post[VPT][kSlot] = {}, acc_gate[VPT][kSlot] = {};
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t g = p.gate ? t / p.gate_every : 0;
    const float r2 = p.da ? p.r_pre[t] : 0.0f, r1 = p.post_norm ? p.r_post[t] : 1.0f;
    float sum[3] = {0.0f, 0.0f, 0.0f};
    Slot<RF32> xs[VPT], ds[VPT];
    Slot<AF32> ys[VPT], as[VPT];
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = (q * blockDim.x + threadIdx.x) * kSlot, left = d - c;
      const int64_t e = t * d + c;
      xs[q] = p.da ? load_slot<RF32>(p.x_out, e, left) : Slot<RF32>{};
      as[q] = p.da ? load_slot<AF32>(p.da, e, left) : Slot<AF32>{};
      ds[q] = p.dx_out ? load_slot<RF32>(p.dx_out, e, left) : Slot<RF32>{};
      ys[q] = p.y ? load_slot<AF32>(p.y, e, left) : Slot<AF32>{};
    }
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = (q * blockDim.x + threadIdx.x) * kSlot, left = d - c;
      float x[kSlot], a[kSlot], dz[kSlot], y[kSlot], w[kSlot], cf[kSlot];
      unpack_slot<RF32>(xs[q], x);
      unpack_slot<AF32>(as[q], a);
      unpack_slot<RF32>(ds[q], dz);
      unpack_slot<AF32>(ys[q], y);
      if (p.w_pre) unpack_slot<true>(load_slot<true>(p.w_pre, c, left), w);
#pragma unroll
      for (int i = 0; i < kSlot; ++i) {
        const float xh = x[i] * r2;
        acc_pre[q][i] = fmaf(a[i], xh, acc_pre[q][i]);
        const float u = p.w_pre ? a[i] * w[i] : a[i];
        sum[0] = fmaf(u, xh, sum[0]);
        dz[i] = fmaf(r2, u, dz[i]);
        x[i] = xh;
      }
      if (p.post_norm) {
        if (p.w_post) unpack_slot<true>(load_slot<true>(p.w_post, c, left), cf);
        if (p.gate) unpack_slot<true>(load_slot<true>(p.gate, g * d + c, left), w);
#pragma unroll
        for (int i = 0; i < kSlot; ++i) {
          float s = p.beta * (y[i] * r1);
          if (p.w_post) s *= cf[i];
          if (p.gate) s *= w[i];
          sum[1] = fmaf(s, dz[i], sum[1]);
          sum[2] = fmaf(s * r2, x[i], sum[2]);
        }
      }
    }
    team_sum<3>(sum, lds, waves, phase);
    const float m2 = sum[0] / d, m1 = (sum[1] - m2 * sum[2]) / d;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int c = (q * blockDim.x + threadIdx.x) * kSlot, left = d - c;
      const int64_t e = t * d + c;
      float x[kSlot], a[kSlot], dz[kSlot], y[kSlot], w[kSlot], gt[kSlot];
      unpack_slot<RF32>(xs[q], x);
      unpack_slot<AF32>(as[q], a);
      unpack_slot<RF32>(ds[q], dz);
      if (p.w_pre) unpack_slot<true>(load_slot<true>(p.w_pre, c, left), w);
#pragma unroll
      for (int i = 0; i < kSlot; ++i) {
        const float u = p.w_pre ? a[i] * w[i] : a[i];
        dz[i] = fmaf(r2, u - (x[i] * r2) * m2, dz[i]);
        x[i] = p.y ? p.alpha * dz[i] : dz[i];
      }
      store_slot<RF32>(p.dx, e, left, pack_slot<RF32>(x));
      if (!p.y) continue;
      unpack_slot<AF32>(ys[q], y);
      if (p.w_post) unpack_slot<true>(load_slot<true>(p.w_post, c, left), w);
      if (p.gate) unpack_slot<true>(load_slot<true>(p.gate, g * d + c, left), gt);
#pragma unroll
      for (int i = 0; i < kSlot; ++i) {
        const float ev = p.beta * dz[i], yh = y[i] * r1, wp = p.w_post ? w[i] : 1.0f;
        acc_gate[q][i] = fmaf(ev, yh * wp, acc_gate[q][i]);
        const float dn = p.gate ? ev * gt[i] : ev;
        acc_post[q][i] = fmaf(dn, yh, acc_post[q][i]);
        y[i] = p.post_norm ? r1 * (dn * wp - yh * m1) : dn;
      }
      store_slot<AF32>(p.dy, e, left, pack_slot<AF32>(y));
    }
    // the gate's group ends here, or this team's rows do
    if (p.dgate && (t + 1 == t1 || (t + 1) % p.gate_every == 0)) {
      const bool head = g * p.gate_every < t0, tail = t + 1 < p.T && (t + 1) % p.gate_every != 0;
      float* out = head ? p.part_gate + 2 * b * p.ldp : tail ? p.part_gate + (2 * b + 1) * p.ldp : p.dgate + g * d;
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int c = (q * blockDim.x + threadIdx.x) * kSlot;
        store_slot<true>(out, c, d - c, pack_slot<true>(acc_gate[q]));
#pragma unroll
        for (int i = 0; i < kSlot; ++i) acc_gate[q][i] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    const int c = (q * blockDim.x + threadIdx.x) * kSlot;
    if (p.dw_pre) store_slot<true>(p.part_pre + b * p.ldp, c, d - c, pack_slot<true>(acc_pre[q]));
    if (p.dw_post) store_slot<true>(p.part_post + b * p.ldp, c, d - c, pack_slot<true>(acc_post[q]));
  }
}

// Sums of the teams' rows, 64 columns per workgroup: blockIdx.y 0 is dw_pre,
// 1 dw_post, 2 + i the i-th gate group that may span teams.  Sixteen threads
// share four columns, each summing every sixteenth row; the sixteen sums are
// then added in order.
__global__ void __launch_bounds__(256) sum_parts_kernel(BlockNormBwd p, int64_t teams) {
  __shared__ float lds[16][64];
  const int job = blockIdx.y;
  const float* src;
  float* dst;
  int64_t n, first = 0, ld = p.ldp;
  if (job < 2) {
    src = job == 0 ? p.part_pre : p.part_post;
    dst = job == 0 ? p.dw_pre : p.dw_post;
    n = teams;
    if (!dst) return;
  } else {
    int64_t g = job - 2;
    const int64_t groups = ceil_div(p.T, p.gate_every);
    if (groups > teams) g = min(((int64_t)(job - 1) * p.per - 1), p.T - 1) / p.gate_every;  // team's last group
    const int64_t b0 = g * p.gate_every / p.per, b1 = (min((g + 1) * p.gate_every, p.T) - 1) / p.per;
    if (b0 == b1 || (groups > teams && b0 != job - 2)) return;
    src = p.part_gate;
    dst = p.dgate + g * p.d;
    // row 2 b0 + 1, then rows 2b for b in (b0, b1]
    n = b1 - b0 + 1;
    first = b0;
    ld = 0;
  }
  const int col = threadIdx.x & 15, sub = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + col * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < p.ldp) {
    for (int64_t i = sub; i < n; i += 16) {
      const int64_t row = ld ? i : (i == 0 ? 2 * first + 1 : 2 * (first + i));
      const float4 v = *reinterpret_cast<const float4*>(src + row * p.ldp + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  lds[sub][col * 4] = s.x;
  lds[sub][col * 4 + 1] = s.y;
  lds[sub][col * 4 + 2] = s.z;
  lds[sub][col * 4 + 3] = s.w;
  __syncthreads();
  const int out = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x < 64 && out < p.d) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += lds[i][threadIdx.x];
    dst[out] = v;
  }
}

// Threads per row (whole waves) for VPT slots each.
int team_threads(int d, int vpt) { return (int)ceil_div(ceil_div(d, kSlot * vpt), 64) * 64; }

template <bool AF32, bool RF32>
void launch_fwd(const BlockNorm& p, hipStream_t s) {
  const int vpt = p.d <= 1024 * kSlot ? 1 : 2, th = team_threads(p.d, vpt), teams = th == 64 ? 4 : 1;
  const dim3 grid((unsigned)ceil_div(p.T, teams)), block(th, teams);
  if (vpt == 1)
    block_norm_kernel<AF32, RF32, 1><<<grid, block, 0, s>>>(p);
  else
    block_norm_kernel<AF32, RF32, 2><<<grid, block, 0, s>>>(p);
}

template <bool AF32, bool RF32>
void launch_bwd(const BlockNormBwd& p, int64_t teams, hipStream_t s) {
  const int vpt = p.d <= 1024 * kSlot ? 1 : 2, th = team_threads(p.d, vpt), tpb = th == 64 ? 4 : 1;
  const dim3 grid((unsigned)ceil_div(teams, tpb)), block(th, tpb);
  if (vpt == 1)
    block_norm_bwd_kernel<AF32, RF32, 1><<<grid, block, 0, s>>>(p);
  else
    block_norm_bwd_kernel<AF32, RF32, 2><<<grid, block, 0, s>>>(p);
}

constexpr int64_t kMaxTeams = 512;

// Rows of a team: as even as kMaxTeams teams allow.
int64_t rows_per_team(int64_t T) { return ceil_div(T, kMaxTeams); }

}  // namespace

size_t block_norm_scratch_bytes(int64_t T, int d) {
  const int64_t teams = T ? ceil_div(T, rows_per_team(T)) : 0;
  return (size_t)(4 * teams) * (size_t)(ceil_div(d, kSlot) * kSlot) * sizeof(float);
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
  p.ldp = ceil_div(p.d, kSlot) * kSlot;
  p.per = p.T ? rows_per_team(p.T) : 1;
  const int64_t teams = ceil_div(p.T, p.per);  // none for an empty batch: the sums below are zero
  float* part = static_cast<float*>(scratch);
  p.part_pre = part;
  p.part_post = part + teams * p.ldp;
  p.part_gate = part + 2 * teams * p.ldp;
  if (teams == 0)
    ;
  else if (act_f32)
    launch_bwd<true, true>(p, teams, s);
  else if (res_f32)
    launch_bwd<false, true>(p, teams, s);
  else
    launch_bwd<false, false>(p, teams, s);
  const int64_t groups = p.dgate ? ceil_div(p.T, p.gate_every) : 0;
  const unsigned jobs = 2 + (unsigned)(groups < teams ? groups : teams);
  if (p.dw_pre || p.dw_post || p.dgate)
    sum_parts_kernel<<<dim3((unsigned)ceil_div(p.ldp, 64), jobs), 256, 0, s>>>(p, teams);
  return hipGetLastError();
}

}  // namespace moe
