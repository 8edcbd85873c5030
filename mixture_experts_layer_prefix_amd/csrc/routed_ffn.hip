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
// rows against sixteen tokens.  One token through 8 of 256 experts of 7,168 x
// 2,048 takes 36 us for 187 MB (5.3 TB/s, two launches; the gate and up
// projections by themselves 5.7 TB/s), sixteen tokens 377 for 2.4 GB (6.3
// TB/s).  From a mean of some 40 tokens an expert on the weights, read
// once for every 48 tokens, and the tokens, read once for every 128 rows, come
// from L2 with little to hide their way behind (512 tokens of eight, 32 experts:
// 366 us, 1.0 PFLOP/s).
#include <algorithm>
#include <type_traits>

#include "mxfp4.h"
#include "parts.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kWaves = 4;  // of a workgroup, which share the K of a tile
// Routes that a workgroup can look through for its expert's tokens.
constexpr int kDirect = 1024;

// The wave's number in its workgroup, in a scalar register.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Lane l = 16 g + r of the operation feeds weight row r with K[32g, 32g+32)
// and its scale, and token r with K[16g, 16g+16), K[64+16g, 64+16g+16) and the
// scale of block g.  Accumulator element i of the lane is weight row 4g + i,
// token r.  In each eight products along K the operation keeps a product's bits
// down to 2^-13 of the largest only; sums of sixteen then join the accumulator in
// fp32, one after another.  That is a choice: bf16 operations would keep 24 bits,
// but take unpacked operands and four times as many instructions, and the cut is
// far below the 2^-4 to which h is rounded next.  y is as far from 64 bits as with
// products in fp32 (0.0017 of y in the norm either way, 16 tokens, 256 experts of
// 7,168 x 2,048: its own rounding).
__device__ __forceinline__ f32x4 mma(u32x4 w, uint32_t ws, u32x4 lo, u32x4 hi, uint32_t xs, f32x4 acc) {
  const i32x8 a{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i32x8 b{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 0, 0, (int)ws, 0, (int)xs);
}

// Bytes that are read through a buffer address: reads at or past the end (the
// sum of a scalar and a lane's offset) give zeros and cost no traffic.  The
// scalar offset alone never passes the end (part_at()).
struct Bytes {
  const uint8_t* p;
  uint32_t n;
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, (int)n, 0x00027000);
  }
};

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Reads of LDS that came before have arrived.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// What is written before is issued before: waits count loads in their order.
__device__ __forceinline__ void in_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A wave's ring in LDS for 16 * TILES weight rows, a stage for each pair of
// slabs (256 of K).  Codes: direct loads to LDS of eight rows' whole 128-byte
// lines, which the streaming hint needs (1.6 GB read so reach 7.0 TB/s, without
// the hint 6.3; as sixteen rows of half a line with the hint 5.0), and which
// hold no registers while they are under way.  After a schedule, without the
// hint are weights that several workgroups or rounds read, which are to stay in
// L2 (512 tokens of eight, 32 experts of 7,168 x 2,048: 366 us, all with the hint
// 440).  Without a schedule all weights have it: the choice by an expert's tokens
// gains nothing where they take many rounds and costs the others (64 routes at
// one of 256 experts of 7,168 x 2,048, 57.1 us, with the choice 56.9, at random
// ones 202 and 206; 700 at one of 900 of 128 x 256, 123 and 137).  A
// lane's 16 bytes are put in a place turned by its row, so that the reads of
// sixteen rows of a slab meet no bank twice.  Scales: a word per row and slab.
template <int TILES, int STAGES>
struct Ring {
  static constexpr int kCodes = TILES * 2048, kScales = TILES * 128, kStage = kCodes + kScales;
  static constexpr int kMats = TILES >= 2 ? 2 : 1;                    // halves of the rows, from a matrix each
  static constexpr int kRows = 16 * TILES / kMats;                    // of a half
  static constexpr int kScaleLoads = kRows > 32 ? kRows / 32 : 1;     // of a half: 64 words each
  static constexpr int kLoads = TILES * 2 + kMats * kScaleLoads;      // of a stage
  static_assert(kRows <= 64, "a scale load takes whole slabs");
  uint8_t* lds;                    // the wave's ring
  Bytes w[kMats], ws[kMats];       // the halves' codes, scales from their first rows on
  uint32_t even, odd, scale;       // a lane's offsets in eight rows' codes, and in the scales
  uint32_t ld, ws_step;            // bytes of eight rows' codes, between slabs of scales
  uint32_t read, read_scale;       // a lane's place in a stage
  int pairs, slabs;
  bool again;                      // the weights are read more than once

  __device__ __forceinline__ void begin(uint8_t* ring, int K, int64_t all_rows, bool reread) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    lds = ring;
    again = reread;
    slabs = K / 128;
    pairs = (slabs + 1) / 2;
    ld = 4 * K;
    ws_step = (uint32_t)all_rows * 4;
    even = (lane >> 3) * (K / 2) + ((lane & 7) ^ g) * 16;
    odd = (lane >> 3) * (K / 2) + ((lane & 7) ^ (g + 4)) * 16;
    scale = lane % kRows * 4 + lane / kRows * ws_step;
    read = r * 128 + (g ^ (r >> 1)) * 16;
    read_scale = kCodes + r * 4 + g;
  }
  // Half i begins at row `row` of the stacked matrix [all rows][K].
  __device__ __forceinline__ void rows(int i, const uint8_t* codes, const uint8_t* scales, int64_t row, int K) {
    w[i] = {codes + row * (K / 2), (uint32_t)kRows * (K / 2)};
    ws[i] = {scales + row * 4, ws_step * (K / 128) - (uint32_t)row * 4};
  }
  template <int AUX>
  __device__ __forceinline__ void issue_tile(int i, int t, uint8_t* to) const {
    const int m = t / (TILES / kMats), q = t % (TILES / kMats) * 2;
    lds_dma<16, AUX>(w[m].rsrc(), to + t * 2048, even, part_at(i, pairs, i * 128 + q * ld, w[m].n));
    lds_dma<16, AUX>(w[m].rsrc(), to + t * 2048 + 1024, odd,
                     part_at(i, pairs, i * 128 + (q + 1) * ld, w[m].n));
  }
  // Starts the loads of pair i into its stage, whole or in parts: the codes of
  // tile t, the scales.  Past the last pair they read nothing.
  __device__ __forceinline__ void issue(int i, int stage) const {
#pragma unroll
    for (int t = 0; t < TILES; ++t) issue_codes(i, stage, t);
    issue_scales(i, stage);
  }
  __device__ __forceinline__ void issue_codes(int i, int stage, int t) const {
    if (again)
      issue_tile<0>(i, t, lds + stage * kStage);
    else
      issue_tile<2>(i, t, lds + stage * kStage);
  }
  __device__ __forceinline__ void issue_scales(int i, int stage) const {
    uint8_t* to = lds + stage * kStage;
    if (2 * kRows < 64 && (threadIdx.x & 63) >= 2 * kRows) return;
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
      for (int v = 0; v < kScaleLoads; ++v)
        lds_dma<4>(ws[m].rsrc(), to + kCodes + (m * kScaleLoads + v) * 256, scale,
                   part_at(2 * i + v, slabs, (2 * i + v) * ws_step, ws[m].n));
  }
  // Tile m's operand and scale of the stage's slab u.
  __device__ __forceinline__ u32x4 codes(int stage, int m, int u) const {
    return *reinterpret_cast<const u32x4*>(lds + stage * kStage + m * 2048 + (read ^ (u * 64)));
  }
  __device__ __forceinline__ uint32_t scales(int stage, int m, int u) const {
    const int half = m / (TILES / kMats), q = m % (TILES / kMats);
    return lds[stage * kStage + half * (kRows * 8) + u * (kRows * 4) + q * 64 + read_scale];
  }
};

// The dword of lane `from` / 4.
__device__ __forceinline__ uint32_t of_lane(int from, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v);
}
__device__ __forceinline__ u32x4 of_lane(int from, u32x4 v) {
  return u32x4{of_lane(from, v[0]), of_lane(from, v[1]), of_lane(from, v[2]), of_lane(from, v[3])};
}

// Sixteen tokens' part of a pair of slabs.  DEAL: it is loaded with a token's
// 64 bytes in four lanes side by side, which cost the L1 cache one access, and
// then dealt to the lanes that feed it; else as it is fed, where the four lanes
// lie apart and cost four.  Many tokens are bound by these accesses (512 of
// eight, 32 experts of 7,168 x 2,048: 446 us, dealt 366); where an expert has one
// or two the others' lanes load nothing, and dealing only delays the product (5
// tokens, 64 of 2,048 x 768: 21.0 us, dealt 21.5).
template <bool DEAL>
struct TokenPair {
  u32x4 lo[2], hi[2];
  uint32_t xs;  // a token's scales of slab 0 in one of its lanes, of slab 1 in the next
  __device__ __forceinline__ void deal() {
    if constexpr (!DEAL) return;
    const int lane = threadIdx.x & 63, from = (lane & 15) * 16 + (lane >> 4) * 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      lo[u] = of_lane(from, lo[u]);
      hi[u] = of_lane(from, hi[u]);
    }
  }
  // The lane's scale of slab u.
  __device__ __forceinline__ uint32_t scale(int u) const {
    const int lane = threadIdx.x & 63;
    return of_lane(DEAL ? (lane & 15) * 16 + u * 4 : (lane & 15) * 4 + u * 64, xs) >> ((lane >> 4) * 8);
  }
};

// Tokens [][K] in E4M3 and their scales.
template <bool DEAL>
struct Tokens {
  Bytes x, xs;
  int K;
  // Which of sixteen tokens a lane loads, and which quarter of its 64 bytes.
  __device__ static __forceinline__ int token() { return DEAL ? (threadIdx.x & 63) >> 2 : threadIdx.x & 15; }
  __device__ static __forceinline__ int quarter() { return DEAL ? threadIdx.x & 3 : (threadIdx.x & 63) >> 4; }
  __device__ __forceinline__ uint32_t offset(bool on, uint32_t row) const {
    return on ? row * K + quarter() * 16 : x.n;
  }
  __device__ __forceinline__ uint32_t scale_offset(bool on, uint32_t row) const {
    return on ? row * (K / 32) + quarter() % 2 * 4 : xs.n;
  }
  // Pair i; past the last pair nothing is read.  The second slab of an odd last
  // pair is not used.
  __device__ __forceinline__ void load(int i, uint32_t o, uint32_t so, TokenPair<DEAL>& t) const {
    const int pairs = (K + 255) / 256;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t at = part_at(i, pairs, i * 256 + u * 128, x.n);
      t.lo[u] = __builtin_amdgcn_raw_buffer_load_b128(x.rsrc(), o, at, 0);
      t.hi[u] = __builtin_amdgcn_raw_buffer_load_b128(x.rsrc(), o + 64, at, 0);
    }
    t.xs = __builtin_amdgcn_raw_buffer_load_b32(xs.rsrc(), so, part_at(i, pairs, i * 8, xs.n), 0);
  }
};

// LDS of a workgroup: the waves' rings of one stage, and after a tile's product
// its sums; and the routes of a DIRECT workgroup.  One object, whatever it
// holds: between several the compiler tells the loads to LDS apart and waits
// for all of them before each read.
template <int TILES, int NT, bool DIRECT>
struct Shared {
  typedef Ring<TILES, 1> R;
  static constexpr int kAtOnce = TILES == 8 ? 2 : NT;  // tokens' tiles whose sums LDS holds at a time
  static constexpr int kPart = 1024 * TILES * kAtOnce, kWave = R::kStage > kPart ? R::kStage : kPart;
  int32_t list[DIRECT ? kDirect : 1], found[DIRECT ? kDirect / 256 : 1][kWaves];
  uint8_t bytes[kWaves * kWave] __attribute__((aligned(16)));

  __device__ __forceinline__ uint8_t* wave(int w) { return bytes + w * kWave; }

  // The same by each wave for itself, without a barrier, for up to 64 routes;
  // id: the lane's.  The wave's list begins at 64 * wave.
  __device__ __forceinline__ int find_few(int32_t id, int e, int mine) {
    const int lane = threadIdx.x & 63;
    const uint64_t m = __ballot(id == e), before = (1ull << lane) - 1;
    if (m & ((1ull << mine) - 1)) return 0;
    if ((m >> lane) & 1) list[64 * wave_id() + __popcll(m & before)] = lane;
    in_order();
    return __popcll(m);
  }
  // The routes of expert e, in order, into `list`; id: the thread's ids of the
  // routes threadIdx.x, 256 + threadIdx.x, ...  Their number, or 0 if one comes
  // before route `mine`.
  __device__ __forceinline__ int find(const int32_t (&id)[kDirect / 256], int e, int mine) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    uint64_t m[kDirect / 256];
#pragma unroll
    for (int q = 0; q < kDirect / 256; ++q) {
      m[q] = __ballot(id[q] == e);
      const bool early = __any(id[q] == e && q * 256 + (int)threadIdx.x < mine);
      if (lane == 0) found[q][wave] = early ? -65536 : __popcll(m[q]);
    }
    __syncthreads();
    int count = 0;
    bool early = false;
#pragma unroll
    for (int q = 0; q < kDirect / 256; ++q) {
      for (int w = 0; w < kWaves; ++w) {
        const int n = found[q][w];
        early |= n < 0;
        if (w == wave && !early && ((m[q] >> lane) & 1))
          list[count + __popcll(m[q] & ((1ull << lane) - 1))] = q * 256 + (int)threadIdx.x;
        count += n;
      }
    }
    __syncthreads();
    return early ? 0 : count;
  }

  // acc[m][n] += the slab pairs first, first + kWaves, ... of 16 * TILES rows
  // and N (up to NT) times sixteen tokens; the first pair's weights are under
  // way.  No barrier: the ring is the wave's own.  One pair of each wave is in
  // flight, a tile's codes of the next one as soon as the tile's operand is in
  // registers: 8.5 or 17 KB, 139 KB on a compute unit with the
  // sixteen or eight waves that fit.  Two stages of half as many waves took 2%
  // longer (16 tokens, 256 experts of 7,168 x 2,048).
  template <int N>
  __device__ __forceinline__ void product_of(const R& ring, const Tokens<!DIRECT>& x, const uint32_t (&xo)[NT],
                                             const uint32_t (&xso)[NT], int first, f32x4 (&acc)[TILES][NT]) const {
    const bool odd = (x.K / 128) & 1;
    TokenPair<!DIRECT> t[N];
#pragma unroll
    for (int n = 0; n < N; ++n) x.load(first, xo[n], xso[n], t[n]);
    for (int i = first; i < ring.pairs; i += kWaves) {
      in_order();
      wait_loads<0>();
      in_order();
      uint32_t xs[N][2];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        t[n].deal();
        xs[n][0] = t[n].scale(0);
        xs[n][1] = t[n].scale(1);
      }
      const bool two = !(odd && i + 1 == ring.pairs);  // slabs
      u32x4 w[2][2];
      uint32_t ws[2][2];
      auto read = [&](int m) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          w[m & 1][u] = ring.codes(0, m, u);
          ws[m & 1][u] = ring.scales(0, m, u);
        }
      };
      read(0);
#pragma unroll
      for (int m = 0; m < TILES; ++m) {
        in_order();
        wait_lds();
        in_order();
        ring.issue_codes(i + kWaves, 0, m);
        in_order();
        if (m + 1 < TILES) read(m + 1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (u == 1 && !two) break;
#pragma unroll
          for (int n = 0; n < N; ++n)
            acc[m][n] = mma(w[m & 1][u], ws[m & 1][u], t[n].lo[u], t[n].hi[u], xs[n][u], acc[m][n]);
        }
      }
      in_order();
#pragma unroll
      for (int n = 0; n < N; ++n) x.load(i + kWaves, xo[n], xso[n], t[n]);
      ring.issue_scales(i + kWaves, 0);
    }
    in_order();
    wait_loads<0>();  // the ring is free again
    in_order();
  }
  // The first `tiles` times sixteen tokens, NT at most: a product for each
  // number, without tests between the matrix operations.
  __device__ __forceinline__ void product(const R& ring, const Tokens<!DIRECT>& x, const uint32_t (&xo)[NT],
                                          const uint32_t (&xso)[NT], int first, int tiles,
                                          f32x4 (&acc)[TILES][NT]) const {
    if (NT >= 3 && tiles >= 3)
      product_of<NT>(ring, x, xo, xso, first, acc);
    else if (NT >= 2 && tiles >= 2)
      product_of<NT < 2 ? NT : 2>(ring, x, xo, xso, first, acc);
    else
      product_of<1>(ring, x, xo, xso, first, acc);
  }
  // Where a wave's sum of rows 4 j to 4 j + 3 for token r of tokens' tile n
  // lies.  The token's place is turned by j, so that neither neighbouring j of
  // a token nor neighbouring tokens of a j meet in one bank when they are read.
  __device__ __forceinline__ int place(int n, int j, int r) const {
    return ((j / 4) * kAtOnce + n) * 64 + (j % 4) * 16 + (r ^ (j & 15) ^ ((j & 1) << 3));
  }
  // The sums of the tokens' tiles from n0 on.
  __device__ __forceinline__ void put(int w, int n0, const f32x4 (&acc)[TILES][NT]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int m = 0; m < TILES; ++m)
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n)
        if (n0 + n < NT)
          reinterpret_cast<f32x4*>(wave(w))[place(n, 4 * m + (lane >> 4), lane & 15)] = acc[m][n0 + n];
  }
  // Rows 4 j to 4 j + 3 of the tile for token r of tokens' tile n0 + n, the waves' sums in order.
  __device__ __forceinline__ f32x4 get(int n, int j, int r) {
    f32x4 v = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += reinterpret_cast<const f32x4*>(wave(w))[place(n, j, r)];
    return v;
  }
};

// Which rows of a matrix a tile kernel's workgroup serves.  DIRECT: workgroup
// (., i) serves the expert of route i if no earlier route has it, and finds the
// others by reading all ids; h and o have a row per route.  ALONE: sixteen
// routes at most, of which hardly any shares its expert.  Else workgroup
// (., e) serves expert e after the sort's schedule, whose rows h and o have.
template <bool DIRECT, bool ALONE>
struct Served {
  int e, first, count;
  int tile, part, parts;  // of the columns; of the tokens, and how many there are
  int32_t id[kDirect / 256];
  bool few;                 // routes: each wave finds them by itself

  // False: there is nothing to do.
  __device__ __forceinline__ bool begin(const RoutedFfn& p, const int32_t* offsets, int tiles) {
    tile = blockIdx.x;
    part = 0;
    parts = 1;
    if constexpr (DIRECT) {
      e = p.topk_idx[blockIdx.y];
      first = 0;
      count = 1;  // at least, until find()
      const int routes = (int)p.T * p.k;
      few = ALONE || routes <= 64;
      if ((unsigned)e >= (unsigned)p.E) return false;
#pragma unroll
      for (int q = 0; q < kDirect / 256; ++q) {
        const int i = q * 256 + (few ? (int)threadIdx.x & 63 : (int)threadIdx.x);
        id[q] = i < routes ? p.topk_idx[i] : -1;
      }
      in_order();  // waited for behind the first weights, these would wait for them too
      return true;
    } else {
      // The parts behind the last token come last: one beside another they
      // would leave every second compute unit without work (parts of a tile in
      // turn: 209 us where this takes 142, 2,048 routes of which 256 are here).
      e = blockIdx.y;
      parts = gridDim.x / tiles;
      part = blockIdx.x / tiles;
      tile = blockIdx.x % tiles;
      first = offsets[e];
      count = offsets[e + 1] - first;
      return true;
    }
  }
  // The first weights are under way while the tokens are found; without a
  // schedule only up to sixteen routes of no fewer experts, as of more many
  // workgroups find that they have none and have read for nothing.  us, after
  // and before the tokens are found (routes, experts of d x I, random ids):
  //   12, 64 of 2,048 x 768       15.8 15.1    24, 256 of 7,168 x 2,048   87.3 87.6
  //   18                          15.0 14.8    64                         206  211
  //   30                          19.5 19.3    64, 128 of 4,096 x 1,536   93.0 98.1
  //   48                          25.0 25.9    32, one a token, 64 of
  //   60                          31.6 32.8      2,048 x 768              20.8 20.3
  // 64 routes at one of 256 experts of 7,168 x 2,048: 57.1 and 67.2.
  template <class S, class Issue>
  __device__ __forceinline__ bool start(S& shared, Issue issue) {
    if constexpr (!DIRECT || ALONE) {
      issue();
      return find(shared);
    } else {
      if (!find(shared)) return false;
      issue();
      return true;
    }
  }
  template <class S>
  __device__ __forceinline__ bool find(S& shared) {
    if constexpr (DIRECT) {
      if (ALONE || few)
        count = shared.find_few(id[0], e, blockIdx.y);
      else
        count = shared.find(id, e, blockIdx.y);
      if (few) first = 64 * wave_id();
      if (count == 0) wait_loads<0>();  // no load may reach LDS that is another workgroup's by then
    }
    return count > 0;
  }
  template <class S>
  __device__ __forceinline__ int row(const S& shared, int i) const {
    return DIRECT ? shared.list[first + i] : first + i;
  }
};

// 8 * TILES columns of h for an expert's tokens.
template <int TILES, int NT, bool DIRECT, bool ALONE>
__global__ void __launch_bounds__(256, 2) gate_up_kernel(RoutedFfn p, const int32_t* __restrict__ offsets,
                                                         const int32_t* __restrict__ row_token,
                                                         uint8_t* __restrict__ h, uint8_t* __restrict__ h_scale) {
  __shared__ Shared<TILES, NT, DIRECT> shared;
  constexpr int kCols = 8 * TILES, kAtOnce = Shared<TILES, NT, DIRECT>::kAtOnce;
  const int lane = threadIdx.x & 63, wave = wave_id();
  Served<DIRECT, ALONE> my;
  if (!my.begin(p, offsets, p.I / kCols) || my.part * 16 * NT >= my.count) return;
  const int c0 = my.tile * kCols;
  Ring<TILES, 1> ring;
  ring.begin(shared.wave(wave), p.d, (int64_t)p.E * p.I, !DIRECT && my.count > 16 * NT);
  ring.rows(0, p.w.q_gate, p.w.q_gate_scale, (int64_t)my.e * p.I + c0, p.d);
  ring.rows(1, p.w.q_up, p.w.q_up_scale, (int64_t)my.e * p.I + c0, p.d);
  if (!my.start(shared, [&] { ring.issue(wave, 0); })) return;
  const Tokens<!DIRECT> x{{p.x, (uint32_t)(p.T * p.d)}, {p.x_scale, (uint32_t)(p.T * (p.d / 32))}, p.d};
  for (int n0 = my.part * 16 * NT; n0 < my.count; n0 += my.parts * 16 * NT) {
    if (n0 > my.part * 16 * NT) ring.issue(wave, 0);
    uint32_t xo[NT], xso[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int i = n0 + 16 * n + x.token();
      const bool on = i < my.count;
      const int row = on ? my.row(shared, i) : 0;
      const uint32_t t = !on ? 0 : DIRECT ? row / p.k : row_token[row];
      xo[n] = x.offset(on, t);
      xso[n] = x.scale_offset(on, t);
    }
    f32x4 acc[TILES][NT] = {};
    shared.product(ring, x, xo, xso, wave, (my.count - n0 + 15) / 16, acc);
#pragma unroll
    for (int n1 = 0; n1 < NT; n1 += kAtOnce) {
      shared.put(wave, n1, acc);
      __syncthreads();
      // eight lanes per token and 32 columns, four columns each
      for (int q = threadIdx.x >> 3; q < 16 * kAtOnce * (kCols / 32); q += 32) {
        const int token = q % (16 * kAtOnce), j = q / (16 * kAtOnce) * 8 + (lane & 7), i = n0 + 16 * n1 + token;
        if (i >= min(my.count, n0 + 16 * NT)) continue;
        const f32x4 gate = shared.get(token >> 4, j, token & 15);
        const f32x4 up = shared.get(token >> 4, kCols / 4 + j, token & 15);
        float z[4];
        uint32_t mx = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          z[v] = silu_f32(gate[v]) * up[v];
          mx = max(mx, __float_as_uint(z[v]) & 0x7FFFFFFFu);
        }
        mx = max(mx, dpp_u32<0xB1>(mx));   // lane ^ 1
        mx = max(mx, dpp_u32<0x4E>(mx));   // lane ^ 2
        mx = max(mx, dpp_u32<0x141>(mx));  // the other four of eight lanes
        const int be = mx_block_exp_bits(mx);
        const float inv = mx_inv_scale(be);
        const int64_t row = my.row(shared, i);
        *reinterpret_cast<uint32_t*>(h + row * p.I + c0 + 4 * j) =
            e4m3x4_rne_sat(z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv);
        if (j % 8 == 0) h_scale[row * (p.I / 32) + (c0 + 4 * j) / 32] = (uint8_t)(be + 127);
      }
      __syncthreads();
    }
  }
}

// 16 * TILES columns of o for an expert's tokens.
template <int TILES, int NT, bool DIRECT, bool ALONE>
__global__ void __launch_bounds__(256, 2) down_kernel(RoutedFfn p, const int32_t* __restrict__ offsets,
                                                      const uint8_t* h, const uint8_t* h_scale,
                                                      float* __restrict__ o) {
  __shared__ Shared<TILES, NT, DIRECT> shared;
  constexpr int kCols = 16 * TILES, kAtOnce = Shared<TILES, NT, DIRECT>::kAtOnce;
  const int wave = wave_id();
  Served<DIRECT, ALONE> my;
  if (!my.begin(p, offsets, p.d / kCols) || my.part * 16 * NT >= my.count) return;
  const int c0 = my.tile * kCols;
  Ring<TILES, 1> ring;
  ring.begin(shared.wave(wave), p.I, (int64_t)p.E * p.d, !DIRECT && my.count > 16 * NT);
  ring.rows(0, p.w.q_down, p.w.q_down_scale, (int64_t)my.e * p.d + c0, p.I);
  ring.rows(1, p.w.q_down, p.w.q_down_scale, (int64_t)my.e * p.d + c0 + kCols / 2, p.I);
  if (!my.start(shared, [&] { ring.issue(wave, 0); })) return;
  const Tokens<!DIRECT> x{{h, (uint32_t)(p.T * p.k * p.I)}, {h_scale, (uint32_t)(p.T * p.k * (p.I / 32))}, p.I};
  for (int n0 = my.part * 16 * NT; n0 < my.count; n0 += my.parts * 16 * NT) {
    if (n0 > my.part * 16 * NT) ring.issue(wave, 0);
    uint32_t xo[NT], xso[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int i = n0 + 16 * n + x.token();
      const bool on = i < my.count;
      const uint32_t row = on ? my.row(shared, i) : 0;
      xo[n] = x.offset(on, row);
      xso[n] = x.scale_offset(on, row);
    }
    f32x4 acc[TILES][NT] = {};
    shared.product(ring, x, xo, xso, wave, (my.count - n0 + 15) / 16, acc);
#pragma unroll
    for (int n1 = 0; n1 < NT; n1 += kAtOnce) {
      shared.put(wave, n1, acc);
      __syncthreads();
      // four columns of a token each
      for (int q = threadIdx.x; q < 16 * kAtOnce * (kCols / 4); q += 256) {
        const int j = q % (kCols / 4), token = q / (kCols / 4), i = n0 + 16 * n1 + token;
        if (i < min(my.count, n0 + 16 * NT))
          *reinterpret_cast<f32x4*>(o + (int64_t)my.row(shared, i) * p.d + c0 + 4 * j) =
              shared.get(token >> 4, j, token & 15);
      }
      __syncthreads();
    }
  }
}

constexpr int kDownWaves = 8;
// Two stages let four workgroups onto a compute unit (four stages two of them,
// with as much in flight: 4 tokens, 256 experts of 7,168 x 2,048, 120.4 us, with
// two 113.4; 5 tokens, 64 of 2,048 x 768, 23.9, 21.1).
constexpr int kTokenStages = 2;

// A token's sixteen columns of y, h with a row per route: each wave takes the
// routes wave, wave + waves, ... with all of K, and the weighted sum runs over
// the routes in slot order.  Sums are made as in down_kernel, in kWaves chains
// of slab pairs, so that a token's bits do not depend on which of the two it
// went through.  Workgroups are numbered so that an XCD takes neighbouring
// columns, whose scales share lines, and all tokens of the same columns one
// after another: an expert that several of them chose is read into its L2 once.
__global__ void __launch_bounds__(64 * kDownWaves, 4) down_token_kernel(RoutedFfn p, const uint8_t* h,
                                                                        const uint8_t* h_scale) {
  typedef Ring<1, kTokenStages> R;
  // a stage of the token: 256 bytes of h, 8 scales
  constexpr int kRing = kTokenStages * R::kStage, kToken = 272;
  __shared__ struct {
    uint8_t rings[kDownWaves][kRing + kTokenStages * kToken] __attribute__((aligned(16)));
    float part[16][16];
  } shared;
  const int lane = threadIdx.x & 63, wave = wave_id(), waves = blockDim.x >> 6, r = lane & 15, g = lane >> 4;
  const int T = (int)p.T, xcd = blockIdx.x % 8, i = blockIdx.x / 8;
  const int t = i % T, c0 = (xcd * (p.d / 128) + i / T) * 16;
  const bool odd = (p.I / 128) & 1;
  uint8_t* lds = shared.rings[wave];
  R ring;
  ring.begin(lds, p.I, (int64_t)p.E * p.d, false);
  for (int j = wave; j < p.k; j += waves) {
    const int e = __builtin_amdgcn_readfirstlane(p.topk_idx[t * p.k + j]);
    if ((unsigned)e >= (unsigned)p.E) continue;
    ring.rows(0, p.w.q_down, p.w.q_down_scale, (int64_t)e * p.d + c0, p.I);
    const int64_t row = t * p.k + j;
    const Bytes x{h + row * p.I, (uint32_t)p.I}, xs{h_scale + row * (p.I / 32), (uint32_t)p.I / 32};
    auto issue = [&](int i, int u) {
      uint8_t* to = lds + kRing + u * kToken;
      ring.issue(i, u);
      if (lane < 16) lds_dma<16>(x.rsrc(), to, lane * 16, part_at(i, ring.pairs, i * 256, x.n));
      if (lane < 2) lds_dma<4>(xs.rsrc(), to + 256, lane * 4, part_at(i, ring.pairs, i * 8, xs.n));
    };
    f32x4 acc[kWaves] = {};
    auto multiply = [&](int u, int stage, int slab) {
      const uint8_t* x = lds + kRing + stage * kToken + slab * 128 + 16 * g;  // the token in every column
      acc[u] = mma(ring.codes(stage, 0, slab), ring.scales(stage, 0, slab), *reinterpret_cast<const u32x4*>(x),
                   *reinterpret_cast<const u32x4*>(x + 64), lds[kRing + stage * kToken + 256 + slab * 4 + g], acc[u]);
    };
#pragma unroll
    for (int u = 0; u < kTokenStages; ++u) {
      in_order();
      issue(u, u);
    }
    for (int q = 0; q < ring.pairs; q += kWaves) {
#pragma unroll
      for (int u = 0; u < kWaves; ++u) {
        in_order();
        wait_loads<(kTokenStages - 1) * (R::kLoads + 2)>();
        in_order();
        if (q + u < ring.pairs) multiply(u, u % kTokenStages, 0);
        if (q + u + (odd ? 1 : 0) < ring.pairs) multiply(u, u % kTokenStages, 1);
        in_order();
        issue(q + u + kTokenStages, u % kTokenStages);
      }
    }
    in_order();
    wait_loads<0>();  // the ring is free again
    in_order();
    f32x4 v = {};
#pragma unroll
    for (int u = 0; u < kWaves; ++u) v += acc[u];
    if (r == 0) *reinterpret_cast<f32x4*>(&shared.part[j][4 * g]) = v;
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    const int64_t at = (int64_t)t * p.d + c0 + threadIdx.x;
    float v = 0.0f;
    for (int j = 0; j < p.k; ++j)
      if ((unsigned)p.topk_idx[t * p.k + j] < (unsigned)p.E) v = fmaf(p.topk_w[t * p.k + j], shared.part[j][threadIdx.x], v);
    if (p.y_add) v += bf16_to_f32(p.y_add[at]);
    p.y[at] = f32_to_bf16(v);
  }
}

// y[t] = y_add[t] + sum_j w_j o[row_j] over the present routes in slot order;
// DIRECT: o has a row per route.  The rows of eight routes are in flight before
// the first is added.
template <bool DIRECT>
__global__ void __launch_bounds__(256) weighted_sum_kernel(RoutedFfn p, const int32_t* __restrict__ token_row,
                                                           const float* __restrict__ o) {
  constexpr int kRoutes = 8;
  const int per = (p.d + 1023) / 1024;  // workgroup steps of a token
  const int32_t* ids = DIRECT ? p.topk_idx : token_row;
  for (int64_t b = blockIdx.x; b < p.T * per; b += gridDim.x) {
    const int t = (int)(b / per), c = ((int)(b - (int64_t)t * per) * 256 + (int)threadIdx.x) * 4;
    if (c >= p.d) continue;
    Slot<false, 4> add;
    if (p.y_add) add = load_slot<false, false, false, 4>(p.y_add, (int64_t)t * p.d + c, 4);
    f32x4 acc = {};
    for (int j0 = 0; j0 < p.k; j0 += kRoutes) {
      bool here[kRoutes];
      f32x4 v[kRoutes];
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        const int r = t * p.k + j0 + j, id = j0 + j < p.k ? ids[r] : -1;
        here[j] = DIRECT ? (unsigned)id < (unsigned)p.E : id >= 0;
        if (here[j]) v[j] = *reinterpret_cast<const f32x4*>(o + (int64_t)(DIRECT ? r : id) * p.d + c);
      }
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        if (!here[j]) continue;
        const float g = p.topk_w[t * p.k + j0 + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(g, v[j][i], acc[i]);
      }
    }
    if (p.y_add) {
      float v[4];
      unpack_slot(add, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += v[i];
    }
    const float out[4] = {acc[0], acc[1], acc[2], acc[3]};
    store_slot<false, false, false, 4>(p.y, (int64_t)t * p.d + c, 4, pack_slot<false>(out));
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

// With or without a schedule.  Without one there is a workgroup for every route,
// which finds its expert's tokens by itself, sixteen at a time, or that an earlier
// route has the expert: some R^2 / 2E of R at random, weighed here by the
// workgroups of a route.  us (tokens, experts of d x I, k: without, with):
//   1, 8 of 256 of 7,168 x 2,048    37.0 -      10, 64 of 2,048 x 768, 6   31.6  39.2
//   8, 256, 8                      205.6 220.3  14                         41.1  44.5
//   16                             380.9 377.2  20                         48.2  46.3
//   12, 8 of 4,096 x 1,536, 2       29.7 28.1   16, 8 of 2,048 x 768, 2    18.1  20.9
// Up to sixteen routes are one tile of tokens whatever they share, and the
// schedule is never worth its launches (16 tokens, one expert of 7,168 x 2,048:
// 22.9, 26.5).
constexpr int64_t kTwice = 500000;

// Which down projection, without a schedule.  By token it needs no sum of its
// own, which saves a launch and o's way through memory, but reads an expert anew
// for every token that chose it, weighed here in weights, and a token's routes
// are its waves (one route: 32 tokens, 64 experts of 2,048 x 768, 25.9, by expert
// 22.3).  us (tokens, experts of d x I, k: by token, by expert):
//   2, 256 of 7,168 x 2,048, 8      62.3 68.0   10, 64 of 2,048 x 768, 6   31.6  31.8
//   4                              112.1 115.6  14                         41.1  42.7
//   8                              208.2 205.6  6, 16 of 4,096 x 1,536, 4  35.5  33.5
//   8, 128 of 4,096 x 1,536, 8      92.5 90.3   32, 512 of 2,048 x 512, 8  86.8  90.6
constexpr int64_t kRepeats = 200000000;

// Which tiles, after the schedule.  An expert's tokens are shared by as many
// workgroups as the mean calls for (512 tokens, one expert of 7,168 x 2,048: 220
// us with one, 59 with eleven).
//   128 weight rows against 48 tokens, from a mean of 24 tokens an expert on:
//     most experts' tokens are then together and their weights read once (32
//     experts of 7,168 x 2,048, 128 tokens of eight: 165 us, with 32 tokens at a
//     time 215; 96 tokens 151 and 149).
//   128 against 32: each token read half as often as by 64 rows (333 tokens, 128
//     experts of 4,096 x 1,536: 260 us, 280).
//   64 against 32 where workgroups are few, for twice as many (64 tokens, one
//     expert of 7,168 x 2,048: 27.3 us, by 128 rows 32.2; 16 tokens, 8 of 4,096 x
//     1,536: 28.6, 30.3).
constexpr int64_t kManyTokens = 24, kFewGroups = 512;

hipError_t launch_routed_ffn(const RoutedFfn& p, void* scratch, hipStream_t s) {
  const Scratch b = carve(static_cast<char*>(scratch), p.T, p.d, p.E, p.k, p.I);
  const int64_t R = p.T * p.k, steps = p.T * ceil_div(p.d, 1024);
  const unsigned sums = (unsigned)(steps < 65536 ? steps : 65536);
  if (R <= 16 || (R <= kDirect && R * R * (2 * p.I + p.d) / p.E <= kTwice)) {
    const unsigned routes = (unsigned)R;
    const bool alone = R <= 16 && R <= p.E;  // hardly a route shares its expert
    const auto gate_up = alone ? gate_up_kernel<4, 1, true, true> : gate_up_kernel<4, 1, true, false>;
    gate_up<<<dim3(p.I / 32, routes), 256, 0, s>>>(p, nullptr, nullptr, b.h, b.h_scale);
    if (p.T == 1 || (p.k > 1 && R * R * p.I * p.d / p.E <= kRepeats)) {
      const int waves = p.k < kDownWaves ? p.k : kDownWaves;
      down_token_kernel<<<(unsigned)(p.T * (p.d / 16)), 64 * waves, 0, s>>>(p, b.h, b.h_scale);
      return hipGetLastError();
    }
    const auto down = alone ? down_kernel<4, 1, true, true> : down_kernel<4, 1, true, false>;
    down<<<dim3(p.d / 64, routes), 256, 0, s>>>(p, nullptr, b.h, b.h_scale, b.o);
    weighted_sum_kernel<true><<<sums, 256, 0, s>>>(p, nullptr, b.o);
    return hipGetLastError();
  }
  const hipError_t e = launch_sort(false, p.topk_idx, nullptr, p.T, p.d, p.E, p.k, b.counts, b.offsets, b.row_token,
                                   b.token_row, nullptr, b.sort, s);
  if (e != hipSuccess) return e;
  const int64_t most = (1 << 22) / (p.I / 32 + p.d / 64);  // workgroups in x: threads stay below 2^32
  auto parts = [&](int nt) {
    return std::max<int64_t>(1, std::min<int64_t>({ceil_div(R, (int64_t)p.E * 16 * nt), most, 64}));
  };
  auto groups = [&](int nt) { return p.E * (p.I / 64) * parts(nt); };
  auto run = [&](auto TILES, auto NT) {
    constexpr int t = TILES.value, nt = NT.value;
    const int64_t n = parts(nt);
    gate_up_kernel<t, nt, false, false><<<dim3((unsigned)(p.I / (8 * t) * n), (unsigned)p.E), 256, 0, s>>>(
        p, b.offsets, b.row_token, b.h, b.h_scale);
    down_kernel<t, nt, false, false><<<dim3((unsigned)(p.d / (16 * t) * n), (unsigned)p.E), 256, 0, s>>>(
        p, b.offsets, b.h, b.h_scale, b.o);
  };
  constexpr std::integral_constant<int, 2> two;
  constexpr std::integral_constant<int, 3> three;
  constexpr std::integral_constant<int, 4> four;
  constexpr std::integral_constant<int, 8> eight;
  if (R >= kManyTokens * p.E && groups(three) >= kFewGroups)
    run(eight, three);
  else if (groups(two) >= kFewGroups)
    run(eight, two);
  else
    run(four, two);
  weighted_sum_kernel<false><<<sums, 256, 0, s>>>(p, b.token_row, b.o);
  return hipGetLastError();
}

}  // namespace moe
