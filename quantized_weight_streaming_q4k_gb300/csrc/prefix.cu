// prefix.cu -- one decode step's attention for a batch whose sequences share a
// prefix: sequence b's query heads attend to the n_prefix positions of ONE
// shared cache and then to the n_ctx[b] positions of its own,
//   s_t = softcap(scale * q_bh . k_t),  out_bh = sum_t softmax(s)_t v_t
// over both; a row with no position at all gives zeros.
//
// The shared part is computed once for all: the rows of all sequences that
// read a kv head form row tiles against each piece of the shared cache, so the
// cache is read once per row tile and not once per sequence.  The own parts are
// a few rows against many keys, read once.  Each piece leaves a partial result
// (running max, sum, unnormalised output); a last kernel joins them in a fixed
// order.
#include <cuda_runtime.h>

#include <algorithm>

#include "attend_mma.cuh"
#include "attend_rows.cuh"
#include "launch.h"

namespace qws {

__device__ unsigned g_err_prefix;

constexpr int kOwnWarps = 8, kOwnKeys = 4;
constexpr int kOwnChunk = kOwnWarps * kOwnKeys;     // keys of an own-cache item
constexpr int kMaxBatch = 256;      // sequences of one launch

struct PrefixParams {
  qws_heads q, out;
  const float *kp, *vp, *kc, *vc;
  float* part;          // [prefix piece][kv head][row], then [own item][kv head][group]
  float* own;
  int64_t max_prefix, max_seq;
  int b0, batch;        // sequences b0 .. b0 + batch - 1 of the call
  int n_q, n_kv, group;
  int n_prefix, chunk, pieces, row_tiles;
  int beside;           // the own parts run beside the shared part
  float scale, cap;
  int n_ctx[kMaxBatch];
  int first[kMaxBatch + 1];   // first own item of each sequence
};

template <int kPL>
__device__ __forceinline__ int64_t prefix_part(const PrefixParams& p, int piece, int g,
                                               int row) {
  return ((static_cast<int64_t>(piece) * p.n_kv + g) * (p.batch * p.group) + row) *
         (kPL * 32 + kPartPad);
}

// ------------------------------------------------------------ tensor cores
// The shared part of 128 rows of one kv head against one piece of the prefix, on
// the core of attend_mma.cuh.  The prefix is read once, as f32, straight from the cache:
// a loader copies runs of rows into a staging ring, eight converter warps scale, split
// and lay them out for the tensor cores.  Bound by that read (8 * head_dim bytes a key
// and kv head; at head_dim 256 a tile of 64 keys is 128 KB, about 5800 cycles of an
// SM's share of the memory, against 3100 cycles of MMAs).
//
// The converters bound it next (with a maximum over every row and a scale of its own
// they took 12200 cycles a tile).  So a piece has one scale for its keys and one for its
// values, taken from its first run of rows: that run's largest value at [2^7, 2^8).
// Rows whose largest scaled value is in [2^-3, 65504], or zero, keep 22 bits with it, which
// one vote checks; the others, 2^8 times larger or 2^10 times smaller than that run, are
// rare.  Such a key gets a scale of its own.  A tile with such a value row is laid out once
// more, with a scale of its own, which the tile after next goes on with, by a warp that is
// there for this (prefix_refit).  64 rows against 32768 keys of 4 heads of 256: 69 us, 3.9 TB/s
// (268 MB at the copy rate: 40 us), some 8000 cycles a tile.
template <int kHd>
struct PrefixCfg : MmaCfg<kHd, (kHd > 128 ? 1 : kHd > 64 ? 2 : 4), true, 1> {
  using Base = MmaCfg<kHd, (kHd > 128 ? 1 : kHd > 64 ? 2 : 4), true, 1>;
  static constexpr int kDepth = kHd > 128 ? 1 : kHd > 64 ? 2 : 4;   // tiles of a ring
  static constexpr int kConvWarps = 8;
  static constexpr int kConv = Base::kRowsWarps + 4;        // first converter warp
  static constexpr int kThreads = 32 * (kConv + kConvWarps);
  static constexpr int kRun = kHd >= 64 ? 4096 / kHd : 64;  // rows of a staging stage
  static constexpr int kRuns = kTileKeys / kRun;            // stages of K or V of a tile
  static constexpr int kRunRows = kRun / kConvWarps;        // of a stage, a warp's
  static constexpr uint32_t kRunBytes = kRun * kHd * 4;
  static constexpr int kStaging = 5;
};
constexpr int kMaxPieceTiles = 64;

template <int kHd>
struct PrefixShared {
  uint64_t stg_full[PrefixCfg<kHd>::kStaging], stg_empty[PrefixCfg<kHd>::kStaging];
  uint64_t v_done[2];                // the converters are done with a slot's values
  uint32_t left_out[kMaxPieceTiles][2];
  uint32_t misfit[kMaxPieceTiles];   // the scale in force did not fit the tile's values
  float scale[2][2];                 // in force, of the keys and of the values of a slot
  float vmax[2][PrefixCfg<kHd>::kConvWarps];
  MmaShared<PrefixCfg<kHd>> mma;
};

// 640 threads, 96 registers each at launch; per scheduler 2 softmax warps at 160, a
// helper at 48 and 2 converters at 56: 2 x 160 + 48 + 2 x 56 of 5 x 96.

template <int kHd>
__device__ __forceinline__ void prefix_load(PrefixShared<kHd>& sh, uint8_t* staging,
                                            const float* K, const float* V, int keys, int n) {
  using Cfg = PrefixCfg<kHd>;
  const uint64_t pol = l2_policy_evict_first();
  RingAt<Cfg::kStaging> at;
  int units = 0;
  bool ok = true;
  for (int j = 0; j < n && ok; ++j)
    for (int half = 0; half < 2 && ok; ++half)
      for (int r = 0; r < Cfg::kRuns && ok; ++r) {
        const int key = j * kTileKeys + r * Cfg::kRun, rows = min(Cfg::kRun, keys - key);
        if (rows <= 0) continue;
        ok = mbar_wait(&sh.stg_empty[at.stage], at.phase ^ 1u);
        if (!ok) break;
        const uint32_t bytes = static_cast<uint32_t>(rows) * kHd * 4u;
        mbar_arrive_expect_tx(&sh.stg_full[at.stage], bytes);
        bulk_copy_g2s(staging + at.stage * Cfg::kRunBytes,
                      (half ? V : K) + static_cast<int64_t>(key) * kHd, bytes,
                      &sh.stg_full[at.stage], pol);
        at.next();
        ++units;
      }
  // do not leave with copies into shared memory in flight
  for (int u = max(0, units - Cfg::kStaging); u < units; ++u)
    ok = mbar_wait(&sh.stg_full[u % Cfg::kStaging],
                   static_cast<uint32_t>(u / Cfg::kStaging) & 1u) && ok;
  if (!ok) atomicOr(&g_err_prefix, kErrAttLoad);
}

template <int kHd>
__device__ __forceinline__ void prefix_convert(PrefixShared<kHd>& sh, const uint8_t* staging,
                                               uint8_t* k_ring, uint8_t* v_ring, int keys, int n) {
  using Cfg = PrefixCfg<kHd>;
  constexpr int kPL = kHd / 32, kNC = Cfg::kNC, kRows = Cfg::kRunRows;
  static_assert(Cfg::kConvWarps == 8 && Cfg::kRun % 8 == 0, "the rows' places below");
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int cw = static_cast<int>(threadIdx.x >> 5) - Cfg::kConv;
  // A warp's row i of a run is row cw + 8 i: in the swizzled units rows 8 apart have the
  // same pattern, 1024 bytes apart.
  const uint32_t col = static_cast<uint32_t>(lane_col<kPL>(lane, 0));
  const uint32_t place = (col / 64) * Cfg::kUnit + (col % 8) * 2 +
                         sw128_off(static_cast<uint32_t>(cw), col % 64 / 8);
  RingAt<Cfg::kStaging> at;
  bool dead = false;           // a wait gave up: no more waits, the barriers go on
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
  };
  bool seen = false;           // the next run of rows was seen to be there
#pragma unroll 1
  for (int jh = 0; jh < 2 * n; ++jh) {
    const int j = jh >> 1, slot = j & 1;
    const bool is_v = jh & 1;
    const uint32_t free_par = (static_cast<uint32_t>(j >> 1) & 1u) ^ 1u;
    const int stage = (j % Cfg::kDepth) * kNC;
    uint64_t* empty = is_v ? sh.mma.v_empty : sh.mma.k_empty;
    // the V ring is the softmax warps' scratch until Q is stored
    if (jh == 1) wait(&sh.mma.q_ready, 0);
    wait2(is_v ? &sh.mma.vmeta_free[slot] : &sh.mma.meta_free[slot], free_par, &empty[stage],
          (static_cast<uint32_t>(j / Cfg::kDepth) & 1u) ^ 1u, dead);
    uint8_t* dst = (is_v ? v_ring : k_ring) + stage * Cfg::kUnit;
    TileMeta& meta = sh.mma.meta[slot];
    bool misfit = false;                          // values that need another scale
#pragma unroll 1
    for (int r = 0; r < Cfg::kRuns; ++r) {
      const int rows = min(Cfg::kRun, keys - j * kTileKeys - r * Cfg::kRun);
      float x[kRows][kPL], m[kRows];
      if (rows > 0 && !__all_sync(0xFFFFFFFFu, seen)) wait(&sh.stg_full[at.stage], at.phase);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int row = cw + 8 * i;
#pragma unroll
        for (int c = 0; c < kPL; ++c) x[i][c] = 0.f;
        if (row < rows)
          load_row<kPL>(reinterpret_cast<const float*>(staging + at.stage * Cfg::kRunBytes) +
                            row * kHd,
                        lane, x[i]);
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        m[i] = fabsf(x[i][0]);
#pragma unroll
        for (int c = 1; c < kPL; ++c) m[i] = fmaxf(m[i], fabsf(x[i][c]));
      }
      if (j == 0 && r == 0) {
        // the piece's scale
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (m[i] <= 3.4028235e38f) a = fmaxf(a, m[i]);
        a = warp_max(a);
        if (lane == 0) sh.vmax[is_v][cw] = a;
        bar_sync(5, 32 * Cfg::kConvWarps);
#pragma unroll
        for (int w = 0; w < Cfg::kConvWarps; ++w) a = fmaxf(a, sh.vmax[is_v][w]);
        const int e = a > 0.f ? max(split_exp(a) - 7, -126) : 0;
        if (lane < 2) sh.scale[is_v][lane] = exp2i(e);        // by every warp, the same
        __syncwarp();
      }
      // a power of two; vmeta_free has shown this warp what became of the slot's last tile
      const float sc = sh.scale[is_v][slot];
      // bit i: row i has a value of 2^-3 or more; bit 31: some value does not fit
      uint32_t has = 0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        has |= static_cast<uint32_t>(m[i] * sc >= 0.125f) << i;
        has |= static_cast<uint32_t>(m[i] * sc > 65504.f) << 31;
      }
      const bool fit = __reduce_or_sync(0xFFFFFFFFu, has) == (1u << kRows) - 1u;
      if (rows > 0) {
        // the stage may be overwritten once every lane HAS its values: loads that nothing
        // has used yet may be scheduled behind the arrival, so it hangs on the vote
        if (lane == 0 && (fit || has != 0xFFFFFFFFu)) mbar_arrive(&sh.stg_empty[at.stage]);
        at.next();
        seen = mbar_test(&sh.stg_full[at.stage], at.phase);
      }
      float mine = 1.0f / sc;        // lane i: 2^-e of key row i
      float by[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) by[i] = sc;
      if (!fit) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          bool fin;
          const float am = row_amax<kPL>(x[i], fin);
          const bool in = fin && (am == 0.f || (am * sc >= 0.125f && am * sc <= 65504.f));
          if (in) continue;
          if (is_v) {
            misfit = true;
          } else {
            const int e = split_exp(am);
            by[i] = exp2i(e);
            if (lane == i) mine = exp2i(-e);
          }
        }
      }
      if (!is_v && lane < kRows) meta.kscale[r * Cfg::kRun + cw + 8 * lane] = mine;
      uint8_t* at_rows = dst + r * (Cfg::kRun / 8) * 1024;
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        store_split_at<typename Cfg::Base>(x[i], by[i], lane, at_rows + i * 1024 + place);
    }
    if (is_v && lane == 0) {
      if (cw == 0) meta.vscale = 1.0f / sh.scale[1][slot];
      if (misfit) sh.misfit[j] = 1;
    }
    fence_proxy_async_smem();                     // generic stores -> visible to the MMAs
    __syncwarp();
    if (lane == 0) {
      if (is_v) {
        mbar_arrive(&sh.v_done[slot]);            // prefix_refit hands them on
      } else {
        mbar_arrive(&sh.mma.k_full[stage]);
        mbar_arrive(&sh.mma.meta_full[slot]);
      }
    }
  }
  if (dead && lane == 0) atomicOr(&g_err_prefix, kErrAttLoad);
}

// One warp hands the converters' tiles of values on to the MMAs.  A tile that the scale in force
// did not fit it lays out once more, over what is there, from memory: with the scale and the
// rows left out that pack_values would choose.  The tile after next goes on with that scale, its
// largest value at [2^7, 2^8).  It takes 25 us at head_dim 256 (9 at 64), the time of some six
// tiles: a value row 2^12 times the others among a piece's first (16 rows over 16384 positions,
// 4 heads of 256) costs 47 -> 123 us, a scale that is wrong for every tile 47 -> 190; with
// its rows left out one by one the first took 4.4 ms.  As part of the converters' code,
// by the last of them, it cost ordinary values 40 %; this way 2 (32 x 32768: 72.3 -> 73.9 us).
template <int kHd>
__device__ __forceinline__ void prefix_refit(PrefixShared<kHd>& sh, const float* V, uint8_t* v_ring,
                                             int keys, int n) {
  using Cfg = PrefixCfg<kHd>;
  constexpr int kPL = kHd / 32, kAt = 16 / kPL < 4 ? 16 / kPL : 4;      // rows in flight
  const int lane = static_cast<int>(threadIdx.x & 31);
  bool dead = false;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int slot = j & 1, stage = (j % Cfg::kDepth) * Cfg::kNC;
    if (!dead)
      dead = !__all_sync(0xFFFFFFFFu,
                         mbar_wait(&sh.v_done[slot], static_cast<uint32_t>(j >> 1) & 1u));
    if (__any_sync(0xFFFFFFFFu, sh.misfit[j] != 0)) {
      const float* from = V + static_cast<int64_t>(j) * kTileKeys * kHd;
      const int there = min(kTileKeys, keys - j * kTileKeys);
      float x[kAt][kPL], a = 0.f, b = 0.f;       // rows; the largest of rows lane and lane + 32
      const auto load = [&](int r) {
#pragma unroll
        for (int i = 0; i < kAt; ++i) {
#pragma unroll
          for (int c = 0; c < kPL; ++c) x[i][c] = 0.f;
          if (r + i < there) load_row<kPL>(from + (r + i) * kHd, lane, x[i]);
        }
      };
#pragma unroll 1
      for (int r = 0; r < kTileKeys; r += kAt) {
        load(r);
#pragma unroll
        for (int i = 0; i < kAt; ++i) {
          bool fin;
          const float m = row_amax<kPL>(x[i], fin), top = fin ? m : INFINITY;
          if (r + i == lane) a = top;
          if (r + i == lane + 32) b = top;
        }
      }
      const ValueScale sc = choose_value_scale(a, b);
      const int e = split_exp(sc.top);
#pragma unroll 1
      for (int r = 0; r < kTileKeys; r += kAt) {
        load(r);
#pragma unroll
        for (int i = 0; i < kAt; ++i) {
          const bool out = ((r < 32 ? sc.out[0] : sc.out[1]) >> ((r + i) & 31)) & 1u;
#pragma unroll
          for (int c = 0; c < kPL; ++c) x[i][c] = out ? 0.f : x[i][c];
          store_split_row<typename Cfg::Base>(x[i], exp2i(e), r + i, lane,
                                              v_ring + stage * Cfg::kUnit);
        }
      }
      if (lane == 0) {
        sh.mma.meta[slot].vscale = exp2i(-e);
        sh.left_out[j][0] = sc.out[0];
        sh.left_out[j][1] = sc.out[1];
        if (sc.top > 0.f) sh.scale[1][slot] = exp2i(max(e - 7, -126));
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (lane == 0) {
      mbar_arrive(&sh.mma.v_full[stage]);
      mbar_arrive(&sh.mma.vmeta_full[slot]);
    }
  }
  if (dead && lane == 0) atomicOr(&g_err_prefix, kErrAttLoad);
}

// Softmax and output of a row's half: two threads share a query row, each has half of a
// tile's keys and, of each chunk of head_dim, half of the output columns.
template <class Cfg, bool kCap>
__device__ __forceinline__ void prefix_rows(MmaShared<Cfg>& sh, const uint32_t (*left_out)[2],
                                            int n, int keys, float scale, float cap,
                                            RowState<Cfg>& st, bool& dead) {
  constexpr int kKeys = kTileKeys / 2;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int quad = warp & 3, part = warp >> 2;
  const int row = 32 * quad + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
  auto row_sync = [&]() { bar_sync(1 + quad, 64); };
  dead = false;
  st.m = -INFINITY;
  st.l = 0.f;
  st.any_left_out = false;
  const float qscale = q_unscale(sh, row);
#pragma unroll
  for (int c = 0; c < Cfg::kNC; ++c)
#pragma unroll
    for (int i = 0; i < Cfg::kOC / 2; ++i) st.o[c][i] = make_float2(0.f, 0.f);
  const float rowf = qscale * scale * kLog2e;
  const SoftCap soft(kCap ? cap : 1.f);
  const uint32_t t_o = lanes + Cfg::kTmO + static_cast<uint32_t>(part * Cfg::kOC);
  float alpha = 1.f, vs = 1.f;
  uint32_t w[kKeys];           // of every 16 keys hi, then lo
  // waits unless an earlier mbar_test saw the phase over
  auto wait = [&](uint64_t* bar, uint32_t parity, bool seen) {
    if (!__all_sync(0xFFFFFFFFu, seen) && !dead)
      dead = !__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
  };
  RingAt<2> buf;
  bool s_seen = false, o_seen = false;
  // S(j) -> the weights of tile j, split, in registers
  auto weights = [&](int j) {
    const uint32_t ph = static_cast<uint32_t>(j) & 1u;
    const uint32_t mph = static_cast<uint32_t>(j >> 1) & 1u;
    if (!__all_sync(0xFFFFFFFFu, s_seen) && !dead)
      dead = !__all_sync(0xFFFFFFFFu,
                         mbar_wait(&sh.meta_full[ph], mph) && mbar_wait(&sh.s_full[0], ph));
    tc_fence_after();
    float x[kKeys];
    {
      uint32_t v[kKeys];
      tc_ld<kKeys>(lanes + Cfg::kTmS + static_cast<uint32_t>(kKeys * part), v);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_free[0]);
      const float4* ks = reinterpret_cast<const float4*>(sh.meta[ph].kscale + kKeys * part);
#pragma unroll
      for (int i = 0; i < kKeys / 4; ++i) {
        const float4 f = ks[i];
        const float2 rf = make_float2(rowf, rowf);
        const float2 a =
            __fmul2_rn(bits2(v[4 * i], v[4 * i + 1]), __fmul2_rn(make_float2(f.x, f.y), rf));
        const float2 b =
            __fmul2_rn(bits2(v[4 * i + 2], v[4 * i + 3]), __fmul2_rn(make_float2(f.z, f.w), rf));
        x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
      }
    }
    if constexpr (kCap) soft_caps<kKeys>(x, soft);
    if ((j + 1) * kTileKeys > keys) {
      const int left = keys - j * kTileKeys - kKeys * part;    // of this thread's keys, how many
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (i >= left) x[i] = -INFINITY;                      // a select: nothing is multiplied
    }
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < kKeys; ++i) mx = fmaxf(mx, x[i]);
    sh.x[ph][part][row] = mx;
    row_sync();
    // what was stored came of the scales: they have been read
    if (lane == 0) mbar_arrive(&sh.meta_free[ph]);
#pragma unroll
    for (int c = 0; c < 2; ++c) mx = fmaxf(mx, sh.x[ph][c][row]);
    const float mn = fmaxf(st.m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    alpha = ex2(st.m - base);
    st.m = mn;
    const float sub = static_cast<float>(kPShift) - base;
    o_seen = mbar_test(&sh.o_full[buf.stage], buf.phase);   // the chunk drained next
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kKeys / 2; ++i) {
      float2 a = __fadd2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(sub, sub));
      a.x = ex2(a.x);
      a.y = ex2(a.y);
      sum = __fadd2_rn(sum, a);
      split2(a, w[i / 8 * 16 + i % 8], w[i / 8 * 16 + 8 + i % 8]);
    }
    st.l = fmaf(st.l, alpha, sum.x + sum.y);
  };
  auto store_p = [&](int j) {
    // S of the tile after next, meanwhile
    const uint32_t ph = static_cast<uint32_t>(j + 1) & 1u;
    s_seen = mbar_test(&sh.meta_full[ph], static_cast<uint32_t>((j + 1) >> 1) & 1u) &
             mbar_test(&sh.s_full[0], ph);
    tc_st<kKeys>(lanes + Cfg::kTmP + static_cast<uint32_t>(kKeys * part), w);
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.p_ready[0]);
  };
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    weights(j);
    store_p(j);
    {
      const uint32_t ph = static_cast<uint32_t>(j) & 1u;
      if (!dead)
        dead = !__all_sync(0xFFFFFFFFu,
                           mbar_wait(&sh.vmeta_full[ph], static_cast<uint32_t>(j >> 1) & 1u));
      vs = sh.meta[ph].vscale;
      const bool left = (left_out[j][0] | left_out[j][1]) != 0;
      // the arrival hangs on the values read: loads that nothing has used yet may be
      // scheduled behind it (vs is a power of two; left is the same in all lanes)
      const uint32_t lefts = __ballot_sync(0xFFFFFFFFu, left && vs > 0.f);
      st.any_left_out = st.any_left_out || lefts;
      if (lane == 0 && (vs > 0.f || lefts)) mbar_arrive(&sh.vmeta_free[ph]);
#pragma unroll
    for (int c = 0; c < Cfg::kNC; ++c) {
      wait(&sh.o_full[buf.stage], buf.phase, o_seen);
      tc_fence_after();
      uint32_t v[Cfg::kOC];
      tc_ld<Cfg::kOC>(t_o + static_cast<uint32_t>(buf.stage) * 64u, v);
      uint64_t* free_bar = &sh.o_free[buf.stage];
      buf.next();
      o_seen = c + 1 < Cfg::kNC && mbar_test(&sh.o_full[buf.stage], buf.phase);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(free_bar);
#pragma unroll
      for (int i = 0; i < Cfg::kOC; i += 2) {
        st.o[c][i / 2] = __ffma2_rn(st.o[c][i / 2], make_float2(alpha, alpha),
                                    __fmul2_rn(bits2(v[i], v[i + 1]), make_float2(vs, vs)));
      }
    }
    }
  }
  // the row's whole sum
  row_sync();
  sh.x[0][part][row] = st.l;
  row_sync();
  float l = 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c) l += sh.x[0][c][row];
  st.l = l;
}

// grid (pieces * row tiles, n_kv)
template <int kHd, bool kCap>
__global__ void __launch_bounds__(PrefixCfg<kHd>::kThreads, 1)
    prefix_mma_kernel(const __grid_constant__ PrefixParams p) {
  using Cfg = PrefixCfg<kHd>;
  extern __shared__ uint8_t raw[];
  uint8_t* k_ring = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  uint8_t* v_ring = k_ring + Cfg::kStages * Cfg::kUnit;
  uint8_t* staging = v_ring + Cfg::kStages * Cfg::kUnit;
  auto& sh = *reinterpret_cast<PrefixShared<kHd>*>(staging + Cfg::kStaging * Cfg::kRunBytes);
  const int piece = blockIdx.x / p.row_tiles, rt = blockIdx.x - piece * p.row_tiles;
  const int g = blockIdx.y;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int ka = piece * p.chunk, keys = min(p.n_prefix, ka + p.chunk) - ka;
  const int n = (keys + kTileKeys - 1) / kTileKeys;
  if (threadIdx.x < 2 * kMaxPieceTiles) sh.left_out[threadIdx.x >> 1][threadIdx.x & 1] = 0;
  if (threadIdx.x < kMaxPieceTiles) sh.misfit[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStaging; ++s) {
      mbar_init(&sh.stg_full[s], 1);
      mbar_init(&sh.stg_empty[s], Cfg::kConvWarps);
    }
    for (int s = 0; s < 2; ++s) mbar_init(&sh.v_done[s], Cfg::kConvWarps);
    mma_init_barriers<Cfg>(sh.mma, Cfg::kConvWarps, 1);
  }
  if (warp == Cfg::kMmaQk) {
    tmem_alloc(&sh.mma.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  // only now: own_part_kernel starts with this and reads what the call was given
  pdl_launch_dependents();
  const int64_t at = (static_cast<int64_t>(g) * p.max_prefix + ka) * kHd;
  if (warp >= Cfg::kConv) {
    regs_dec<56>();
    prefix_convert<kHd>(sh, staging, k_ring, v_ring, keys, n);
  } else if (warp >= Cfg::kRowsWarps) {
    regs_dec<48>();
    if (warp == Cfg::kLoadK && lane == 0)
      prefix_load<kHd>(sh, staging, p.kp + at, p.vp + at, keys, n);
    if (warp == Cfg::kLoadV) prefix_refit<kHd>(sh, p.vp + at, v_ring, keys, n);
    if (warp == Cfg::kMmaQk) mma_issue_qk<Cfg>(sh.mma, k_ring, nullptr, n, &g_err_prefix);
    if (warp == Cfg::kMmaPv) mma_issue_pv<Cfg>(sh.mma, v_ring, n, &g_err_prefix);
  } else {
    regs_inc<160>();
    const int row = 32 * (warp & 3) + lane, part = warp >> 2;
    const int r = rt * kTileRows + row, live = p.batch * p.group;
    const bool alive = r < live;
    const int rc = min(r, live - 1);
    const float* q = p.q.data + static_cast<int64_t>(p.b0 + rc / p.group) * p.q.token_stride +
                     (g * p.group + rc % p.group) * p.q.head_stride;
    RowState<Cfg> st;
    bool dead;
    float* scratch = reinterpret_cast<float*>(v_ring);
    store_q<Cfg>(sh.mma, scratch, nullptr, alive ? q : nullptr);
    prefix_rows<Cfg, kCap>(sh.mma, sh.left_out, n, keys, p.scale, p.cap, st, dead);
    if (dead && lane == 0) atomicOr(&g_err_prefix, kErrAttRows);
    if (st.any_left_out && alive) {
      for (int t = 0; t < keys; ++t)
        if ((sh.left_out[t / kTileKeys][(t % kTileKeys) >> 5] >> (t & 31)) & 1u)
          add_left_out<Cfg>(st, q, p.kp + at + static_cast<int64_t>(t) * kHd,
                            p.vp + at + static_cast<int64_t>(t) * kHd, part, p.scale, p.cap);
    }
    constexpr float kUnshift = 1.0f / (1 << kPShift);
    const bool store = alive && !dead;
    float* dst = p.part + prefix_part<kHd / 32>(p, piece, g, rc);
    store_rows<Cfg>(st, scratch, store ? dst : nullptr, kUnshift);
    if (store && part == 0)
      *reinterpret_cast<float2*>(dst + kHd) = make_float2(st.m, st.l * kUnshift);
  }
  // every MMA has completed before tensor memory is freed
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::kMmaQk) {
    for (int i = 0; i < 2; ++i)
      if (lane == 0 && !mbar_wait(&sh.mma.done[i], 0)) atomicOr(&g_err_prefix, kErrAttMma);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(sh.mma.tmem, 512);
  }
}

// Own parts: grid (own items, n_kv).  A warp takes four neighbouring keys: K and V
// rows straight from memory, all at once, a lane holding its columns, the dot products
// by warp sums; the warps are joined in shared memory in order.  Short items, because
// one costs three trips to memory however long it is: with 128 keys an item, four
// sequences of up to 130 keys took 10.6 us.
//
// This kernel does not need the shared part's results: it runs beside that kernel, on the
// SMs that one leaves free or has left, and waits for it only at its end, so that the joining
// kernel behind finds both done.  (The shared part lets it start only after everything before
// the call has completed.)
template <int kPL, int kG>
__global__ void __launch_bounds__(kOwnWarps * 32)
    own_part_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int kHd = kPL * 32;
  __shared__ __align__(16) float sacc[kOwnWarps][kG][kHd];
  __shared__ float sm[kOwnWarps][kG], sl[kOwnWarps][kG];
  if (!p.beside) pdl_wait();
  pdl_launch_dependents();
  const int b = find_seq(p.first, p.batch, blockIdx.x);
  const int g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ka = (blockIdx.x - p.first[b]) * kOwnChunk, kb = min(p.n_ctx[b], ka + kOwnChunk);
  const int64_t head = (static_cast<int64_t>(p.b0 + b) * p.n_kv + g) * p.max_seq * kHd;
  const int t = ka + warp * kOwnKeys;
  float q[kG][kPL], acc[kG][kPL], m[kG], l[kG];
  float k[kOwnKeys][kPL], v[kOwnKeys][kPL];
#pragma unroll
  for (int i = 0; i < kOwnKeys; ++i) {
    const int64_t at = head + static_cast<int64_t>(min(t + i, kb - 1)) * kHd;
    load_row<kPL>(p.kc + at, lane, k[i]);
    load_row<kPL>(p.vc + at, lane, v[i]);
  }
#pragma unroll
  for (int h = 0; h < kG; ++h)
    load_row<kPL>(p.q.data + static_cast<int64_t>(p.b0 + b) * p.q.token_stride +
                      (g * kG + h) * p.q.head_stride,
                  lane, q[h]);
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    float s[kOwnKeys];
    m[h] = -INFINITY;
#pragma unroll
    for (int i = 0; i < kOwnKeys; ++i) {
      float d = 0.f;
#pragma unroll
      for (int j = 0; j < kPL; ++j) d = fmaf(q[h][j], k[i][j], d);
      s[i] = t + i < kb ? soft_cap(warp_sum(d) * p.scale, p.cap) * kLog2e : -INFINITY;
      m[h] = fmaxf(m[h], s[i]);
    }
    const float base = m[h] == -INFINITY ? 0.f : m[h];
    float pr[kOwnKeys];
    l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < kOwnKeys; ++i) {
      pr[i] = exp2f(s[i] - base);
      l[h] += pr[i];
    }
#pragma unroll
    for (int j = 0; j < kPL; ++j) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < kOwnKeys; ++i)
        if (t + i < kb) a = fmaf(pr[i], v[i][j], a);
      acc[h][j] = a;
    }
  }
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    store_row<kPL>(sacc[warp][h], lane, acc[h]);
    if (lane == 0) {
      sm[warp][h] = m[h];
      sl[warp][h] = l[h];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kG * kHd; e += kOwnWarps * 32) {
    const int h = e / kHd, c = e - h * kHd;
    float M = -INFINITY;
    for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, sm[w][h]);
    const float base = M == -INFINITY ? 0.f : M;
    float a = 0.f, L = 0.f;
    for (int w = 0; w < kOwnWarps; ++w) {
      const float f = exp2f(sm[w][h] - base);
      a = fmaf(sacc[w][h][c], f, a);
      L = fmaf(sl[w][h], f, L);
    }
    float* dst =
        p.own + ((static_cast<int64_t>(blockIdx.x) * p.n_kv + g) * kG + h) * (kHd + kPartPad);
    dst[c] = a;
    if (c == 0) {
      dst[kHd] = M;
      dst[kHd + 1] = L;
    }
  }
  if (p.beside) pdl_wait();
}

// Few keys in all: one CTA per sequence and kv head takes the shared and the own
// positions, kOwnKeys neighbours a warp in turns, and writes out; no partial results, one
// launch in place of three.  grid (batch, n_kv).
template <int kPL, int kG>
__global__ void __launch_bounds__(kOwnWarps * 32)
    prefix_few_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int kHd = kPL * 32;
  __shared__ __align__(16) float sacc[kOwnWarps][kG][kHd];
  __shared__ float sm[kOwnWarps][kG], sl[kOwnWarps][kG];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t shared_at = static_cast<int64_t>(g) * p.max_prefix * kHd;
  const int64_t own_at = (static_cast<int64_t>(p.b0 + b) * p.n_kv + g) * p.max_seq * kHd;
  const int n = p.n_prefix + p.n_ctx[b];
  float q[kG][kPL], acc[kG][kPL], m[kG], l[kG];
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    load_row<kPL>(p.q.data + static_cast<int64_t>(p.b0 + b) * p.q.token_stride +
                      (g * kG + h) * p.q.head_stride,
                  lane, q[h]);
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int j = 0; j < kPL; ++j) acc[h][j] = 0.f;
  }
  for (int t = warp * kOwnKeys; t < n; t += kOwnChunk) {
    float k[kOwnKeys][kPL], v[kOwnKeys][kPL];
#pragma unroll
    for (int i = 0; i < kOwnKeys; ++i) {
      const int key = min(t + i, n - 1);
      const bool own = key >= p.n_prefix;
      const int64_t at = own ? own_at + static_cast<int64_t>(key - p.n_prefix) * kHd
                             : shared_at + static_cast<int64_t>(key) * kHd;
      load_row<kPL>((own ? p.kc : p.kp) + at, lane, k[i]);
      load_row<kPL>((own ? p.vc : p.vp) + at, lane, v[i]);
    }
#pragma unroll
    for (int h = 0; h < kG; ++h) {
      float s[kOwnKeys], mn = m[h];
#pragma unroll
      for (int i = 0; i < kOwnKeys; ++i) {
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < kPL; ++j) d = fmaf(q[h][j], k[i][j], d);
        s[i] = t + i < n ? soft_cap(warp_sum(d) * p.scale, p.cap) * kLog2e : -INFINITY;
        mn = fmaxf(mn, s[i]);
      }
      const float base = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m[h] - base);
      float pr[kOwnKeys];
      l[h] *= alpha;
#pragma unroll
      for (int i = 0; i < kOwnKeys; ++i) {
        pr[i] = exp2f(s[i] - base);
        l[h] += pr[i];
      }
#pragma unroll
      for (int j = 0; j < kPL; ++j) {
        float a = acc[h][j] * alpha;
#pragma unroll
        for (int i = 0; i < kOwnKeys; ++i)
          if (t + i < n) a = fmaf(pr[i], v[i][j], a);
        acc[h][j] = a;
      }
      m[h] = mn;
    }
  }
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    store_row<kPL>(sacc[warp][h], lane, acc[h]);
    if (lane == 0) {
      sm[warp][h] = m[h];
      sl[warp][h] = l[h];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kG * kHd; e += kOwnWarps * 32) {
    const int h = e / kHd, c = e - h * kHd;
    float M = -INFINITY;
    for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, sm[w][h]);
    const float base = M == -INFINITY ? 0.f : M;
    float a = 0.f, L = 0.f;
    for (int w = 0; w < kOwnWarps; ++w) {
      const float f = exp2f(sm[w][h] - base);
      a = fmaf(sacc[w][h][c], f, a);
      L = fmaf(sl[w][h], f, L);
    }
    p.out.data[static_cast<int64_t>(p.b0 + b) * p.out.token_stride +
               (g * kG + h) * p.out.head_stride + c] = L == 0.f ? 0.f : a / L;
  }
}

// One CTA per (sequence, query head, 64 columns): the prefix pieces, then the own ones, a
// quarter of them a warp (at least 8), and the warps in order.  By one warp, 37 pieces and
// up to 32 own ones were six trips to memory in turn, 10 us.
constexpr int kJoinWarps = 4;
template <int kPL>
__global__ void __launch_bounds__(kJoinWarps * 32)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int kHd = kPL * 32, kV = kPL >= 2 ? 2 : 1, kWide = kHd / (32 * kV);
  __shared__ float sacc[kJoinWarps][32 * kV], sm[kJoinWarps], sl[kJoinWarps];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rh = blockIdx.x / kWide, c0 = (blockIdx.x - rh * kWide) * 32 * kV;
  const int b = rh / p.n_q, h = rh - b * p.n_q, g = h / p.group;
  const int row = b * p.group + (h - g * p.group);
  const auto part = [&](int c) {
    return c < p.pieces
               ? p.part + prefix_part<kPL>(p, c, g, row)
               : p.own + ((static_cast<int64_t>(p.first[b] + c - p.pieces) * p.n_kv + g) * p.group +
                          (h - g * p.group)) * (kHd + kPartPad);
  };
  const int n = p.pieces + p.first[b + 1] - p.first[b];
  const int each = max(8, (n + kJoinWarps - 1) / kJoinWarps), from = warp * each;
  pdl_wait();
  float acc[kV], m;
  const float l = join_parts<kHd, kV>(from, min(n, from + each), lane, c0 + lane * kV, part, part,
                                      acc, m);
#pragma unroll
  for (int i = 0; i < kV; ++i) sacc[warp][lane * kV + i] = acc[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  if (warp > 0) return;
  float M = sm[0], L = 0.f;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) M = fmaxf(M, sm[w]);
  const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = exp2f(sm[w] - base);
    L = fmaf(sl[w], f, L);
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] = fmaf(sacc[w][lane * kV + i], f, acc[i]);
  }
  store_final<kV>(p.out.data + static_cast<int64_t>(p.b0 + b) * p.out.token_stride +
                      h * p.out.head_stride + c0,
                  lane, acc, L);
}

// ------------------------------------------------------------ host side
namespace {

// Shared and own positions of the longest sequence up to which one CTA a sequence and kv
// head takes them all.  Device time this way / in three kernels, at 96, 256 and 384 positions: 4
// sequences of 8 q / 4 kv heads of 256 6.7 / 14.4, 14.0 / 14.5, 19.8 / 14.8 us; 32 of 256
// 7.5 / 17.0, 15.5 / 21.1, 21.9 / 21.8; 32 of 8 / 4 heads of 128 6.2 / 10.8, 13.2 / 12.4, 18.6 / 12.5.
// Four heads a kv head make it longer: 4 of 8 / 2 heads of 64 8.3 / 8.8, 19.1 / 10.4.
constexpr int64_t kFewKeys = 256;

struct PrefixPlan {
  bool few;              // all positions by one kernel
  int chunk, pieces;
  size_t part_floats, own_floats;    // of the largest launch
};

PrefixPlan plan_prefix(int64_t n_prefix, const int64_t* n_ctx, int batch, int n_q, int n_kv,
                       int head_dim) {
  PrefixPlan pl = {};
  const int group = n_q / n_kv, some = std::min(batch, kMaxBatch);
  int64_t longest = 0;
  for (int b = 0; b < batch; ++b) longest = std::max(longest, n_ctx[b]);
  pl.few = n_prefix + longest <= kFewKeys;
  if (pl.few) return pl;
  const int64_t tiles = (static_cast<int64_t>(some) * group + kTileRows - 1) / kTileRows;
  // one item an SM
  const int64_t want = std::max<int64_t>(1, 152 / (tiles * n_kv));
  const int64_t key_tiles = (n_prefix + kTileKeys - 1) / kTileKeys;
  const int64_t chunk =
      std::max<int64_t>(1, std::min<int64_t>((key_tiles + want - 1) / want, kMaxPieceTiles)) *
      kTileKeys;
  pl.chunk = static_cast<int>(chunk);
  pl.pieces = static_cast<int>((n_prefix + chunk - 1) / chunk);
  const size_t row = static_cast<size_t>(head_dim) + kPartPad;
  pl.part_floats = static_cast<size_t>(pl.pieces) * n_q * some * row;
  int64_t most = 0;
  for (int b0 = 0; b0 < batch; b0 += kMaxBatch) {
    int64_t items = 0;
    for (int b = b0; b < std::min(batch, b0 + kMaxBatch); ++b)
      items += (n_ctx[b] + kOwnChunk - 1) / kOwnChunk;
    most = std::max(most, items);
  }
  pl.own_floats = static_cast<size_t>(most) * n_q * row;
  return pl;
}

template <int kPL>
cudaError_t run_prefix(const PrefixParams& p, const PrefixPlan& pl, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  const unsigned nkv = static_cast<unsigned>(p.n_kv);
  if (pl.few) {
    const dim3 grid(static_cast<unsigned>(p.batch), nkv);
    switch (p.group) {
      case 1: return pdl_launch(prefix_few_kernel<kPL, 1>, grid, kOwnWarps * 32, 0, st, p);
      case 2: return pdl_launch(prefix_few_kernel<kPL, 2>, grid, kOwnWarps * 32, 0, st, p);
      case 3: return pdl_launch(prefix_few_kernel<kPL, 3>, grid, kOwnWarps * 32, 0, st, p);
      case 4: return pdl_launch(prefix_few_kernel<kPL, 4>, grid, kOwnWarps * 32, 0, st, p);
    }
    return cudaErrorInvalidValue;
  }
  if (p.pieces > 0) {
    constexpr int kHd = kPL * 32;
    using Cfg = PrefixCfg<kHd>;
    constexpr size_t kSmem =
        1024 + Cfg::kRing + Cfg::kStaging * Cfg::kRunBytes + sizeof(PrefixShared<kHd>);
    static_assert(kSmem <= 227 * 1024, "shared memory");
    const auto kernel = p.cap > 0.f ? prefix_mma_kernel<kHd, true> : prefix_mma_kernel<kHd, false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    e = pdl_launch(kernel, dim3(static_cast<unsigned>(p.pieces * p.row_tiles), nkv), Cfg::kThreads,
                   kSmem, st, p);
    if (e != cudaSuccess) return e;
  }
  if (const int items = p.first[p.batch]) {
    const dim3 grid(static_cast<unsigned>(items), nkv);
    switch (p.group) {
      case 1: e = pdl_launch(own_part_kernel<kPL, 1>, grid, kOwnWarps * 32, 0, st, p); break;
      case 2: e = pdl_launch(own_part_kernel<kPL, 2>, grid, kOwnWarps * 32, 0, st, p); break;
      case 3: e = pdl_launch(own_part_kernel<kPL, 3>, grid, kOwnWarps * 32, 0, st, p); break;
      case 4: e = pdl_launch(own_part_kernel<kPL, 4>, grid, kOwnWarps * 32, 0, st, p); break;
      default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
  }
  constexpr int kWide = kPL > 2 ? kPL / 2 : 1;          // CTAs of a row
  return pdl_launch(prefix_merge_kernel<kPL>, dim3(static_cast<unsigned>(p.batch * p.n_q * kWide)),
                    kJoinWarps * 32, 0, st, p);
}

}  // namespace

size_t prefix_attention_workspace_bytes(int64_t n_prefix, const int64_t* n_ctx, int batch,
                                        int n_q, int n_kv, int head_dim) {
  const PrefixPlan pl = plan_prefix(n_prefix, n_ctx, batch, n_q, n_kv, head_dim);
  return (pl.part_floats + pl.own_floats) * sizeof(float);
}

cudaError_t launch_prefix_attention(const qws_heads& q, const float* kp, const float* vp,
                                    int64_t max_prefix, int64_t n_prefix, const float* kc,
                                    const float* vc, int64_t max_seq, const int64_t* n_ctx,
                                    const qws_heads& out, int batch, int n_q, int n_kv,
                                    int head_dim, float scale, float cap, void* ws,
                                    cudaStream_t st) {
  const PrefixPlan pl = plan_prefix(n_prefix, n_ctx, batch, n_q, n_kv, head_dim);
  PrefixParams p;
  p.q = q; p.out = out;
  p.kp = kp; p.vp = vp; p.kc = kc; p.vc = vc;
  p.part = static_cast<float*>(ws);
  p.own = p.part + pl.part_floats;
  p.max_prefix = max_prefix; p.max_seq = max_seq;
  p.n_q = n_q; p.n_kv = n_kv; p.group = n_q / n_kv;
  p.n_prefix = static_cast<int>(n_prefix);
  p.chunk = pl.chunk; p.pieces = pl.pieces;
  p.beside = pl.pieces > 0;
  p.scale = scale; p.cap = cap;
  for (int b0 = 0; b0 < batch; b0 += kMaxBatch) {
    p.b0 = b0;
    p.batch = std::min(batch - b0, kMaxBatch);
    p.row_tiles = (p.batch * p.group + kTileRows - 1) / kTileRows;
    p.first[0] = 0;
    for (int b = 0; b < p.batch; ++b) {
      p.n_ctx[b] = static_cast<int>(n_ctx[b0 + b]);
      p.first[b + 1] = p.first[b] + (p.n_ctx[b] + kOwnChunk - 1) / kOwnChunk;
    }
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 32: e = run_prefix<1>(p, pl, st); break;
      case 64: e = run_prefix<2>(p, pl, st); break;
      case 128: e = run_prefix<4>(p, pl, st); break;
      case 256: e = run_prefix<8>(p, pl, st); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

unsigned read_clear_prefix_errors() {
  unsigned v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_prefix, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_err_prefix, &z, sizeof(z));
  return v;
}

}  // namespace qws
