// prompt.cu -- causal attention over packed prompts (the seq > 1 counterpart
// of kv_attention): for query row i of a sequence with n_q rows and n_k keys,
// head h reading kv head h / group,
//   s_j = softcap(scale * q_ih . k_j)  for the visible keys j <= i + n_k - n_q,
//   out_ih = sum_j softmax(s)_j v_j;   a row without a visible key gives zeros.
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "attend_mma.cuh"
#include "attend_rows.cuh"
#include "launch.h"

namespace qws {

__device__ unsigned g_err_prompt;

// ------------------------------------------------------------ work items
// A tile is `rows` query rows of one kv head: tok = rows / group tokens with
// the group's heads side by side, row r = token r / group, head r % group.  Its
// keys are cut into pieces of `chunk`; an item is one piece.  The sequences with the most
// keys come first (a ragged batch of 12, heads of 256: 88 -> 79 us).  A sequence's items come
// by piece, first every tile's piece 0, the longest tile first, then piece 1 of the tiles that
// have one, and so on.  A tile of one piece writes out, the others leave partials that
// prompt_merge_kernel joins.
struct PromptParams {
  qws_heads q, k, v, out;
  float* part;
  uint8_t* packed;      // tensor-core form: packed key tiles [tile][kv head]
  TileMeta* meta;
  int n_q, n_kv, group, tok, rows, chunk;
  float scale, cap;
  SeqTab seqs;
};

struct PromptItem {
  int s, tile, piece, tiles;
  int i0, n_tok;        // first token (in the sequence) and tokens of the tile
  int n_q, n_k;         // of the sequence
  int vis;              // keys that the tile's last row sees
  int pieces;           // of the tile, at least 1
};

__device__ __forceinline__ int visible(int i, int n_q, int n_k) {
  return max(0, min(n_k, i + 1 + n_k - n_q));
}

__device__ __forceinline__ void tile_span(const PromptParams& p, PromptItem& it) {
  it.i0 = it.tile * p.tok;
  it.n_tok = min(p.tok, it.n_q - it.i0);
  it.vis = visible(it.i0 + it.n_tok - 1, it.n_q, it.n_k);
  it.pieces = max(1, (it.vis + p.chunk - 1) / p.chunk);
}

// Tiles from this one on have a piece `piece` (they see more than piece * chunk keys).
__host__ __device__ __forceinline__ int first_tile(int piece, int chunk, int tok, int n_q,
                                                   int n_k) {
  const int64_t need = static_cast<int64_t>(piece) * chunk - (static_cast<int64_t>(n_k) - n_q);
  return piece == 0 || need <= 0 ? 0 : static_cast<int>(need / tok);
}

__device__ __forceinline__ PromptItem prompt_item(const PromptParams& p, int item) {
  PromptItem it;
  const int place = find_seq(p.seqs.item, p.seqs.n, item);
  it.s = p.seqs.order[place];
  it.n_q = p.seqs.q0[it.s + 1] - p.seqs.q0[it.s];
  it.n_k = p.seqs.k0[it.s + 1] - p.seqs.k0[it.s];
  it.tiles = (it.n_q + p.tok - 1) / p.tok;
  int local = item - p.seqs.item[place];
  for (it.piece = 0;; ++it.piece) {
    const int have = it.tiles - first_tile(it.piece, p.chunk, p.tok, it.n_q, it.n_k);
    if (local < have) break;
    local -= have;
  }
  it.tile = it.tiles - 1 - local;
  tile_span(p, it);
  return it;
}

// the item number of piece 0 of a tile; of the next piece: + next_piece()
__device__ __forceinline__ int first_item(const PromptParams& p, const PromptItem& it) {
  return p.seqs.first[it.s] + it.tiles - 1 - it.tile;
}
__device__ __forceinline__ int next_piece(const PromptParams& p, const PromptItem& it,
                                          int piece) {
  return it.tiles - first_tile(piece, p.chunk, p.tok, it.n_q, it.n_k);
}
__device__ __forceinline__ float* part_rows(const PromptParams& p, int item, int g, int hd) {
  return p.part + (static_cast<int64_t>(item) * p.n_kv + g) * p.rows * (hd + kPartPad);
}

// ------------------------------------------------------------ CUDA cores, f32
template <int kPL, int kR>
__global__ void __launch_bounds__(kRowThreads)
    prompt_rows_kernel(const __grid_constant__ PromptParams p) {
  using Tile = RowTile<kPL, kR>;
  constexpr int kHd = Tile::kHd;
  extern __shared__ __align__(16) float smem[];
  pdl_launch_dependents();
  pdl_wait();
  const int item = blockIdx.x / p.n_kv, g = blockIdx.x - item * p.n_kv;
  const PromptItem it = prompt_item(p, item);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t q_base = p.seqs.q0[it.s], k_base = p.seqs.k0[it.s];
  const int ka = it.piece * p.chunk, kb = min(it.vis, ka + p.chunk);
  const int live = it.n_tok * p.group;
  Tile tile;
  tile.init();
  int vis[kR];
  float* qs = Tile::q_rows(smem);
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int row = warp * kR + r;
    float x[kPL];
#pragma unroll
    for (int j = 0; j < kPL; ++j) x[j] = 0.f;
    vis[r] = 0;
    if (row < live) {
      const int i = it.i0 + row / p.group, h = g * p.group + row % p.group;
      vis[r] = visible(i, it.n_q, it.n_k);
      load_row<kPL>(p.q.data + (q_base + i) * p.q.token_stride + h * p.q.head_stride, lane, x);
    }
    store_row<kPL>(qs + r * kHd, lane, x);
  }
  tile.run(smem, p.k.data + k_base * p.k.token_stride + g * p.k.head_stride,
           p.v.data + k_base * p.v.token_stride + g * p.v.head_stride, p.k.token_stride,
           p.v.token_stride, ka, kb, vis, p.scale, p.cap);
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int row = warp * kR + r;
    if (row >= live) continue;
    if (it.pieces > 1) {
      store_partial<kPL>(part_rows(p, item, g, kHd) + row * (kHd + kPartPad), lane, tile.acc[r],
                         tile.m[r], tile.l[r]);
    } else {
      const int i = it.i0 + row / p.group, h = g * p.group + row % p.group;
      store_final<kPL>(p.out.data + (q_base + i) * p.out.token_stride + h * p.out.head_stride,
                       lane, tile.acc[r], tile.l[r]);
    }
  }
}

// One warp per query row: joins the pieces of its tile in order.
template <int kPL>
__global__ void __launch_bounds__(256)
    prompt_merge_kernel(const __grid_constant__ PromptParams p) {
  constexpr int kHd = kPL * 32;
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int total = p.seqs.q0[p.seqs.n] - p.seqs.q0[0];
  const int64_t t = w / p.n_q;
  // every warp waits, also one with nothing to do: who comes behind this kernel counts on
  // the one before it to be done
  if (t >= total) {
    pdl_wait();
    return;
  }
  const int h = static_cast<int>(w - t * p.n_q), g = h / p.group;
  const int token = p.seqs.q0[0] + static_cast<int>(t);
  PromptItem it;
  it.s = find_seq(p.seqs.q0, p.seqs.n, token);
  it.n_q = p.seqs.q0[it.s + 1] - p.seqs.q0[it.s];
  it.n_k = p.seqs.k0[it.s + 1] - p.seqs.k0[it.s];
  it.tiles = (it.n_q + p.tok - 1) / p.tok;
  const int i = token - p.seqs.q0[it.s];
  it.tile = i / p.tok;
  tile_span(p, it);
  if (it.pieces < 2) {
    pdl_wait();
    return;
  }
  const int row = (i - it.i0) * p.group + (h - g * p.group);
  // lane c holds where piece c is (a tile has at most 32: the plan sees to it)
  int64_t where = first_item(p, it);
  for (int c = 1; c <= lane && c < it.pieces; ++c) where += next_piece(p, it, c - 1);
  where = ((where * p.n_kv + g) * p.rows + row) * (kHd + kPartPad);
  pdl_wait();
  const auto mine = [&](int) { return p.part + where; };
  const auto part = [&](int c) { return p.part + __shfl_sync(0xFFFFFFFFu, where, c); };
  constexpr int kV = kPL >= 4 ? 4 : kPL;
  float* dst = p.out.data + static_cast<int64_t>(token) * p.out.token_stride +
               h * p.out.head_stride;
#pragma unroll
  for (int c = 0; c < kHd; c += 32 * kV) {
    float acc[kV], m;
    const float l = join_parts<kHd, kV>(0, it.pieces, lane, c + lane * kV, mine, part, acc, m);
    store_final<kV>(dst + c, lane, acc, l);
  }
}

// ------------------------------------------------------------ tensor cores
// 20 warps: 0..7 keep the output, 8..11 and 12..15 turn the scores of the even and of the
// odd tiles into weights, 16..19 load and issue (attend_mma.cuh).  Each has its own warps
// because each is a chain of waits, tensor memory accesses and exchanges: when the same
// warps did both in turn, a tile took 4750 cycles (2830 at head_dim 128; 3590 with a
// softcap) where its MMAs take 3330 (1540).  S and P have two buffers, so that Q K(j+2)^T
// and P V(j+1) do not wait for one tile's softmax.  8192 positions, 8 q / 4 kv heads of 256:
// 616 -> 525 us; 16 q / 4 kv heads of 128: 619 -> 572 us, with a softcap 785 -> 683 us.  Since
// then Q K^T takes two passes (for accuracy) and the scores stay in registers up to head_dim
// 128: 541, 544 and 605 us (the MMAs at the measured rate: 428 us).  At head_dim 256 a tile
// takes 3780 cycles; below, the softmax's instructions bind (1400 a scheduler and tile).
template <int kHd>
struct PromptCfg : MmaCfg<kHd, (kHd > 128 ? 1 : 0), false, 2> {
  static constexpr int kThreads = 32 * 20;
  static constexpr uint32_t kSmem = MmaCfg<kHd, (kHd > 128 ? 1 : 0), false, 2>::kRing +
                                    MmaCfg<kHd, (kHd > 128 ? 1 : 0), false, 2>::kQLoBytes;
};
// 96 registers a thread at launch; per scheduler 2 output warps, 2 softmax warps and a
// helper: 2 x 160 + 2 x 64 + 32, or 2 x 104 + 2 x 104 + 64, of 5 x 96.
template <int kHd>
constexpr int kRegsOut = kHd > 128 ? 160 : 104;
template <int kHd>
constexpr int kRegsSoft = kHd > 128 ? 64 : 104;
template <int kHd>
constexpr int kRegsHelp = kHd > 128 ? 32 : 64;

// The weights of the tiles first, first + 2, ... of a row: a thread has the whole row, so
// nothing is exchanged.  Above head_dim 128, 64 scores and their packed weights do not fit the
// registers, and the scores wait for the second pass in tensor memory.  Each of the two groups
// of warps
// has its own running maximum; the output warps bring the tiles to one.  vis: the row sees
// the keys below vis; all_vis: below this one, every row of the CTA does.
template <class Cfg, bool kCap>
__device__ __forceinline__ bool tile_weights(MmaShared<Cfg>& sh, int first, int n, int vis,
                                             int all_vis, float scale, float cap) {
  const int lane = static_cast<int>(threadIdx.x & 31), quad = (threadIdx.x >> 5) & 3;
  const int row = 32 * quad + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
  const uint32_t t_s = lanes + Cfg::kTmS + static_cast<uint32_t>(first) * 64u;
  const uint32_t t_p = lanes + Cfg::kTmP + static_cast<uint32_t>(first) * 64u;
  float m = -INFINITY, l = 0.f;
  bool dead = false;
  // As registers allow: the tile's scores are held from one pass to the next, or go to where
  // its weights will be, a run of keys at a time; S is free from then on either way.
  constexpr bool kHold = Cfg::kHd <= 128;
  constexpr int kRun = kHold ? 32 : 16, kHeld = kHold ? kTileKeys / kRun : 1;
  dead = !__all_sync(0xFFFFFFFFu, mbar_wait(&sh.q_ready, 0));
  const float qs = q_unscale(sh, row);
  const float rowf = qs * scale * kLog2e;
  const SoftCap soft(kCap ? cap : 1.f);
  uint32_t ph = 0;
#pragma unroll 1
  for (int j = first; j < n; j += 2, ph ^= 1u) {
    const bool masked = (j + 1) * kTileKeys > all_vis;
    const int left = vis - j * kTileKeys;       // of the tile's keys, how many the row sees
    const int slot = j % Cfg::kMetas;
    const float* ks = sh.meta[slot].kscale;
    wait2(&sh.meta_full[slot], static_cast<uint32_t>(j / Cfg::kMetas) & 1u, &sh.s_full[first], ph,
          dead);
    tc_fence_after();
    uint32_t v[kHeld][kRun];
    if constexpr (kHold) {
#pragma unroll
      for (int r = 0; r < kHeld; ++r) tc_ld<kRun>(t_s + static_cast<uint32_t>(r * kRun), v[r]);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_free[first]);
    } else {
      // the buffer's last tile has been multiplied: the scores go there
      if (!__all_sync(0xFFFFFFFFu, mbar_test(&sh.p_free[first], ph ^ 1u)) && !dead)
        dead = !__all_sync(0xFFFFFFFFu, mbar_wait(&sh.p_free[first], ph ^ 1u));
      tc_fence_after();
    }
    float mx = -INFINITY;
#pragma unroll kHeld
    for (int r = 0; r < kTileKeys / kRun; ++r) {
      const int h = r * kRun;
      uint32_t(&vr)[kRun] = v[kHold ? r : 0];
      float x[kRun];
      if constexpr (!kHold) {
        tc_ld<kRun>(t_s + static_cast<uint32_t>(h), vr);
        tc_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < kRun; i += 4) {
        const float4 k = *reinterpret_cast<const float4*>(ks + h + i);
        const float2 f = make_float2(rowf, rowf);
        const float2 a = __fmul2_rn(bits2(vr[i], vr[i + 1]), __fmul2_rn(make_float2(k.x, k.y), f));
        const float2 b =
            __fmul2_rn(bits2(vr[i + 2], vr[i + 3]), __fmul2_rn(make_float2(k.z, k.w), f));
        x[i] = a.x; x[i + 1] = a.y; x[i + 2] = b.x; x[i + 3] = b.y;
      }
      if constexpr (kCap) soft_caps<kRun>(x, soft);
      if (masked) {
#pragma unroll
        for (int i = 0; i < kRun; ++i)
          if (h + i >= left) x[i] = -INFINITY;     // a select: nothing is multiplied
      }
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        mx = fmaxf(mx, x[i]);
        vr[i] = __float_as_uint(x[i]);
      }
      if constexpr (!kHold) tc_st<kRun>(t_p + static_cast<uint32_t>(h), vr);
    }
    if constexpr (!kHold) {
      tc_wait_st();
      tc_fence_before();
    }
    __syncwarp();
    // the scales are in what was stored, or in the maximum
    if (lane == 0 && (!kHold || !(mx > INFINITY))) {
      mbar_arrive(&sh.meta_free[slot]);
      if (!kHold) mbar_arrive(&sh.s_free[first]);
    }
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    l *= ex2(m - base);
    m = mn;
    const float sub = static_cast<float>(kPShift) - base;
    // the buffer's last tile has been multiplied (kHold), and its maximum read
    wait2(&sh.p_free[first], ph ^ 1u, &sh.m_free[first], ph ^ 1u, dead);
    tc_fence_after();
    sh.x[0][first][row] = m;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll kHeld
    for (int r = 0; r < kTileKeys / kRun; ++r) {
      uint32_t(&vr)[kRun] = v[kHold ? r : 0];
      if constexpr (!kHold) {
        tc_ld<kRun>(t_p + static_cast<uint32_t>(r * kRun), vr);
        tc_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < kRun; e += 16) {
        uint32_t w[16];              // hi, then lo
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float2 a = __fadd2_rn(bits2(vr[e + i], vr[e + i + 1]), make_float2(sub, sub));
          a.x = ex2(a.x);
          a.y = ex2(a.y);
          sum = __fadd2_rn(sum, a);
          split2(a, w[i / 2], w[8 + i / 2]);
        }
        tc_st<16>(t_p + static_cast<uint32_t>(r * kRun + e), w);
      }
    }
    l += sum.x + sum.y;
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.p_ready[first]);
  }
  sh.x[0][first][row] = m;
  sh.x[1][first][row] = l;
  return dead;
}

// O = sum over tiles of 2^(m_j - m) O_tile(j), in registers: a thread has half a row.
template <class Cfg>
__device__ __forceinline__ bool tile_sums(MmaShared<Cfg>& sh, int n, RowState<Cfg>& st) {
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int quad = warp & 3, part = warp >> 2, row = 32 * quad + lane;
  const uint32_t t_o = (static_cast<uint32_t>(32 * quad) << 16) + Cfg::kTmO +
                       static_cast<uint32_t>(part * Cfg::kOC);
  st.m = -INFINITY;
  st.any_left_out = false;
#pragma unroll
  for (int c = 0; c < Cfg::kNC; ++c)
#pragma unroll
    for (int i = 0; i < Cfg::kOC / 2; ++i) st.o[c][i] = make_float2(0.f, 0.f);
  bool dead = false;
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
  };
  RingAt<2> tile, buf;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const int b = tile.stage, slot = j % Cfg::kMetas;
    wait2(&sh.vmeta_full[slot], static_cast<uint32_t>(j / Cfg::kMetas) & 1u, &sh.p_ready[b],
          tile.phase, dead);
    tile.next();
    const float mj = sh.x[0][b][row], vs = sh.meta[slot].vscale;
    const bool left = (sh.meta[slot].left_out[0] | sh.meta[slot].left_out[1]) != 0;
    const float mn = fmaxf(st.m, mj), base = mn == -INFINITY ? 0.f : mn;
    const float alpha = ex2(st.m - base), beta = ex2(mj - base) * vs;
    st.m = mn;
    // the arrivals hang on the values read: loads that nothing has used yet may be
    // scheduled behind them (the vote is true in every lane: vs is a power of two)
    const uint32_t lefts = __ballot_sync(0xFFFFFFFFu, left && vs > 0.f);
    const bool read = __all_sync(0xFFFFFFFFu, !(beta < 0.f)) && (vs > 0.f || lefts);
    st.any_left_out = st.any_left_out || lefts;
    if (lane == 0 && read) {
      mbar_arrive(&sh.vmeta_free[slot]);
      mbar_arrive(&sh.m_free[b]);
    }
#pragma unroll
    for (int c = 0; c < Cfg::kNC; ++c) {
      wait(&sh.o_full[buf.stage], buf.phase);
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < Cfg::kOC; h += 16) {
        uint32_t v[16];
        tc_ld<16>(t_o + static_cast<uint32_t>(buf.stage) * 64u + static_cast<uint32_t>(h), v);
        tc_wait_ld();
        if (h + 16 == Cfg::kOC) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.o_free[buf.stage]);
          buf.next();
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float2& o = st.o[c][(h + i) / 2];
          o = __ffma2_rn(o, make_float2(alpha, alpha),
                         __fmul2_rn(bits2(v[i], v[i + 1]), make_float2(beta, beta)));
        }
      }
    }
  }
  return dead;
}

// Key tiles of every sequence and kv head, split and laid out once (they are
// read by all of the sequence's query tiles).  grid (key tiles, n_kv, 2): K, then V, apart,
// as a CTA is one chain of a read, a reduction and a write.
template <int kHd>
__global__ void __launch_bounds__(256) prompt_pack_kernel(const __grid_constant__ PromptParams p) {
  using Cfg = PromptCfg<kHd>;
  pdl_launch_dependents();
  pdl_wait();
  const int tile = blockIdx.x, g = blockIdx.y;
  const int s = find_seq(p.seqs.ktile, p.seqs.n, tile);
  const int64_t key = p.seqs.k0[s] + static_cast<int64_t>(tile - p.seqs.ktile[s]) * kTileKeys;
  const int n = static_cast<int>(min(static_cast<int64_t>(kTileKeys), p.seqs.k0[s + 1] - key));
  const int64_t at = static_cast<int64_t>(tile) * p.n_kv + g;
  uint8_t* dst = p.packed + at * Cfg::kTile;
  if (blockIdx.z == 0)
    pack_keys<Cfg>(p.k.data + key * p.k.token_stride + g * p.k.head_stride, p.k.token_stride, n,
                   dst, p.meta + at);
  else
    pack_values<Cfg>(p.v.data + key * p.v.token_stride + g * p.v.head_stride, p.v.token_stride,
                     n, dst + Cfg::kHalfTile, p.meta + at);
}

// One item per CTA: 128 rows of one kv head against its piece of the keys.
template <int kHd, bool kCap>
__global__ void __launch_bounds__(PromptCfg<kHd>::kThreads, 1)
    prompt_mma_kernel(const __grid_constant__ PromptParams p) {
  using Cfg = PromptCfg<kHd>;
  extern __shared__ uint8_t raw[];
  uint8_t* stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  uint8_t* q_lo = stages + Cfg::kRing;
  auto& sh = *reinterpret_cast<MmaShared<Cfg>*>(stages + Cfg::kSmem);
  pdl_launch_dependents();
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  // before the item is looked up, which takes the other warps as long
  if (warp == Cfg::kMmaPv && lane == 0) mma_init_barriers<Cfg>(sh, 1, 1);
  if (warp == Cfg::kMmaQk) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  const int item = blockIdx.x / p.n_kv, g = blockIdx.x - item * p.n_kv;
  const PromptItem it = prompt_item(p, item);
  const int ka = it.piece * p.chunk, kb = min(it.vis, ka + p.chunk);
  const int n = kb > ka ? (kb - ka + kTileKeys - 1) / kTileKeys : 0;
  const int64_t tile0 = p.seqs.ktile[it.s] + ka / kTileKeys;    // its packed tiles
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  uint8_t* k_ring = stages;
  uint8_t* v_ring = stages + Cfg::kStages * Cfg::kUnit;
  // this thread's row, as output or as softmax warp
  const int row = 32 * (warp & 3) + lane;
  const int live = it.n_tok * p.group;
  const int r = min(row, live - 1);
  const int i = it.i0 + r / p.group, h = g * p.group + r % p.group;
  const int vis = visible(i, it.n_q, it.n_k) - ka;
  if (warp >= Cfg::kLoadK) {
    regs_dec<kRegsHelp<kHd>>();
    const auto packed = [&](int j) { return p.packed + ((tile0 + j) * p.n_kv + g) * Cfg::kTile; };
    if (warp == Cfg::kLoadK && lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      mma_load<Cfg>(
          sh.k_full, sh.k_empty, n,
          [&](int j) {
            const int s = j % Cfg::kMetas;
            if (!mbar_wait(&sh.meta_free[s], (static_cast<uint32_t>(j / Cfg::kMetas) & 1u) ^ 1u))
              return false;
            mbar_arrive_expect_tx(&sh.meta_full[s], sizeof(TileMeta::kscale));
            bulk_copy_g2s(&sh.meta[s], p.meta + (tile0 + j) * p.n_kv + g,
                          sizeof(TileMeta::kscale), &sh.meta_full[s], pol);
            return true;
          },
          [&](int s, int j, int c) {
            mbar_arrive_expect_tx(&sh.k_full[s], Cfg::kUnit);
            bulk_copy_g2s(k_ring + s * Cfg::kUnit, packed(j) + c * Cfg::kUnit, Cfg::kUnit,
                          &sh.k_full[s], pol);
          },
          &g_err_prompt);
    }
    if (warp == Cfg::kLoadV && lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      mma_load<Cfg>(
          sh.v_full, sh.v_empty, n,
          [&](int j) {
            // the ring is the softmax warps' scratch until Q is stored
            if (j == 0 && !mbar_wait(&sh.q_ready, 0)) return false;
            const int s = j % Cfg::kMetas;
            if (!mbar_wait(&sh.vmeta_free[s], (static_cast<uint32_t>(j / Cfg::kMetas) & 1u) ^ 1u))
              return false;
            mbar_arrive_expect_tx(&sh.vmeta_full[s], 16);
            bulk_copy_g2s(&sh.meta[s].vscale, &p.meta[(tile0 + j) * p.n_kv + g].vscale, 16,
                          &sh.vmeta_full[s], pol);
            return true;
          },
          [&](int s, int j, int c) {
            mbar_arrive_expect_tx(&sh.v_full[s], Cfg::kUnit);
            bulk_copy_g2s(v_ring + s * Cfg::kUnit, packed(j) + Cfg::kHalfTile + c * Cfg::kUnit,
                          Cfg::kUnit, &sh.v_full[s], pol);
          },
          &g_err_prompt);
    }
    if (warp == Cfg::kMmaQk) mma_issue_qk<Cfg>(sh, k_ring, q_lo, n, &g_err_prompt);
    if (warp == Cfg::kMmaPv) mma_issue_pv<Cfg>(sh, v_ring, n, &g_err_prompt);
  } else if (warp >= Cfg::kRowsWarps) {
    if constexpr (kHd > 128) regs_dec<kRegsSoft<kHd>>();
    else regs_inc<kRegsSoft<kHd>>();
    const bool dead = tile_weights<Cfg, kCap>(sh, (warp - Cfg::kRowsWarps) >> 2, n, vis,
                                              visible(it.i0, it.n_q, it.n_k) - ka, p.scale, p.cap);
    if (dead) sh.dead = 1;
    bar_sync(5, 32 * 16);
  } else {
    regs_inc<kRegsOut<kHd>>();
    const int part = warp >> 2;
    const bool alive = row < live;
    const int64_t token = p.seqs.q0[it.s] + i;
    const float* q = p.q.data + token * p.q.token_stride + h * p.q.head_stride;
    RowState<Cfg> st;
    float* scratch = reinterpret_cast<float*>(v_ring);
    store_q<Cfg>(sh, scratch, q_lo, alive ? q : nullptr);
    if (tile_sums<Cfg>(sh, n, st)) sh.dead = 1;
    bar_sync(5, 32 * 16);
    const bool dead = *reinterpret_cast<volatile uint32_t*>(&sh.dead) != 0;
    {
      const float base = st.m == -INFINITY ? 0.f : st.m;
      st.l = sh.x[1][0][row] * ex2(sh.x[0][0][row] - base) +
             sh.x[1][1][row] * ex2(sh.x[0][1][row] - base);
    }
    if (dead && lane == 0) atomicOr(&g_err_prompt, kErrAttRows);
    if (st.any_left_out && alive) {
      for (int j = 0; j < n; ++j) {
        const TileMeta& m = p.meta[(tile0 + j) * p.n_kv + g];
        for (int t = 0; t < kTileKeys; ++t) {
          if (!((m.left_out[t >> 5] >> (t & 31)) & 1u) || j * kTileKeys + t >= vis) continue;
          const int64_t key = p.seqs.k0[it.s] + ka + j * kTileKeys + t;
          add_left_out<Cfg>(st, q, p.k.data + key * p.k.token_stride + g * p.k.head_stride,
                            p.v.data + key * p.v.token_stride + g * p.v.head_stride, part,
                            p.scale, p.cap);
        }
      }
    }
    constexpr float kUnshift = 1.0f / (1 << kPShift);
    const bool store = alive && !dead;
    if (it.pieces > 1) {
      float* dst = part_rows(p, item, g, kHd) + row * (kHd + kPartPad);
      store_rows<Cfg>(st, scratch, store ? dst : nullptr, kUnshift);
      if (store && part == 0)
        *reinterpret_cast<float2*>(dst + kHd) = make_float2(st.m, st.l * kUnshift);
    } else {
      float* dst = p.out.data + token * p.out.token_stride + h * p.out.head_stride;
      store_rows<Cfg>(st, scratch, store ? dst : nullptr, st.l == 0.f ? 0.f : 1.0f / st.l);
    }
  }
  // every MMA has completed before tensor memory is freed
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::kMmaQk) {
    for (int i = 0; i < 2; ++i)
      if (lane == 0 && !mbar_wait(&sh.done[i], 0)) atomicOr(&g_err_prompt, kErrAttMma);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(sh.tmem, 512);
  }
}

// ------------------------------------------------------------ host side
namespace {

// (query row, key) pairs of all heads from which the tensor cores, whose two or three
// launches and packing take 8 us (head_dim 32) to 17 (256) at least, take a call.  Device time
// on CUDA cores / tensor cores at half of it, at it and at twice: 4 q / 4 kv heads of 32 6.6 / 7.9,
// 8.9 / 8.3, 12.4 / 9.4 us; 8 / 2 of 64 7.2 / 8.7, 9.1 / 9.1, 13.4 / 9.9; 8 / 4 of 128 10.3 / 11.3,
// 13.3 / 12.1, 18.6 / 12.8; 8 / 4 of 256 16.0 / 16.9, 21.5 / 18.2, 25.8 / 19.5.  A few queries
// on 2000 keys, just below: 8.7 / 11.6, 10.4 / 11.6, 13.2 / 15.6, 24.3 / 24.7.
constexpr int64_t kMmaFrom = 1 << 16;
// Up to this many tiles of four rows a warp, one row a warp: each then still has its SM.
// 37 tokens of 8 q / 4 kv heads of 256: 16.7 -> 9.4 us.  Longer prompts read the keys more
// often for it (300 tokens of 4 / 1 heads of 64, 38 tiles: 17.9 us with four rows, 20.4 with
// one), but most of those are the tensor cores'.
constexpr int64_t kOneRowTiles = 38;

struct PromptPlan {
  bool mma;             // on the tensor cores
  bool one;             // if not: one row a warp in place of four
  int rows, tok, chunk;
  bool split;           // some tile has several pieces
  int64_t items, ktiles;        // per kv head, of the largest launch
  size_t packed_bytes, meta_bytes, part_bytes;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// items of a sequence, as prompt_item counts them
int64_t seq_items(int64_t nq, int64_t nk, int tok, int chunk) {
  if (nq == 0) return 0;
  const int64_t tiles = ceil_div(nq, tok);
  int64_t items = tiles;
  for (int64_t piece = 1; piece * chunk < nk; ++piece)
    items += tiles - first_tile(static_cast<int>(piece), chunk, tok, static_cast<int>(nq),
                                static_cast<int>(nk));
  return items;
}

// The sequences s0 .. s0 + n - 1 in the order of their items.
void order_seqs(const int64_t* cu_q, const int64_t* cu_k, int s0, int n, int* order) {
  for (int i = 0; i < n; ++i) order[i] = i;
  const auto keys = [&](int i) {
    return cu_q[s0 + i + 1] > cu_q[s0 + i] ? cu_k[s0 + i + 1] - cu_k[s0 + i] : -1;
  };
  std::stable_sort(order, order + n, [&](int a, int b) { return keys(a) > keys(b); });
}

// When the last item ends, in steps of `unit` keys, if pieces are c steps long, an item
// costs kItemSteps more than its steps, and the items start in their order on `slots`
// places: a count of free places per time.  What bounds the host's time: equal items in a row
// are placed together, times are rounded up to 1 / 1024 of a piece, behind kPlaced
// placements the rest (work, as if no tile were cut) is taken to fill the places evenly, and
// after kWeighed placements for all the lengths no other length is weighed.  512 queries on
// 8000 keys 8 us, 64 single ones on 8000 keys each 95, 4000 prompts of 20 tokens beside one of
// 2000 240 (item by item 600; 128 queries on 2^24 keys 9, and were 190).
//
// kItemSteps: an item of 3100 to 3800 cycles a tile has some 15000 beside its tiles (its Q,
// first scores, output and the next launch).
constexpr int64_t kItemSteps = 5;
constexpr int64_t kJoinSteps = 2;        // of prompt_merge_kernel
constexpr int kPlaced = 2048, kWeighed = 16384;
struct SeqWork {
  int64_t nq, nk, tiles;
  int64_t steps;       // of its last tile
  int64_t work;        // of this sequence and all behind it
};
int64_t end_of_items(const std::vector<SeqWork>& seqs, int n_kv, int tok, int64_t c, int unit,
                     int slots, int* placed) {
  const int64_t tick = ceil_div(c, 1024);
  std::vector<int> free_at(static_cast<size_t>((c + kItemSteps) / tick) + 2, 0);
  free_at[0] = slots;
  size_t now = 0, last = 0;
  int64_t held = -1, many = 0;           // items of as many steps, not placed yet
  const auto flush = [&]() {
    if (many == 0) return;
    const size_t size = static_cast<size_t>(ceil_div(held + kItemSteps, tick));
    ++*placed;
    while (many > 0) {
      while (free_at[now] == 0) ++now;
      const int take = static_cast<int>(std::min<int64_t>(many, free_at[now]));
      free_at[now] -= take;
      if (free_at.size() <= now + size) free_at.resize(2 * (now + size) + 1, 0);
      free_at[now + size] += take;
      last = std::max(last, now + size);
      many -= take;
    }
  };
  const auto place = [&](int64_t steps, int64_t m) {
    if (steps != held) {
      flush();
      held = steps;
    }
    many += m;
  };
  const int64_t chunk = c * unit;
  const int limit = *placed + kPlaced;
  for (const SeqWork& q : seqs) {
    if (*placed >= limit) {
      flush();
      int64_t busy = q.work / tick;
      for (size_t t = now; t < free_at.size(); ++t) busy += static_cast<int64_t>(t) * free_at[t];
      last = std::max(last, static_cast<size_t>(ceil_div(busy, slots)));
      break;
    }
    if (q.tiles == 1 && q.nk <= chunk) {
      place(q.steps, n_kv);
      continue;
    }
    for (int64_t piece = 0; q.tiles > 0 && (piece == 0 || piece * chunk < q.nk); ++piece) {
      const int64_t from = first_tile(static_cast<int>(piece), static_cast<int>(chunk), tok,
                                      static_cast<int>(q.nq), static_cast<int>(q.nk));
      const auto steps = [&](int64_t tile) {
        const int64_t row = std::min(q.nq, (tile + 1) * tok) + q.nk - q.nq;
        return std::min(c,
                        ceil_div(std::max<int64_t>(0, std::min(row, q.nk) - piece * chunk), unit));
      };
      int64_t tile = q.tiles - 1;
      if (steps(tile) == c) {
        // so do the tiles before it, down to the first that sees the whole piece
        int64_t lo = from, hi = tile;
        while (lo < hi) {
          const int64_t mid = (lo + hi) / 2;
          if (steps(mid) == c) hi = mid;
          else lo = mid + 1;
        }
        place(c, (tile - lo + 1) * n_kv);
        tile = lo - 1;
      }
      for (; tile >= from && *placed < limit; --tile) place(steps(tile), n_kv);
    }
  }
  flush();
  return static_cast<int64_t>(last) * tick;
}

// The form, tile and piece lengths of a call, and the sizes of its workspace.
PromptPlan plan_prompt(const int64_t* cu_q, const int64_t* cu_k, int n_seqs, int n_q, int n_kv,
                       int head_dim) {
  PromptPlan pl = {};
  const int group = n_q / n_kv;
  // (row, key) pairs that are scored, per kv head, and the longest sequence's keys
  int64_t pairs = 0, longest = 1;
  for (int s = 0; s < n_seqs; ++s) {
    const int64_t nq = cu_q[s + 1] - cu_q[s], nk = cu_k[s + 1] - cu_k[s];
    pairs += nq * group * std::max<int64_t>(1, nk - std::min(nq, nk) / 2);
    if (nq) longest = std::max(longest, nk);
  }
  pl.mma = pairs * n_kv >= kMmaFrom;
  int64_t tiles = 0;           // of 4 rows a warp
  for (int s = 0; s < n_seqs; ++s)
    tiles += ceil_div(cu_q[s + 1] - cu_q[s], 4 * kRowWarps / group) * n_kv;
  pl.one = tiles <= kOneRowTiles;
  pl.rows = pl.mma ? kTileRows : pl.one ? kRowWarps : 4 * kRowWarps;
  pl.tok = pl.rows / group;
  const int unit = pl.mma ? kTileKeys : 32;         // keys of a step
  const int slots = pl.mma ? 152 : 304;             // items that run at once
  // steps of the longest tile, and an SM's share of all
  const int64_t steps = ceil_div(longest, unit);
  const int64_t total = ceil_div(pairs * n_kv, static_cast<int64_t>(pl.rows) * unit);
  // A tile is cut where it is longer than an SM's share of the work, into pieces of the
  // length that ends first: a k-th of the longest tile, k = 1 .. 32, or some less, which
  // leaves the last pieces short enough to fill up the rest (512 queries on 8000 keys: 27
  // steps in place of 32, 115 -> 107 us).  Cutting sooner evens the SMs out, but costs more
  // partial results than that (8192 positions: 551 us whole, 569 cut).
  int64_t best = steps;
  if (steps * slots > total) {
    int64_t best_end = INT64_MAX, tried = steps + 1;
    std::vector<SeqWork> seqs(static_cast<size_t>(n_seqs));
    for (int s0 = 0; s0 < n_seqs; s0 += kMaxSeqs) {
      int order[kMaxSeqs];
      const int n = std::min(n_seqs - s0, kMaxSeqs);
      order_seqs(cu_q, cu_k, s0, n, order);
      for (int i = 0; i < n; ++i) {
        SeqWork& q = seqs[static_cast<size_t>(s0 + i)];
        const int s = s0 + order[i];
        q.nq = cu_q[s + 1] - cu_q[s];
        q.nk = cu_k[s + 1] - cu_k[s];
        q.tiles = ceil_div(q.nq, pl.tok);
        q.steps = ceil_div(q.nk, unit);
      }
    }
    int64_t work = 0;
    for (size_t i = seqs.size(); i-- > 0;) {
      const int64_t keys = seqs[i].nk - std::min(seqs[i].nq, seqs[i].nk) / 2 + unit / 2;
      work += seqs[i].tiles * n_kv * (kItemSteps + keys / unit);
      seqs[i].work = work;
    }
    int placed = 0;
    for (int64_t k = 1; k <= 32 && placed < kWeighed; k += k < 6 ? 1 : k < 12 ? 2 : 4) {
      for (int less = 0; less < (k < 6 ? 3 : 1); ++less) {
        const int64_t c = ceil_div(steps, k) * (16 - less) / 16;
        if (c >= tried) continue;
        tried = c;
        if (c < 2 && c < steps) break;
        if (ceil_div(steps, c) > 32) break;             // of a tile, at most
        const int64_t end = end_of_items(seqs, n_kv, pl.tok, c, unit, slots, &placed) +
                            (c < steps ? kJoinSteps : 0);
        if (end < best_end) {
          best_end = end;
          best = c;
        }
      }
    }
  }
  pl.chunk = static_cast<int>(best) * unit;
  for (int s0 = 0; s0 < n_seqs; s0 += kMaxSeqs) {
    int64_t items = 0, ktiles = 0;
    for (int s = s0; s < std::min(n_seqs, s0 + kMaxSeqs); ++s) {
      const int64_t nq = cu_q[s + 1] - cu_q[s], nk = cu_k[s + 1] - cu_k[s];
      if (nq == 0) continue;
      items += seq_items(nq, nk, pl.tok, pl.chunk);
      ktiles += ceil_div(nk, kTileKeys);
      pl.split = pl.split || nk > pl.chunk;
    }
    pl.items = std::max(pl.items, items);
    pl.ktiles = std::max(pl.ktiles, ktiles);
  }
  const auto pad = [](size_t v) { return (v + 255) / 256 * 256; };
  if (pl.mma) {
    const size_t tile = head_dim == 32   ? PromptCfg<32>::kTile
                        : head_dim == 64 ? PromptCfg<64>::kTile
                        : head_dim == 128 ? PromptCfg<128>::kTile
                                          : PromptCfg<256>::kTile;
    pl.packed_bytes = pad(static_cast<size_t>(pl.ktiles) * n_kv * tile);
    pl.meta_bytes = pad(static_cast<size_t>(pl.ktiles) * n_kv * sizeof(TileMeta));
  }
  if (pl.split)
    pl.part_bytes = pad(static_cast<size_t>(pl.items) * n_kv * pl.rows *
                        (head_dim + kPartPad) * sizeof(float));
  return pl;
}

template <int kPL>
cudaError_t run_prompt(PromptParams& p, const PromptPlan& pl, int64_t items, int64_t ktiles,
                       cudaStream_t st) {
  constexpr int kHd = kPL * 32;
  const dim3 grid(static_cast<unsigned>(items * p.n_kv));
  cudaError_t e;
  if (pl.mma) {
    using Cfg = PromptCfg<kHd>;
    constexpr size_t kSmem = 1024 + Cfg::kSmem + sizeof(MmaShared<Cfg>);
    static_assert(kSmem <= 227 * 1024, "shared memory");
    if (ktiles > 0) {
      e = pdl_launch(prompt_pack_kernel<kHd>,
                     dim3(static_cast<unsigned>(ktiles), static_cast<unsigned>(p.n_kv), 2), 256, 0,
                     st, p);
      if (e != cudaSuccess) return e;
    }
    const auto kernel = p.cap > 0.f ? prompt_mma_kernel<kHd, true> : prompt_mma_kernel<kHd, false>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    e = pdl_launch(kernel, grid, Cfg::kThreads, kSmem, st, p);
  } else {
    const auto kernel = pl.one ? prompt_rows_kernel<kPL, 1> : prompt_rows_kernel<kPL, 4>;
    const size_t smem = pl.one ? RowTile<kPL, 1>::kSmem : RowTile<kPL, 4>::kSmem;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    e = pdl_launch(kernel, grid, kRowThreads, smem, st, p);
  }
  if (e != cudaSuccess || !pl.split) return e;
  const int64_t rows = static_cast<int64_t>(p.seqs.q0[p.seqs.n] - p.seqs.q0[0]) * p.n_q;
  return pdl_launch(prompt_merge_kernel<kPL>, dim3(static_cast<unsigned>((rows + 7) / 8)), 256,
                    0, st, p);
}

}  // namespace

size_t prompt_attention_workspace_bytes(const int64_t* cu_q, const int64_t* cu_k, int n_seqs,
                                        int n_q, int n_kv, int head_dim) {
  const PromptPlan pl = plan_prompt(cu_q, cu_k, n_seqs, n_q, n_kv, head_dim);
  return pl.packed_bytes + pl.meta_bytes + pl.part_bytes;
}

qws_status launch_prompt_attention(const qws_heads& q, const qws_heads& k, const qws_heads& v,
                                   const qws_heads& out, const int64_t* cu_q,
                                   const int64_t* cu_k, int n_seqs, int n_q, int n_kv,
                                   int head_dim, float scale, float cap, void* ws,
                                   size_t ws_bytes, size_t* need, cudaStream_t st,
                                   cudaError_t* err) {
  const PromptPlan pl = plan_prompt(cu_q, cu_k, n_seqs, n_q, n_kv, head_dim);
  *need = pl.packed_bytes + pl.meta_bytes + pl.part_bytes;
  if (*need && (!ws || ws_bytes < *need)) return QWS_ERR_WORKSPACE;
  PromptParams p;
  p.q = q; p.k = k; p.v = v; p.out = out;
  p.packed = static_cast<uint8_t*>(ws);
  p.meta = reinterpret_cast<TileMeta*>(p.packed + pl.packed_bytes);
  p.part = reinterpret_cast<float*>(p.packed + pl.packed_bytes + pl.meta_bytes);
  p.n_q = n_q; p.n_kv = n_kv; p.group = n_q / n_kv;
  p.tok = pl.tok; p.rows = pl.rows; p.chunk = pl.chunk;
  p.scale = scale; p.cap = cap;
  for (int s0 = 0; s0 < n_seqs; s0 += kMaxSeqs) {
    SeqTab& t = p.seqs;
    t.n = std::min(n_seqs - s0, kMaxSeqs);
    int64_t items = 0, ktiles = 0;
    for (int s = 0; s <= t.n; ++s) {
      t.q0[s] = static_cast<int>(cu_q[s0 + s]);
      t.k0[s] = static_cast<int>(cu_k[s0 + s]);
      t.ktile[s] = static_cast<int>(ktiles);
      if (s < t.n && t.q0[s] < cu_q[s0 + s + 1])
        ktiles += ceil_div(cu_k[s0 + s + 1] - cu_k[s0 + s], kTileKeys);
    }
    order_seqs(cu_q, cu_k, s0, t.n, t.order);
    for (int i = 0; i < t.n; ++i) {
      const int s = t.order[i];
      t.item[i] = t.first[s] = static_cast<int>(items);
      items += seq_items(t.q0[s + 1] - t.q0[s], t.k0[s + 1] - t.k0[s], pl.tok, pl.chunk);
    }
    t.item[t.n] = static_cast<int>(items);
    if (items == 0) continue;
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 32: e = run_prompt<1>(p, pl, items, ktiles, st); break;
      case 64: e = run_prompt<2>(p, pl, items, ktiles, st); break;
      case 128: e = run_prompt<4>(p, pl, items, ktiles, st); break;
      case 256: e = run_prompt<8>(p, pl, items, ktiles, st); break;
    }
    if (e != cudaSuccess) {
      *err = e;
      return QWS_ERR_CUDA;
    }
  }
  return QWS_OK;
}

unsigned read_clear_prompt_errors() {
  unsigned v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_prompt, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_err_prompt, &z, sizeof(z));
  return v;
}

}  // namespace qws
