// prompt.cu -- causal attention over packed prompts (the seq > 1 counterpart
// of kv_attention): for query row i of a sequence with n_q rows and n_k keys,
// head h reading kv head h / group,
//   s_j = softcap(scale * q_ih . k_j)  for the visible keys j <= i + n_k - n_q,
//   out_ih = sum_j softmax(s)_j v_j;   a row without a visible key gives zeros.
#include <cuda_runtime.h>

#include <algorithm>

#include "attend_rows.cuh"
#include "launch.h"

namespace qws {

// ------------------------------------------------------------ work items
// A tile is `rows` query rows of one kv head: tok = rows / group tokens with
// the group's heads side by side, row r = token r / group, head r % group.  Its
// keys are cut into pieces of `chunk`; an item is one piece.  A sequence's
// items are a rectangle (pieces of its last tile x tiles): pieces beyond a
// tile's visible keys do nothing.  A tile of one piece writes out, the others
// leave partials that prompt_merge_kernel joins.
struct PromptParams {
  qws_heads q, k, v, out;
  float* part;
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

__device__ __forceinline__ PromptItem prompt_item(const PromptParams& p, int item) {
  PromptItem it;
  it.s = find_seq(p.seqs.item, p.seqs.n, item);
  it.n_q = p.seqs.q0[it.s + 1] - p.seqs.q0[it.s];
  it.n_k = p.seqs.k0[it.s + 1] - p.seqs.k0[it.s];
  it.tiles = (it.n_q + p.tok - 1) / p.tok;
  const int local = item - p.seqs.item[it.s];
  it.piece = local / it.tiles;
  it.tile = it.tiles - 1 - (local - it.piece * it.tiles);   // the longest first
  tile_span(p, it);
  return it;
}

__device__ __forceinline__ int64_t part_slot(const PromptParams& p, const PromptItem& it,
                                             int piece, int g) {
  const int item = p.seqs.item[it.s] + piece * it.tiles + (it.tiles - 1 - it.tile);
  return static_cast<int64_t>(item) * p.n_kv + g;
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
  const PromptItem it = prompt_item(p, blockIdx.x);
  if (it.piece >= it.pieces) return;
  const int g = blockIdx.y;
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
      store_partial<kPL>(
          p.part + (part_slot(p, it, it.piece, g) * p.rows + row) * (kHd + kPartPad), lane,
          tile.acc[r], tile.m[r], tile.l[r]);
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
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int total = p.seqs.q0[p.seqs.n] - p.seqs.q0[0];
  const int64_t t = w / p.n_q;
  if (t >= total) return;
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
  if (it.pieces < 2) return;
  const int row = (i - it.i0) * p.group + (h - g * p.group);
  float m = -INFINITY, l = 0.f, acc[kPL];
#pragma unroll
  for (int j = 0; j < kPL; ++j) acc[j] = 0.f;
  for (int c = 0; c < it.pieces; ++c) {
    const float* src = p.part + (part_slot(p, it, c, g) * p.rows + row) * (kHd + kPartPad);
    float x[kPL];
    load_row<kPL>(src, lane, x);
    const float mc = src[kHd], lc = src[kHd + 1];
    const float mn = fmaxf(m, mc);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float a = expf(m - base), b = expf(mc - base);
    l = fmaf(l, a, lc * b);
#pragma unroll
    for (int j = 0; j < kPL; ++j) acc[j] = fmaf(acc[j], a, x[j] * b);
    m = mn;
  }
  store_final<kPL>(p.out.data + static_cast<int64_t>(token) * p.out.token_stride +
                       h * p.out.head_stride,
                   lane, acc, l);
}

// ------------------------------------------------------------ host side
namespace {

struct PromptPlan {
  int rows, tok, chunk;
  int64_t items;        // work items per kv head of the largest launch
  bool split;           // some tile has several pieces
};

// The tile and piece lengths of a call, and the workspace of its partials.
PromptPlan plan_prompt(const int64_t* cu_q, const int64_t* cu_k, int n_seqs, int group) {
  PromptPlan pl;
  pl.rows = 4 * kRowWarps;
  pl.tok = pl.rows / group;
  pl.chunk = 512;
  pl.items = 0;
  pl.split = false;
  for (int s0 = 0; s0 < n_seqs; s0 += kMaxSeqs) {
    int64_t items = 0;
    for (int s = s0; s < std::min(n_seqs, s0 + kMaxSeqs); ++s) {
      const int64_t nq = cu_q[s + 1] - cu_q[s], nk = cu_k[s + 1] - cu_k[s];
      if (nq == 0) continue;
      const int64_t pieces = std::max<int64_t>(1, (nk + pl.chunk - 1) / pl.chunk);
      items += (nq + pl.tok - 1) / pl.tok * pieces;
      pl.split = pl.split || pieces > 1;
    }
    pl.items = std::max(pl.items, items);
  }
  return pl;
}

template <int kPL>
cudaError_t run_prompt(PromptParams& p, const PromptPlan& pl, int64_t items, cudaStream_t st) {
  using Tile = RowTile<kPL, 4>;
  cudaError_t e = cudaFuncSetAttribute(prompt_rows_kernel<kPL, 4>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(Tile::kSmem));
  if (e != cudaSuccess) return e;
  e = pdl_launch(prompt_rows_kernel<kPL, 4>,
                 dim3(static_cast<unsigned>(items), static_cast<unsigned>(p.n_kv)), kRowThreads,
                 Tile::kSmem, st, p);
  if (e != cudaSuccess || !pl.split) return e;
  const int64_t rows = static_cast<int64_t>(p.seqs.q0[p.seqs.n] - p.seqs.q0[0]) * p.n_q;
  return pdl_launch(prompt_merge_kernel<kPL>, dim3(static_cast<unsigned>((rows + 7) / 8)), 256,
                    0, st, p);
}

}  // namespace

size_t prompt_attention_workspace_bytes(const int64_t* cu_q, const int64_t* cu_k, int n_seqs,
                                        int n_q, int n_kv, int head_dim) {
  const PromptPlan pl = plan_prompt(cu_q, cu_k, n_seqs, n_q / n_kv);
  if (!pl.split) return 0;
  return static_cast<size_t>(pl.items) * n_kv * pl.rows * (head_dim + kPartPad) * sizeof(float);
}

cudaError_t launch_prompt_attention(const qws_heads& q, const qws_heads& k, const qws_heads& v,
                                    const qws_heads& out, const int64_t* cu_q,
                                    const int64_t* cu_k, int n_seqs, int n_q, int n_kv,
                                    int head_dim, float scale, float cap, void* ws,
                                    cudaStream_t st) {
  const PromptPlan pl = plan_prompt(cu_q, cu_k, n_seqs, n_q / n_kv);
  PromptParams p;
  p.q = q; p.k = k; p.v = v; p.out = out;
  p.part = static_cast<float*>(ws);
  p.n_q = n_q; p.n_kv = n_kv; p.group = n_q / n_kv;
  p.tok = pl.tok; p.rows = pl.rows; p.chunk = pl.chunk;
  p.scale = scale; p.cap = cap;
  for (int s0 = 0; s0 < n_seqs; s0 += kMaxSeqs) {
    SeqTab& t = p.seqs;
    t.n = std::min(n_seqs - s0, kMaxSeqs);
    int64_t items = 0;
    for (int s = 0; s <= t.n; ++s) {
      t.q0[s] = static_cast<int>(cu_q[s0 + s]);
      t.k0[s] = static_cast<int>(cu_k[s0 + s]);
      t.item[s] = static_cast<int>(items);
      if (s == t.n) break;
      const int64_t nq = cu_q[s0 + s + 1] - cu_q[s0 + s], nk = cu_k[s0 + s + 1] - cu_k[s0 + s];
      if (nq)
        items += (nq + pl.tok - 1) / pl.tok * std::max<int64_t>(1, (nk + pl.chunk - 1) / pl.chunk);
    }
    if (items == 0) continue;
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 32: e = run_prompt<1>(p, pl, items, st); break;
      case 64: e = run_prompt<2>(p, pl, items, st); break;
      case 128: e = run_prompt<4>(p, pl, items, st); break;
      case 256: e = run_prompt<8>(p, pl, items, st); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qws
