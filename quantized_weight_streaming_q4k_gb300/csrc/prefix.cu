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

#include "attend_rows.cuh"
#include "launch.h"

namespace qws {

constexpr int kOwnChunk = 128;      // keys of an own-cache item
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

// grid (pieces * row tiles, n_kv)
template <int kPL, int kR>
__global__ void __launch_bounds__(kRowThreads)
    prefix_rows_kernel(const __grid_constant__ PrefixParams p) {
  using Tile = RowTile<kPL, kR>;
  constexpr int kHd = Tile::kHd;
  extern __shared__ __align__(16) float smem[];
  pdl_launch_dependents();
  pdl_wait();
  const int piece = blockIdx.x / p.row_tiles, rt = blockIdx.x - piece * p.row_tiles;
  const int g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.batch * p.group;
  const int ka = piece * p.chunk, kb = min(p.n_prefix, ka + p.chunk);
  Tile tile;
  tile.init();
  int vis[kR];
  float* qs = Tile::q_rows(smem);
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int row = rt * (kRowWarps * kR) + warp * kR + r;
    float x[kPL];
#pragma unroll
    for (int j = 0; j < kPL; ++j) x[j] = 0.f;
    vis[r] = 0;
    if (row < rows) {
      vis[r] = p.n_prefix;
      load_row<kPL>(p.q.data + static_cast<int64_t>(p.b0 + row / p.group) * p.q.token_stride +
                        (g * p.group + row % p.group) * p.q.head_stride,
                    lane, x);
    }
    store_row<kPL>(qs + r * kHd, lane, x);
  }
  tile.run(smem, p.kp + g * p.max_prefix * kHd, p.vp + g * p.max_prefix * kHd, kHd, kHd, ka, kb,
           vis, p.scale, p.cap);
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int row = rt * (kRowWarps * kR) + warp * kR + r;
    if (row < rows)
      store_partial<kPL>(p.part + prefix_part<kPL>(p, piece, g, row), lane, tile.acc[r],
                         tile.m[r], tile.l[r]);
  }
}

// Own parts: grid (own items, n_kv).  A warp takes keys w, w + 8, ... of the
// item's piece in fours: K and V rows straight from memory, a lane holding its
// columns, the dot products by warp sums; the warps are joined in shared memory
// in order.
constexpr int kOwnWarps = 8;
constexpr int kOwnKeys = 4;

template <int kPL, int kG>
__global__ void __launch_bounds__(kOwnWarps * 32)
    own_part_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int kHd = kPL * 32;
  __shared__ __align__(16) float sacc[kOwnWarps][kG][kHd];
  __shared__ float sm[kOwnWarps][kG], sl[kOwnWarps][kG];
  pdl_launch_dependents();
  pdl_wait();
  const int b = find_seq(p.first, p.batch, blockIdx.x);
  const int g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ka = (blockIdx.x - p.first[b]) * kOwnChunk, kb = min(p.n_ctx[b], ka + kOwnChunk);
  const int64_t head = (static_cast<int64_t>(p.b0 + b) * p.n_kv + g) * p.max_seq * kHd;
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
  for (int t = ka + warp * kOwnKeys; t < kb; t += kOwnWarps * kOwnKeys) {
    float k[kOwnKeys][kPL], v[kOwnKeys][kPL];
#pragma unroll
    for (int i = 0; i < kOwnKeys; ++i) {
      const int64_t at = head + static_cast<int64_t>(min(t + i, kb - 1)) * kHd;
      load_row<kPL>(p.kc + at, lane, k[i]);
      load_row<kPL>(p.vc + at, lane, v[i]);
    }
#pragma unroll
    for (int h = 0; h < kG; ++h) {
      float s[kOwnKeys], mn = m[h];
#pragma unroll
      for (int i = 0; i < kOwnKeys; ++i) {
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < kPL; ++j) d = fmaf(q[h][j], k[i][j], d);
        s[i] = t + i < kb ? soft_cap(warp_sum(d) * p.scale, p.cap) * kLog2e : -INFINITY;
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
          if (t + i < kb) a = fmaf(pr[i], v[i][j], a);
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
    float* dst =
        p.own + ((static_cast<int64_t>(blockIdx.x) * p.n_kv + g) * kG + h) * (kHd + kPartPad);
    dst[c] = a;
    if (c == 0) {
      dst[kHd] = M;
      dst[kHd + 1] = L;
    }
  }
}

// One warp per (sequence, query head): the prefix pieces, then the own ones.
template <int kPL>
__global__ void __launch_bounds__(128)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p) {
  constexpr int kHd = kPL * 32;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int b = w / p.n_q, h = w - b * p.n_q, g = h / p.group;
  if (b >= p.batch) return;
  const int row = b * p.group + (h - g * p.group);
  float m = -INFINITY, l = 0.f, acc[kPL];
#pragma unroll
  for (int j = 0; j < kPL; ++j) acc[j] = 0.f;
  auto join = [&](const float* src) {
    float x[kPL];
    load_row<kPL>(src, lane, x);
    const float mc = src[kHd], lc = src[kHd + 1];
    const float mn = fmaxf(m, mc);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float a = exp2f(m - base), c = exp2f(mc - base);
    l = fmaf(l, a, lc * c);
#pragma unroll
    for (int j = 0; j < kPL; ++j) acc[j] = fmaf(acc[j], a, x[j] * c);
    m = mn;
  };
  for (int c = 0; c < p.pieces; ++c) join(p.part + prefix_part<kPL>(p, c, g, row));
  for (int c = p.first[b]; c < p.first[b + 1]; ++c)
    join(p.own + ((static_cast<int64_t>(c) * p.n_kv + g) * p.group + (h - g * p.group)) *
                     (kHd + kPartPad));
  store_final<kPL>(p.out.data + static_cast<int64_t>(p.b0 + b) * p.out.token_stride +
                       h * p.out.head_stride,
                   lane, acc, l);
}

// ------------------------------------------------------------ host side
namespace {

constexpr int kPrefixR = 4;
constexpr int kPrefixRows = kRowWarps * kPrefixR;

struct PrefixPlan {
  int chunk, pieces;
  size_t part_floats, own_floats;    // of the largest launch
};

PrefixPlan plan_prefix(int64_t n_prefix, const int64_t* n_ctx, int batch, int n_q, int n_kv,
                       int head_dim) {
  PrefixPlan pl;
  const int group = n_q / n_kv, some = std::min(batch, kMaxBatch);
  const int64_t tiles = (static_cast<int64_t>(some) * group + kPrefixRows - 1) / kPrefixRows;
  // about two items an SM
  const int64_t want = std::max<int64_t>(1, 304 / (tiles * n_kv));
  int64_t chunk = (n_prefix + want - 1) / want;
  chunk = std::max<int64_t>(64, (chunk + 31) / 32 * 32);
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
cudaError_t run_prefix(const PrefixParams& p, cudaStream_t st) {
  using Tile = RowTile<kPL, kPrefixR>;
  cudaError_t e = cudaSuccess;
  const unsigned nkv = static_cast<unsigned>(p.n_kv);
  if (p.pieces > 0) {
    e = cudaFuncSetAttribute(prefix_rows_kernel<kPL, kPrefixR>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(Tile::kSmem));
    if (e != cudaSuccess) return e;
    e = pdl_launch(prefix_rows_kernel<kPL, kPrefixR>,
                   dim3(static_cast<unsigned>(p.pieces * p.row_tiles), nkv), kRowThreads,
                   Tile::kSmem, st, p);
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
  const int rows = p.batch * p.n_q;
  return pdl_launch(prefix_merge_kernel<kPL>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128,
                    0, st, p);
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
  p.scale = scale; p.cap = cap;
  for (int b0 = 0; b0 < batch; b0 += kMaxBatch) {
    p.b0 = b0;
    p.batch = std::min(batch - b0, kMaxBatch);
    p.row_tiles = (p.batch * p.group + kPrefixRows - 1) / kPrefixRows;
    p.first[0] = 0;
    for (int b = 0; b < p.batch; ++b) {
      p.n_ctx[b] = static_cast<int>(n_ctx[b0 + b]);
      p.first[b + 1] = p.first[b] + (p.n_ctx[b] + kOwnChunk - 1) / kOwnChunk;
    }
    cudaError_t e = cudaErrorInvalidValue;
    switch (head_dim) {
      case 32: e = run_prefix<1>(p, st); break;
      case 64: e = run_prefix<2>(p, st); break;
      case 128: e = run_prefix<4>(p, st); break;
      case 256: e = run_prefix<8>(p, st); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qws
