// attend_rows.cuh -- attention of a tile of query rows over a range of keys in
// f32 on the CUDA cores, and the tables and partial results shared by the
// prompt and shared-prefix attention (prompt.cu, prefix.cu).
#pragma once

#include <cuda_runtime.h>

#include "launch.h"

namespace qws {

// Sequences of one launch: row (query token) and key offsets into the packed
// arrays, and the first work item of each.  Passed as a kernel argument, so a
// captured launch holds its own copy; longer lists take several launches.
constexpr int kMaxSeqs = 128;
struct SeqTab {
  int n;
  int q0[kMaxSeqs + 1];     // first query token of sequence s
  int k0[kMaxSeqs + 1];     // first key of sequence s
  int item[kMaxSeqs + 1];   // first work item of the sequence order[i]
  int order[kMaxSeqs];      // sequences, those with the most keys first
  int first[kMaxSeqs];      // first work item of sequence s
  int ktile[kMaxSeqs + 1];  // first 64-key tile of sequence s
};

// the sequence s with item[s] <= i < item[s + 1] (empty ones are skipped)
__device__ __forceinline__ int find_seq(const int* first, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Column of value j of a lane's share of a row of 32 * kPL values, in groups
// of up to four neighbours.
template <int kPL>
__device__ __forceinline__ int lane_col(int lane, int j) {
  if constexpr (kPL >= 4) return (j / 4) * 128 + lane * 4 + j % 4;
  else return lane * kPL + j;
}

template <int kPL>
__device__ __forceinline__ void load_row(const float* p, int lane, float (&x)[kPL]) {
  if constexpr (kPL >= 4) {
#pragma unroll
    for (int g = 0; g < kPL / 4; ++g) {
      const float4 v = *reinterpret_cast<const float4*>(p + g * 128 + lane * 4);
      x[4 * g] = v.x; x[4 * g + 1] = v.y; x[4 * g + 2] = v.z; x[4 * g + 3] = v.w;
    }
  } else if constexpr (kPL == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p + lane * 2);
    x[0] = v.x; x[1] = v.y;
  } else {
    x[0] = p[lane];
  }
}

template <int kPL>
__device__ __forceinline__ void store_row(float* p, int lane, const float (&x)[kPL]) {
  if constexpr (kPL >= 4) {
#pragma unroll
    for (int g = 0; g < kPL / 4; ++g)
      *reinterpret_cast<float4*>(p + g * 128 + lane * 4) =
          make_float4(x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]);
  } else if constexpr (kPL == 2) {
    *reinterpret_cast<float2*>(p + lane * 2) = make_float2(x[0], x[1]);
  } else {
    p[lane] = x[0];
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Scores are kept in units of log 2 (times log2 e), so that weights are powers of
// two of differences; running maxima of partial results too.
constexpr float kLog2e = 1.4426950408889634f;

// tanh(y) is y to less than half a step where |y| < 2^-13; y itself may be subnormal there
__device__ __forceinline__ float soft_cap(float s, float cap) {
  if (!(cap > 0.f)) return s;
  const float y = s / cap;
  return fabsf(y) < 0x1p-13f ? s : cap * tanhf(y);
}

// A CTA of kRowWarps warps, kR query rows a warp.  Keys come in tiles of 32
// through shared memory: a lane scores one key against the warp's rows (K row
// and q by 16-byte loads, K rows padded by 16 bytes against bank conflicts),
// the online softmax runs across the lanes, and for p * V a lane holds its
// columns of the output.  Scores, statistics and output are f32.
constexpr int kRowWarps = 8;
constexpr int kRowThreads = kRowWarps * 32;

template <int kPL, int kR>
struct RowTile {
  static constexpr int kHd = kPL * 32;
  static constexpr int kPitch = kHd + 4;
  static constexpr size_t kSmem =
      sizeof(float) * (2 * 32 * kPitch + static_cast<size_t>(kRowWarps) * kR * kHd);
  float m[kR], l[kR], acc[kR][kPL];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int j = 0; j < kPL; ++j) acc[r][j] = 0.f;
    }
  }

  // this warp's q rows in shared memory
  __device__ __forceinline__ static float* q_rows(float* smem) {
    return smem + 2 * 32 * kPitch + (threadIdx.x >> 5) * kR * kHd;
  }

  // keys [ka, kb) (relative to K and V); row r sees the keys below vis[r]
  __device__ __forceinline__ void run(float* smem, const float* K, const float* V,
                                      int64_t k_stride, int64_t v_stride, int ka, int kb,
                                      const int (&vis)[kR], float scale, float cap) {
    float* ks = smem;
    float* vs = smem + 32 * kPitch;
    const float* qs = q_rows(smem);
    const int lane = threadIdx.x & 31;
    int least = vis[0];
#pragma unroll
    for (int r = 1; r < kR; ++r) least = min(least, vis[r]);
    for (int t = ka; t < kb; t += 32) {
      const int n = min(32, kb - t);
      __syncthreads();
      for (int e = threadIdx.x; e < 32 * (kHd / 4); e += kRowThreads) {
        const int row = e / (kHd / 4), c = (e - row * (kHd / 4)) * 4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (row < n) {
          a = *reinterpret_cast<const float4*>(K + (t + row) * k_stride + c);
          b = *reinterpret_cast<const float4*>(V + (t + row) * v_stride + c);
        }
        *reinterpret_cast<float4*>(ks + row * kPitch + c) = a;
        *reinterpret_cast<float4*>(vs + row * kPitch + c) = b;
      }
      __syncthreads();
      float s[kR][2];
#pragma unroll
      for (int r = 0; r < kR; ++r) s[r][0] = s[r][1] = 0.f;
#pragma unroll 4
      for (int c = 0; c < kHd; c += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(ks + lane * kPitch + c);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float4 q4 = *reinterpret_cast<const float4*>(qs + r * kHd + c);
          s[r][0] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, s[r][0]));
          s[r][1] = fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[r][1]));
        }
      }
      float p[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float x = soft_cap((s[r][0] + s[r][1]) * scale, cap) * kLog2e;
        if (t + lane >= vis[r]) x = -INFINITY;      // select: what is masked is not looked at
        const float mn = fmaxf(m[r], warp_max(x));
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m[r] - base);
        p[r] = exp2f(x - base);
        l[r] = fmaf(l[r], alpha, warp_sum(p[r]));
        m[r] = mn;
#pragma unroll
        for (int j = 0; j < kPL; ++j) acc[r][j] *= alpha;
      }
      const bool whole = t + n <= least;     // every row sees every key of the tile
      for (int k = 0; k < n; ++k) {
        float v[kPL];
        load_row<kPL>(vs + k * kPitch, lane, v);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float pk = __shfl_sync(0xFFFFFFFFu, p[r], k);
          // 0 * v of a masked key would let an infinity or NaN there through
          if (whole || t + k < vis[r]) {
#pragma unroll
            for (int j = 0; j < kPL; ++j) acc[r][j] = fmaf(pk, v[j], acc[r][j]);
          }
        }
      }
    }
  }
};

// One row's partial result: unnormalised output, then running max and sum.
// Partials are [slot][row of the tile][head_dim + kPartPad].
constexpr int kPartPad = 4;   // m, l, two unused: keeps rows 16-byte aligned

template <int kPL>
__device__ __forceinline__ void store_partial(float* dst, int lane, const float (&acc)[kPL],
                                              float m, float l) {
  store_row<kPL>(dst, lane, acc);
  if (lane == 0) {
    dst[32 * kPL] = m;
    dst[32 * kPL + 1] = l;
  }
}

// Joins the partial results from .. n - 1 of a row in order, by one warp, for its columns, kV
// neighbours a lane from column col on.  part(c) is piece c's row, called by the whole
// warp with one c; mine(c) the same, called by some lanes, lane i with c = from + i modulo 32
// (so neither may exchange values between lanes there).  The columns of a
// batch of pieces are fetched together with, not after, the maxima that weigh them: one
// trip to memory and not three.  Returns the row's sum, and its maximum in M.
template <int kHd, int kV, class Mine, class Part>
__device__ __forceinline__ float join_parts(int from, int n, int lane, int col, Mine&& mine,
                                            Part&& part, float (&acc)[kV], float& M) {
  constexpr int kBatch = 32 / kV;
  float L = 0.f;
  M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
  for (int c0 = from; c0 < n; c0 += 32) {
    const int m = min(32, n - c0);
    float mc = -INFINITY, lc = 0.f;
    if (lane < m) {
      const float2 ml = *reinterpret_cast<const float2*>(mine(c0 + lane) + kHd);
      mc = ml.x;
      lc = ml.y;
    }
    for (int b0 = 0; b0 < m; b0 += kBatch) {
      float v[kBatch][kV];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[c][i] = 0.f;
        if (b0 + c < m) {
          const float* p = part(c0 + b0 + c) + col;
          if constexpr (kV == 4) {
            const float4 q = *reinterpret_cast<const float4*>(p);
            v[c][0] = q.x; v[c][1] = q.y; v[c][2] = q.z; v[c][3] = q.w;
          } else if constexpr (kV == 2) {
            const float2 q = *reinterpret_cast<const float2*>(p);
            v[c][0] = q.x; v[c][1] = q.y;
          } else {
            v[c][0] = p[0];
          }
        }
      }
      if (b0 == 0) {
        // this group's maximum joins the running one
        const float Mn = fmaxf(M, warp_max(mc));
        const float base = Mn == -INFINITY ? 0.f : Mn;
        const float old = exp2f(M - base);
        lc *= mc = exp2f(mc - base);                  // mc: from here on the weight
        L = fmaf(L, old, warp_sum(lc));
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[i] *= old;
        M = Mn;
      }
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const float f = __shfl_sync(0xFFFFFFFFu, mc, (b0 + c) & 31);
        if (b0 + c < m) {
#pragma unroll
          for (int i = 0; i < kV; ++i) acc[i] = fmaf(v[c][i], f, acc[i]);
        }
      }
    }
  }
  return L;
}

// out = acc / l; a row that saw no key is zero
template <int kPL>
__device__ __forceinline__ void store_final(float* dst, int lane, float (&acc)[kPL], float l) {
  const float r = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < kPL; ++j) acc[j] *= r;
  store_row<kPL>(dst, lane, acc);
}

}  // namespace qws
