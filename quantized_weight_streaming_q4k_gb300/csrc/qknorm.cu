// qknorm.cu -- the norm of every query and key head and the rotation at the
// token's position, for many tokens in one pass (the prompt's form of
// rope_at_pos, with the per-head RMS norm that some models put before it):
//   y = x / sqrt(mean_i x_i^2 + eps) * w        (when w is given)
//   (y_i, y_{i+r/2}) <- (y_i cos - y_{i+r/2} sin, y_i sin + y_{i+r/2} cos),
//   angle pos * base^(-2i/r), i < r/2.
//
// Bound by memory: every head is read once and written once.  One CTA per
// token: its threads compute the token's r/2 sines and cosines once into
// shared memory while the warps' head rows are in flight, then one warp per
// head (in turns) reduces, rotates and stores.  4096 tokens, 8 + 4 heads of 256: 17.5 us,
// 5.8 TB/s (100.7 MB at the copy rate: 14.9 us).  With 8 warps x 2 rows 21.0 us: 12 heads
// leave half of those warps with one row.  With the head's partners through shared memory
// too (the form for rot_dim < head_dim) 22.7 us, its pipe 73 % busy.
//
// The angle: FP64 arithmetic is slow on this GPU, and f32 loses the angle of
// a far position.  The rotation per position in turns, f_i / 2 pi, is rounded
// on the host to a 64-bit fixed-point fraction F_i.  In radians it is off by at most
// 6 x 2^-53: two powers, 2 pi, a division and a product, each 2^-53 of f_i <= 1, and the
// rounded exponent x of base^-x, x ln(base) base^-x <= 1 / e of that.
// pos * F_i modulo 2^64 by one integer product IS the fraction of a turn, exact
// for any position.  Its top two bits (rounded) are the quadrant, the rest,
// at most 1/8 turn either way, is rounded once to f32 for sinpi / cospi: an
// angle error below 2^-24 * pi / 4.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "attend_rows.cuh"
#include "launch.h"

namespace qws {

constexpr int kQkMaxHalf = 128;   // rot_dim <= head_dim <= 256

struct QkParams {
  qws_heads q, k, qo, ko;
  const float *w_q, *w_k;
  const int64_t* positions;
  int n_q, n_kv, rot;
  float eps;
  uint64_t turn[kQkMaxHalf];   // rotation per position, in 2^-64 turns
};

// cos and sin of the angle F * 2^-64 turns
__device__ __forceinline__ void turn_cos_sin(uint64_t F, float& c, float& s) {
  const uint64_t quad = (F + (uint64_t(1) << 61)) >> 62;
  const int64_t rem = static_cast<int64_t>(F - (quad << 62));      // [-2^61, 2^61)
  float s0, c0;
  sincospif(static_cast<float>(rem) * 0x1p-63f, &s0, &c0);         // half turns
  const int qd = static_cast<int>(quad & 3);
  const float a = (qd & 1) ? s0 : c0, b = (qd & 1) ? c0 : s0;
  c = (qd == 1 || qd == 2) ? -a : a;
  s = qd >= 2 ? -b : b;
}

// kV neighbouring values from shared memory
template <int kV>
__device__ __forceinline__ void read_group(const float* p, float (&v)[kV]) {
  if constexpr (kV == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else if constexpr (kV == 2) {
    const float2 q = *reinterpret_cast<const float2*>(p);
    v[0] = q.x; v[1] = q.y;
  } else {
    v[0] = p[0];
  }
}

constexpr int kQkWarps = 4;
constexpr int kQkRounds = 3;   // rows of a warp whose loads are in flight together

// kFull: rot_dim = head_dim.  Then the partner of an element is in the same lane (head_dim
// 256) or 16 lanes away, and a lane has the same angles in every head, so nothing but the
// angles goes through shared memory.
template <int kPL, bool kFull>
__global__ void __launch_bounds__(kQkWarps * 32)
    qk_norm_rope_kernel(const __grid_constant__ QkParams p) {
  constexpr int kHd = kPL * 32;
  constexpr int kV = kPL < 4 ? kPL : 4;
  __shared__ __align__(16) float cs[kQkMaxHalf], sn[kQkMaxHalf];
  // a head, for the partner of each element
  __shared__ __align__(16) float row[kFull ? 1 : kQkWarps][kFull ? 4 : kHd];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rot / 2, heads = p.n_q + p.n_kv;
  float x[kQkRounds][kPL], wv[kQkRounds][kPL];
  auto fetch = [&](int h, float (&v)[kPL], float (&wv)[kPL]) {
    const bool isq = h < p.n_q;
    const qws_heads& in = isq ? p.q : p.k;
    const float* w = isq ? p.w_q : p.w_k;
#pragma unroll
    for (int j = 0; j < kPL; ++j) wv[j] = w ? __ldg(w + lane_col<kPL>(lane, j)) : 1.f;
    load_row<kPL>(in.data + t * in.token_stride + (isq ? h : h - p.n_q) * in.head_stride, lane,
                  v);
  };
  // the rows first, then the angles, whose position is another trip to memory
#pragma unroll
  for (int r = 0; r < kQkRounds; ++r)
    if (warp + r * kQkWarps < heads) fetch(warp + r * kQkWarps, x[r], wv[r]);
  const uint64_t pos = static_cast<uint64_t>(__ldg(p.positions + t));
  for (int i = threadIdx.x; i < half; i += kQkWarps * 32)
    turn_cos_sin(pos * p.turn[i], cs[i], sn[i]);
  __syncthreads();
  float c[kV], s[kV];
  if constexpr (kFull) {
    const int k = (kPL == 8 ? lane : lane & 15) * kV;
    read_group<kV>(cs + k, c);
    read_group<kV>(sn + k, s);
  }
  auto finish = [&](int h, float (&v)[kPL], const float (&wv)[kPL]) {
    const bool isq = h < p.n_q;
    if (isq ? p.w_q : p.w_k) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kPL; ++j) ss = fmaf(v[j], v[j], ss);
      ss = warp_sum(ss);
      const float r = 1.0f / sqrtf(ss * (1.0f / kHd) + p.eps);
#pragma unroll
      for (int j = 0; j < kPL; ++j) v[j] = v[j] * r * wv[j];
    }
    if constexpr (kFull) {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if constexpr (kPL == 8) {
          const float a = v[j], b = v[j + 4];
          v[j] = fmaf(a, c[j], -(b * s[j]));
          v[j + 4] = fmaf(b, c[j], a * s[j]);
        } else {
          const float o = __shfl_xor_sync(0xFFFFFFFFu, v[j], 16);
          v[j] = fmaf(v[j], c[j], lane < 16 ? -(o * s[j]) : o * s[j]);
        }
      }
      const qws_heads& out = isq ? p.qo : p.ko;
      store_row<kPL>(out.data + t * out.token_stride + (isq ? h : h - p.n_q) * out.head_stride,
                     lane, v);
      return;
    }
    __syncwarp();
    store_row<kPL>(row[warp], lane, v);
    __syncwarp();
    if (half % kV == 0) {
      // a lane's neighbours are on one side of every border: vector reads
#pragma unroll
      for (int g = 0; g < kPL; g += kV) {
        const int i = lane_col<kPL>(lane, g);
        if (i >= p.rot) continue;
        const bool first = i < half;
        const int k = first ? i : i - half;
        float c[kV], s[kV], o[kV];
        read_group<kV>(cs + k, c);
        read_group<kV>(sn + k, s);
        read_group<kV>(row[warp] + (first ? i + half : k), o);
#pragma unroll
        for (int j = 0; j < kV; ++j)
          v[g + j] = fmaf(v[g + j], c[j], first ? -(o[j] * s[j]) : o[j] * s[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPL; ++j) {
        const int i = lane_col<kPL>(lane, j);
        if (i < half)
          v[j] = fmaf(v[j], cs[i], -(row[warp][i + half] * sn[i]));
        else if (i < p.rot)
          v[j] = fmaf(v[j], cs[i - half], row[warp][i - half] * sn[i - half]);
      }
    }
    const qws_heads& out = isq ? p.qo : p.ko;
    store_row<kPL>(out.data + t * out.token_stride + (isq ? h : h - p.n_q) * out.head_stride,
                   lane, v);
  };
#pragma unroll
  for (int r = 0; r < kQkRounds; ++r)
    if (warp + r * kQkWarps < heads) finish(warp + r * kQkWarps, x[r], wv[r]);
  for (int h = warp + kQkRounds * kQkWarps; h < heads; h += kQkWarps) {
    fetch(h, x[0], wv[0]);
    finish(h, x[0], wv[0]);
  }
}

cudaError_t launch_qk_norm_rope(const qws_heads& q, const qws_heads& k, const qws_heads& qo,
                                const qws_heads& ko, const float* w_q, const float* w_k,
                                const int64_t* positions, int64_t n_tokens, int n_q, int n_kv,
                                int head_dim, int rot_dim, double base, float eps,
                                cudaStream_t st) {
  QkParams p;
  p.q = q; p.k = k; p.qo = qo; p.ko = ko;
  p.w_q = w_q; p.w_k = w_k;
  p.positions = positions;
  p.n_q = n_q; p.n_kv = n_kv; p.rot = rot_dim;
  p.eps = eps;
  // base^(-2i/r) as base^(-2 (i - i % 16) / r) * base^(-2 (i % 16) / r): 24 powers in place
  // of 128, one rounding more; base >= 1: at most 1 / 2 pi of a turn per position
  double low[16];
  for (int i = 0; i < 16; ++i) low[i] = std::pow(base, -2.0 * i / rot_dim);
  for (int i = 0; i < rot_dim / 2; i += 16) {
    const double high = std::pow(base, -2.0 * i / rot_dim) / 6.283185307179586477;
    for (int j = 0; j < 16 && i + j < rot_dim / 2; ++j)
      p.turn[i + j] = static_cast<uint64_t>(std::ldexp(high * low[j], 64));
  }
  for (int i = rot_dim / 2; i < kQkMaxHalf; ++i) p.turn[i] = 0;
  const dim3 grid(static_cast<unsigned>(n_tokens));
  const auto go = [&](auto* part, auto* full) {
    return pdl_launch(rot_dim == head_dim ? full : part, grid, kQkWarps * 32, 0, st, p);
  };
  switch (head_dim) {
    case 32: return go(qk_norm_rope_kernel<1, false>, qk_norm_rope_kernel<1, true>);
    case 64: return go(qk_norm_rope_kernel<2, false>, qk_norm_rope_kernel<2, true>);
    case 128: return go(qk_norm_rope_kernel<4, false>, qk_norm_rope_kernel<4, true>);
    case 256: return go(qk_norm_rope_kernel<8, false>, qk_norm_rope_kernel<8, true>);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qws
