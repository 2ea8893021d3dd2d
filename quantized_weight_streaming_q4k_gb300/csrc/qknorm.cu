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
// head (in turns) reduces, rotates and stores.
//
// The angle: FP64 arithmetic is slow on this GPU, and f32 loses the angle of
// a far position.  The rotation per position in turns, f_i / 2 pi, is rounded
// on the host to a 64-bit fixed-point fraction F_i (error 2^-53 relative);
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

constexpr int kQkWarps = 8;
constexpr int kQkRounds = 2;   // rows of a warp whose loads are in flight together

template <int kPL>
__global__ void __launch_bounds__(kQkWarps * 32)
    qk_norm_rope_kernel(const __grid_constant__ QkParams p) {
  constexpr int kHd = kPL * 32;
  constexpr int kV = kPL < 4 ? kPL : 4;
  __shared__ __align__(16) float cs[kQkMaxHalf], sn[kQkMaxHalf];
  __shared__ __align__(16) float row[kQkWarps][kHd];   // a head, for the partner of each element
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rot / 2, heads = p.n_q + p.n_kv;
  float x[kQkRounds][kPL];
  auto fetch = [&](int h, float (&v)[kPL]) {
    const bool isq = h < p.n_q;
    const qws_heads& in = isq ? p.q : p.k;
    load_row<kPL>(in.data + t * in.token_stride + (isq ? h : h - p.n_q) * in.head_stride, lane,
                  v);
  };
  // the rows first, then the angles, whose position is another trip to memory
#pragma unroll
  for (int r = 0; r < kQkRounds; ++r)
    if (warp + r * kQkWarps < heads) fetch(warp + r * kQkWarps, x[r]);
  const uint64_t pos = static_cast<uint64_t>(__ldg(p.positions + t));
  for (int i = threadIdx.x; i < half; i += kQkWarps * 32)
    turn_cos_sin(pos * p.turn[i], cs[i], sn[i]);
  __syncthreads();
  auto finish = [&](int h, float (&v)[kPL]) {
    const bool isq = h < p.n_q;
    const float* w = isq ? p.w_q : p.w_k;
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kPL; ++j) ss = fmaf(v[j], v[j], ss);
      ss = warp_sum(ss);
      const float r = 1.0f / sqrtf(ss * (1.0f / kHd) + p.eps);
      float wv[kPL];
#pragma unroll
      for (int j = 0; j < kPL; ++j) wv[j] = __ldg(w + lane_col<kPL>(lane, j));
#pragma unroll
      for (int j = 0; j < kPL; ++j) v[j] = v[j] * r * wv[j];
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
    if (warp + r * kQkWarps < heads) finish(warp + r * kQkWarps, x[r]);
  for (int h = warp + kQkRounds * kQkWarps; h < heads; h += kQkWarps) {
    fetch(h, x[0]);
    finish(h, x[0]);
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
  switch (head_dim) {
    case 32: return pdl_launch(qk_norm_rope_kernel<1>, grid, kQkWarps * 32, 0, st, p);
    case 64: return pdl_launch(qk_norm_rope_kernel<2>, grid, kQkWarps * 32, 0, st, p);
    case 128: return pdl_launch(qk_norm_rope_kernel<4>, grid, kQkWarps * 32, 0, st, p);
    case 256: return pdl_launch(qk_norm_rope_kernel<8>, grid, kQkWarps * 32, 0, st, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qws
