// paged_rows.cu -- rows of keys and values into a paged 4- or 8-bit cache, and back as f32.
//
// Append.  For every token, every query and key head x: y = x / sqrt(mean x^2 + eps) * w when
// w is given, rotated at the token's position (half split, as in qk_norm_rope), rounded once
// to f32; queries are stored as they are, keys and values by blocks of 32: the scale d
// (Q4_0: the value of the largest magnitude / -8, the first one of equals; Q8_0: the largest
// magnitude times the f32 nearest 1 / 127), the codes from the f32 d, d as f16.
//
// A code is a decision: an y that is off by one f32 step now and then moves a code by one, a
// sixteenth of its block's range, and which token did would depend on the arithmetic.  So the
// norm and rotation of keys are carried in pairs of f32 (value and remainder, products by fma, sums by the
// exact error of an addition), to about 2^-44, and rounded once: the f32 that a 64-bit
// computation rounds to, but for some 2^-20 of the values.  FP64 itself runs at 1/64 of the f32
// rate here.
//
// Bound by instructions: 4 bytes read a value, 4 (queries) or 18/32 (keys, values) written, but
// some 440 instructions a row of 256 on average, a key row twice that.  One CTA a token,
// as in qk_norm_rope: its threads compute the token's sines and cosines once into shared memory
// while the warps' first rows are in flight; then a warp a head, one copy of the code for all.
// 4096 tokens of 8 + 4 + 4 heads of 256, Q4_0, take 33.1 us (105 MB: 3.2 TB/s).  Before: 60 with
// queries in pairs too, 50 with the rows' code four times over, 44 with the angles in order, which
// a warp reads with four conflicts each.  More rows in flight per warp: 47 to 51.
#include <cuda_runtime.h>

#include <cmath>

#include "attend_rows.cuh"
#include "paged.cuh"

namespace qws {

__device__ unsigned g_err_paged;

// ------------------------------------------------------------ pairs of f32
struct Pair {
  float h, l;
};

__device__ __forceinline__ Pair two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
// |a| >= |b| or so
__device__ __forceinline__ Pair quick_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  return quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const Pair p = two_prod(a.h, b.h);
  return quick_sum(p.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, p.l)));
}
__device__ __forceinline__ Pair mul(Pair a, float b) {
  const Pair p = two_prod(a.h, b);
  return quick_sum(p.h, __fmaf_rn(a.l, b, p.l));
}

// v^(-1/2): one Newton step with the third-order term on the f32 root's reciprocal
__device__ __forceinline__ Pair rsqrt_pair(Pair v) {
  const float r = 1.0f / sqrtf(v.h);
  const Pair rr = two_prod(r, r);
  const Pair q = two_prod(v.h, rr.h);
  const float rest = __fadd_rn(q.l, __fmaf_rn(v.h, rr.l, __fmul_rn(v.l, rr.h)));
  const float e = __fsub_rn(__fsub_rn(1.0f, q.h), rest);      // 1 - v r^2, some 2^-22
  return quick_sum(r, __fmul_rn(r, __fmaf_rn(__fmul_rn(0.375f, e), e, __fmul_rn(0.5f, e))));
}

// ------------------------------------------------------------ sines and cosines
// cos and sin of k / 256 turns, k < 64, as pairs: (cos.h, cos.l, sin.h, sin.l), by their
// power series in double at compile time.
struct TurnTable {
  float v[64][4];
};
constexpr double series_sin(double x) {
  double t = x, s = x;
  for (int k = 1; k < 16; ++k) {
    t *= -x * x / ((2 * k) * (2 * k + 1));
    s += t;
  }
  return s;
}
constexpr double series_cos(double x) {
  double t = 1, s = 1;
  for (int k = 1; k < 16; ++k) {
    t *= -x * x / ((2 * k - 1) * (2 * k));
    s += t;
  }
  return s;
}
constexpr TurnTable make_turn_table() {
  constexpr double kStep = 6.283185307179586477 / 256;
  TurnTable t{};
  for (int k = 0; k < 64; ++k) {
    // the other function of the complement beyond an eighth of a turn: short series
    const double c = k <= 32 ? series_cos(k * kStep) : series_sin((64 - k) * kStep);
    const double s = k <= 32 ? series_sin(k * kStep) : series_cos((64 - k) * kStep);
    t.v[k][0] = static_cast<float>(c);
    t.v[k][1] = static_cast<float>(c - static_cast<double>(t.v[k][0]));
    t.v[k][2] = static_cast<float>(s);
    t.v[k][3] = static_cast<float>(s - static_cast<double>(t.v[k][2]));
  }
  return t;
}
__device__ const TurnTable kTurns = make_turn_table();

// cos and sin of the angle F * 2^-64 turns (fixed point, as in qk_norm_rope).  The nearest of
// 256 points from the table, the rest, |x| < 0.0123, by series: x - x^3/6 + x^5/120 and
// 1 - x^2/2 + x^4/24 (the next terms are below 2^-51), joined by the sum of angles.
__device__ __forceinline__ void turn_cos_sin(uint64_t F, Pair& c, Pair& s) {
  const uint64_t idx = (F + (uint64_t(1) << 55)) >> 56;
  const int64_t rem = static_cast<int64_t>(F - (idx << 56));            // [-2^55, 2^55)
  // 25 bits and 24 bits, both exact in f32; 2 pi 2^-64 per unit
  const float rh = static_cast<float>(static_cast<int32_t>(rem >> 31)) * 0x1p-33f;
  const float rl = static_cast<float>(static_cast<int32_t>((rem & 0x7FFFFFFF) >> 7)) * 0x1p-57f;
  const Pair x = mul(quick_sum(rh, rl), Pair{6.2831854820251465f, -1.7484556e-7f});
  const Pair xx = mul(x, x);
  const float x3 = __fmul_rn(xx.h, x.h);
  // sin x = x + (-x^3 / 6 + x^5 / 120);  cos x - 1 = -x^2 / 2 + x^4 / 24
  const Pair sx = quick_sum(x.h, __fadd_rn(x.l, __fmul_rn(x3, __fmaf_rn(xx.h, 1.f / 120, -1.f / 6))));
  const Pair cm = quick_sum(-0.5f * xx.h,
                            __fmaf_rn(__fmul_rn(xx.h, xx.h), 1.f / 24, -0.5f * xx.l));
  const float4 t = *reinterpret_cast<const float4*>(kTurns.v[idx & 63]);
  const Pair C{t.x, t.y}, S{t.z, t.w};
  const Pair ms = mul(S, sx);
  const Pair c0 = add(C, add(mul(C, cm), Pair{-ms.h, -ms.l}));
  const Pair s0 = add(S, add(mul(S, cm), mul(C, sx)));
  const int quad = static_cast<int>(idx >> 6) & 3;
  const Pair a = (quad & 1) ? s0 : c0, b = (quad & 1) ? c0 : s0;
  const float sc = (quad == 1 || quad == 2) ? -1.f : 1.f, ss = quad >= 2 ? -1.f : 1.f;
  c = {a.h * sc, a.l * sc};
  s = {b.h * ss, b.l * ss};
}

// a lane's share of a norm's weights, which need not be 16-byte aligned
template <int kPL>
__device__ __forceinline__ void load_weights(const float* w, int lane, float (&x)[kPL]) {
  if (reinterpret_cast<uintptr_t>(w) % 16 == 0) {
    load_row<kPL>(w, lane, x);
  } else {
#pragma unroll
    for (int j = 0; j < kPL; ++j) x[j] = __ldg(w + lane_col<kPL>(lane, j));
  }
}

// ------------------------------------------------------------ append
constexpr int kApWarps = 4;
constexpr int kApMaxHalf = 128;    // rot_dim <= head_dim <= 256

// Heads whose mean square and eps together are below kSmall are taken kUp times as large, and eps
// kUp^2 times: their squares have remainders below f32's range then, and its reciprocal leaves it
// from 2^-128 on.  Above it nothing is lost (mean: from squares of 2^-90 on within 2^-59), below
// it |x| < 2^-41, so the squares of kUp x stay below 2^118, and those of subnormal x above 2^-98.
// What is left, a head of zeros, ends as zeros by the mean's lower limit.
constexpr float kSmall = 0x1p-90f, kUp = 0x1p100f, kLeast = 0x1p-125f;

struct AppendParams {
  PagedView c;
  qws_heads q, k, v, qo;
  const float *w_q, *w_k;
  const int64_t *seqs, *positions;
  int n_q, rot;                    // n_q 0: no queries; rot 0: no rotation
  Pair eps, eps_up;                // eps; the same times kUp^2
  uint64_t turn[kApMaxHalf];       // rotation per position, in 2^-64 turns
};

// One row of keys or values into its place: blocks of 32 / kV lanes.
template <int kPL, int kFmt>
__device__ __forceinline__ void store_codes(uint8_t* slab, int p, bool keys, uint8_t* buf,
                                            int lane, const float (&x)[kPL]) {
  using L = Slab<kPL * 32, kFmt>;
  constexpr int kV = kPL < 4 ? kPL : 4;
  constexpr int kLanes = 32 / kV;          // of a block
  const int first = lane / kLanes * kLanes;
  const uint32_t group = (kLanes == 32 ? 0xFFFFFFFFu : ((1u << (kLanes & 31)) - 1u)) << first;
#pragma unroll
  for (int g = 0; g < kPL / kV; ++g) {
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j) amax = fmaxf(amax, fabsf(x[g * kV + j]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    float d;
    if constexpr (kFmt == QWS_Q4_0) {
      // the sign of the first value of that magnitude
      uint32_t hit = 0;
      bool neg = false;
#pragma unroll
      for (int j = kV - 1; j >= 0; --j) {
        const bool here = fabsf(x[g * kV + j]) == amax;
        hit |= here;
        if (here) neg = signbit(x[g * kV + j]);
      }
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, hit != 0) & group;
      const uint32_t sign = __ballot_sync(0xFFFFFFFFu, neg);
      const int f = __ffs(static_cast<int>(who)) - 1;          // -1: the block holds a NaN alone
      d = (f >= 0 && (sign >> f & 1u) ? amax : -amax) * 0.125f;
    } else {
      d = amax * (1.0f / 127.0f);
    }
    const float inv = d != 0.f ? 1.0f / d : 0.f;
    uint32_t code[4] = {};                     // in the last byte
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      // rounded as the last bits of a number from 2^23 on; what is not a number (of a scale so
      // small that its reciprocal is infinite) counts as 0, and -127
      const float z = __fmul_rn(x[g * kV + j], inv);
      if constexpr (kFmt == QWS_Q4_0) {
        const float t = fminf(fmaxf(__fadd_rn(z, 8.5f), 0.f), 15.5f);
        code[j] = __float_as_uint(__fadd_rz(t, 8388608.f));
      } else {
        // halves away from zero: 0.49999997 is the number before a half
        const float t = fminf(fmaxf(z, -127.f), 127.f);
        const float r = __fadd_rz(__fadd_rn(fabsf(t), 0.49999997f), 8388608.f) - 8388608.f;
        code[j] = __float_as_uint(copysignf(r, t) + (8388608.f + 128.f));
      }
    }
    const uint32_t word = __byte_perm(__byte_perm(code[0], code[1], 0x0040),
                                      __byte_perm(code[2], code[3], 0x0040), 0x5410);
    uint8_t* to = buf + lane_col<kPL>(lane, g * kV);
    if constexpr (kV == 4) *reinterpret_cast<uint32_t*>(to) = word;
    else if constexpr (kV == 2) *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(word);
    else *to = static_cast<uint8_t>(word);
    if (lane == first) {
      const int b = (kPL == 8 ? g * 4 : 0) + lane / kLanes;
      *reinterpret_cast<__half*>(slab + (keys ? L::kKScale : L::kVScale) +
                                 2 * (p * L::kBlocks + b)) = __float2half_rn(d);
    }
  }
  __syncwarp();
  // eight codes a step: a word (Q4_0) or two
  if (lane < kPL * 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(buf + 8 * lane);
    uint32_t a = w.x, b = w.y;
    if constexpr (kFmt == QWS_Q4_0) {        // four codes in two bytes each
      a = (a | a >> 4) & 0x00FF00FFu;
      a = (a | a >> 8) & 0xFFFFu;
      b = (b | b >> 4) & 0x00FF00FFu;
      b = (b | b >> 8) & 0xFFFFu;
    }
    if (keys) {
      uint8_t* to = slab + L::key8(p, lane);
      if constexpr (kFmt == QWS_Q4_0) *reinterpret_cast<uint32_t*>(to) = a | b << 16;
      else *reinterpret_cast<uint2*>(to) = make_uint2(a, b);
    } else {
#pragma unroll
      for (int h = 0; h < 2 / L::kPer; ++h) {
        *reinterpret_cast<uint16_t*>(slab + L::value4(p, 2 * lane, h)) =
            static_cast<uint16_t>(a >> (16 * h));
        *reinterpret_cast<uint16_t*>(slab + L::value4(p, 2 * lane + 1, h)) =
            static_cast<uint16_t>(b >> (16 * h));
      }
    }
  }
  __syncwarp();
}

template <int kPL, int kFmt>
__global__ void __launch_bounds__(kApWarps * 32, 8)
    paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kHd = kPL * 32;
  constexpr int kV = kPL < 4 ? kPL : 4;
  // cos, sin of the token's angles, angle i at turn_at(i): a warp reads every kV-th one at a time
  __shared__ float4 turn[kHd / 2];
  const auto turn_at = [](int i) { return i % kV * (kHd / 2 / kV) + i / kV; };
  __shared__ Pair row[kApWarps][kHd];                  // a head, for partners (rot < head_dim)
  __shared__ __align__(8) uint8_t codes[kApWarps][kHd];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = p.rot / 2, n_kv = p.c.n_kv, rows = p.n_q + 2 * n_kv;
  float x[kPL];                                        // the next row
  const float* q_row = p.q.data + t * p.q.token_stride;
  const float* k_row = p.k.data + t * p.k.token_stride;
  const float* v_row = p.v.data + t * p.v.token_stride;
  auto source = [&](int r) -> const float* {
    if (r < p.n_q) return q_row + r * p.q.head_stride;
    r -= p.n_q;
    return r < n_kv ? k_row + r * p.k.head_stride : v_row + (r - n_kv) * p.v.head_stride;
  };
  // the first rows, then the angles, whose position is another trip to memory
  if (warp < rows) load_row<kPL>(source(warp), lane, x);
  const int64_t seq = __ldg(p.seqs + t), pos = __ldg(p.positions + t);
  const TokenKind kind = token_kind(p.c, seq, pos);
  uint8_t* slab = nullptr;                             // of kv head 0; nullptr: not stored
  if (kind == kTokenFine)
    slab = token_slab(p.c, seq, static_cast<uint32_t>(pos), Slab<kHd, kFmt>::kBytes);
  for (int i = threadIdx.x; i < half; i += kApWarps * 32) {
    Pair c, s;
    turn_cos_sin(static_cast<uint64_t>(pos) * p.turn[i], c, s);
    turn[turn_at(i)] = make_float4(c.h, c.l, s.h, s.l);
  }
  __syncthreads();
  // a query: nothing is decided by its last bit, so f32 as in qk_norm_rope
  auto finish_query = [&](int r, float (&v)[kPL]) {
    if (p.w_q) {
      float mean, w[kPL];
      load_weights<kPL>(p.w_q, lane, w);
#pragma unroll 1
      for (bool up = false;; up = true) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < kPL; ++j) ss = fmaf(v[j], v[j], ss);
        mean = warp_sum(ss) * (1.0f / kHd) + (up ? p.eps_up.h : p.eps.h);
        if (up) mean = fmaxf(mean, kLeast);
        if (up || !(mean < kSmall)) break;
#pragma unroll
        for (int j = 0; j < kPL; ++j) v[j] *= kUp;
      }
      const float rs = 1.0f / sqrtf(mean);
#pragma unroll
      for (int j = 0; j < kPL; ++j) v[j] = v[j] * rs * w[j];
    }
    const auto rotated = [&](float a, float b, float4 cs, bool first) {
      return fmaf(a, cs.x, first ? -(b * cs.z) : b * cs.z);
    };
    if (p.rot == kHd) {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if constexpr (kPL == 8) {
          const float4 cs = turn[turn_at(lane * 4 + j)];
          const float a = v[j], b = v[j + 4];
          v[j] = rotated(a, b, cs, true);
          v[j + 4] = rotated(b, a, cs, false);
        } else {
          const float o = __shfl_xor_sync(0xFFFFFFFFu, v[j], 16);
          v[j] = rotated(v[j], o, turn[turn_at((lane & 15) * kV + j)], lane < 16);
        }
      }
    } else if (p.rot) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kPL; ++j) row[warp][lane_col<kPL>(lane, j)].h = v[j];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kPL; ++j) {
        const int i = lane_col<kPL>(lane, j);
        if (i < half) v[j] = rotated(v[j], row[warp][i + half].h, turn[turn_at(i)], true);
        else if (i < p.rot) v[j] = rotated(v[j], row[warp][i - half].h, turn[turn_at(i - half)], false);
      }
    }
    store_row<kPL>(p.qo.data + t * p.qo.token_stride + r * p.qo.head_stride, lane, v);
  };
  auto finish = [&](int r, float (&v)[kPL]) {
    const bool isq = r < p.n_q, isk = !isq && r < p.n_q + n_kv;
    if (isq) {
      finish_query(r, v);
      return;
    }
    if (isk) {
      // pairs whose parts may overlap by a bit or two: what is rounded is their sum
      Pair y[kPL];
      if (p.w_k) {
        float w[kPL];
        load_weights<kPL>(p.w_k, lane, w);
        Pair mean;
#pragma unroll 1
        for (bool up = false;; up = true) {
          Pair ss{0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kPL; ++j) {
            const Pair q = two_prod(v[j], v[j]), t = two_sum(ss.h, q.h);
            ss = {t.h, __fadd_rn(ss.l, __fadd_rn(t.l, q.l))};
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            ss = add(ss, Pair{__shfl_xor_sync(0xFFFFFFFFu, ss.h, o),
                              __shfl_xor_sync(0xFFFFFFFFu, ss.l, o)});
          mean = add(Pair{ss.h * (1.0f / kHd), ss.l * (1.0f / kHd)}, up ? p.eps_up : p.eps);
          if (up) mean.h = fmaxf(mean.h, kLeast);
          if (up || !(mean.h < kSmall)) break;
#pragma unroll
          for (int j = 0; j < kPL; ++j) v[j] *= kUp;
        }
        const Pair rs = rsqrt_pair(mean);
#pragma unroll
        for (int j = 0; j < kPL; ++j) {
          const Pair x = two_prod(v[j], rs.h), z = two_prod(x.h, w[j]);
          y[j] = {z.h, __fmaf_rn(__fmaf_rn(v[j], rs.l, x.l), w[j], z.l)};
        }
      } else {
#pragma unroll
        for (int j = 0; j < kPL; ++j) y[j] = {v[j], -0.f};      // -0 + -0 is -0
      }
      // a is turned by the angle with its partner b: a cos -+ b sin
      const auto rotated = [&](Pair a, Pair b, float4 cs, bool first) {
        const float sh = first ? -cs.z : cs.z, sl = first ? -cs.w : cs.w;
        const Pair x = two_prod(a.h, cs.x), z = two_prod(b.h, sh), t = two_sum(x.h, z.h);
        float rest = __fadd_rn(x.l, z.l);
        rest = __fmaf_rn(a.h, cs.y, __fmaf_rn(a.l, cs.x, rest));
        rest = __fmaf_rn(b.h, sl, __fmaf_rn(b.l, sh, rest));
        return Pair{t.h, __fadd_rn(t.l, rest)};
      };
      if (p.rot == kHd) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          if constexpr (kPL == 8) {
            const float4 cs = turn[turn_at(lane * 4 + j)];
            const Pair a = y[j], b = y[j + 4];
            y[j] = rotated(a, b, cs, true);
            y[j + 4] = rotated(b, a, cs, false);
          } else {
            const Pair o{__shfl_xor_sync(0xFFFFFFFFu, y[j].h, 16),
                         __shfl_xor_sync(0xFFFFFFFFu, y[j].l, 16)};
            y[j] = rotated(y[j], o, turn[turn_at((lane & 15) * kV + j)], lane < 16);
          }
        }
      } else if (p.rot) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kPL; ++j) row[warp][lane_col<kPL>(lane, j)] = y[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kPL; ++j) {
          const int i = lane_col<kPL>(lane, j);
          if (i < half) y[j] = rotated(y[j], row[warp][i + half], turn[turn_at(i)], true);
          else if (i < p.rot) y[j] = rotated(y[j], row[warp][i - half], turn[turn_at(i - half)], false);
        }
      }
#pragma unroll
      for (int j = 0; j < kPL; ++j) v[j] = __fadd_rn(y[j].h, y[j].l);
    }
    if (slab) {
      const int h = r - p.n_q - (isk ? 0 : n_kv);
      store_codes<kPL, kFmt>(slab + h * p.c.head_bytes, static_cast<int>(pos & 15), isk,
                             codes[warp], lane, v);
    }
  };
  // one copy of the code: unrolled, it does not stay in the instruction cache
#pragma unroll 1
  for (int r = warp; r < rows; r += kApWarps) {
    float v[kPL];
#pragma unroll
    for (int j = 0; j < kPL; ++j) v[j] = x[j];
    if (r + kApWarps < rows) load_row<kPL>(source(r + kApWarps), lane, x);
    finish(r, v);
  }
  if (kind != kTokenPadding && !slab && threadIdx.x == 0) atomicOr(&g_err_paged, kErrPage);
}

void rotation_turns(int rot_dim, double base, uint64_t* turn) {
  // as in qk_norm_rope: base^(-2i/r) as a product of two powers, 24 powers in place of 128
  double low[16];
  for (int i = 0; i < 16; ++i) low[i] = std::pow(base, -2.0 * i / rot_dim);
  for (int i = 0; i < rot_dim / 2; i += 16) {
    const double high = std::pow(base, -2.0 * i / rot_dim) / 6.283185307179586477;
    for (int j = 0; j < 16 && i + j < rot_dim / 2; ++j)
      turn[i + j] = static_cast<uint64_t>(std::ldexp(high * low[j], 64));
  }
}

template <int kFmt>
cudaError_t launch_append_fmt(const AppendParams& p, int64_t n_tokens, int head_dim,
                              cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(n_tokens));
  switch (head_dim) {
    case 32: return pdl_launch(paged_append_kernel<1, kFmt>, grid, kApWarps * 32, 0, st, p);
    case 64: return pdl_launch(paged_append_kernel<2, kFmt>, grid, kApWarps * 32, 0, st, p);
    case 128: return pdl_launch(paged_append_kernel<4, kFmt>, grid, kApWarps * 32, 0, st, p);
    case 256: return pdl_launch(paged_append_kernel<8, kFmt>, grid, kApWarps * 32, 0, st, p);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_paged_append(const PagedView& c, int fmt, const qws_heads* q,
                                const qws_heads& k, const qws_heads& v, const qws_heads* q_out,
                                const float* w_q, const float* w_k, const int64_t* seqs,
                                const int64_t* positions, int64_t n_tokens, int n_q, int head_dim,
                                int rot_dim, double base, double eps, cudaStream_t st) {
  AppendParams p;
  p.c = c;
  p.k = k; p.v = v;
  p.q = q ? *q : k;
  p.qo = q ? *q_out : k;
  p.n_q = q ? n_q : 0;
  p.w_q = w_q; p.w_k = w_k;
  p.seqs = seqs; p.positions = positions;
  p.rot = rot_dim;
  p.eps.h = static_cast<float>(eps);
  p.eps.l = static_cast<float>(eps - static_cast<double>(p.eps.h));
  const double up = eps < kSmall ? eps * kUp * kUp : 0.0;      // (else no head is below kSmall)
  p.eps_up.h = static_cast<float>(up);
  p.eps_up.l = static_cast<float>(up - static_cast<double>(p.eps_up.h));
  for (int i = 0; i < kApMaxHalf; ++i) p.turn[i] = 0;
  if (rot_dim) rotation_turns(rot_dim, base, p.turn);
  return fmt == QWS_Q4_0 ? launch_append_fmt<QWS_Q4_0>(p, n_tokens, head_dim, st)
                         : launch_append_fmt<QWS_Q8_0>(p, n_tokens, head_dim, st);
}

// ------------------------------------------------------------ gather
// Eight dimensions of a token's key or value row a thread.  Bound by the f32 written, behind
// three reads that depend on one another (the token, its page, the codes): 8192 tokens of 4
// heads of 256, Q4_0, take 15.8 us, 4.8 TB/s; 17.5 with a number of 31 bits for the row and
// conversions.  Two or four rows a thread were slower (18.6, 20.2), and so were 16 tokens' slabs
// read as they lie (19.3).
constexpr int kGaThreads = 256;

struct GatherParams {
  PagedView c;
  qws_heads k, v;
  const int64_t *seqs, *positions;
  int64_t n_tokens;
};

template <int kHd, int kFmt>
__global__ void __launch_bounds__(kGaThreads)
    paged_gather_kernel(const __grid_constant__ GatherParams p) {
  using L = Slab<kHd, kFmt>;
  constexpr int kOf = kHd / 8;             // threads of a row
  pdl_launch_dependents();
  pdl_wait();
  // rows of one token, or, if they are fewer than a CTA has, of several
  constexpr int kRows = kGaThreads / kOf;  // of a CTA
  const int rows = 2 * p.c.n_kv;
  int row = static_cast<int>(threadIdx.x) / kOf;
  int64_t t = blockIdx.x;
  if (rows <= kRows / 2) {
    const int slot = row / rows;
    row -= slot * rows;
    if (slot >= kRows / rows) return;
    t = t * (kRows / rows) + slot;
  } else {
    row += static_cast<int>(blockIdx.y) * kRows;
    if (row >= rows) return;
  }
  if (t >= p.n_tokens) return;
  const int i = static_cast<int>(threadIdx.x) % kOf;
  const bool keys = row < p.c.n_kv;
  const int head = keys ? row : row - p.c.n_kv;
  const int64_t seq = __ldg(p.seqs + t), pos = __ldg(p.positions + t);
  const TokenKind kind = token_kind(p.c, seq, pos);
  const uint8_t* slab = nullptr;
  if (kind == kTokenFine) {
    slab = token_slab(p.c, seq, static_cast<uint32_t>(pos), L::kBytes);
    if (slab) slab += head * p.c.head_bytes;
  }
  if (kind != kTokenPadding && !slab && row == 0 && i == 0) atomicOr(&g_err_paged, kErrPage);
  const qws_heads& out = keys ? p.k : p.v;
  float* to = out.data + t * out.token_stride + head * out.head_stride;
  const int at = static_cast<int>(pos & 15);
  uint32_t w[2] = {0, 0};
  float d[2] = {0.f, 0.f};
  // two runs of four dimensions, half a row apart: a warp's stores lie side by side
  if (slab) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int x = i + s * kOf;
      if (keys) {
        const uint8_t* k = slab + L::key8(at, x / 2) + x % 2 * (4 / L::kPer);
        if constexpr (kFmt == QWS_Q4_0) w[s] = *reinterpret_cast<const uint16_t*>(k);
        else w[s] = *reinterpret_cast<const uint32_t*>(k);
      } else {
#pragma unroll
        for (int h = 0; h < 2 / L::kPer; ++h)
          w[s] |= static_cast<uint32_t>(
                      *reinterpret_cast<const uint16_t*>(slab + L::value4(at, x, h)))
                  << (16 * h);
      }
      d[s] = __half2float(*reinterpret_cast<const __half*>(
          slab + (keys ? L::kKScale : L::kVScale) + 2 * (at * L::kBlocks + x / 8)));
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // the code as the last bits of a number from 2^23 on: the conversion takes longer
      const uint32_t code =
          kFmt == QWS_Q4_0 ? w[s] >> (4 * j) & 15u : w[s] >> (8 * j) & 255u;
      // (0 added: rows of nothing are 0 and not -0)
      y[j] = fmaf(d[s], __uint_as_float(code | 0x4B000000u) - static_cast<float>(8388608 + L::kZero),
                  0.f);
    }
    *reinterpret_cast<float4*>(to + 4 * (i + s * kOf)) = make_float4(y[0], y[1], y[2], y[3]);
  }
}

cudaError_t launch_paged_gather(const PagedView& c, int fmt, const qws_heads& k,
                                const qws_heads& v, const int64_t* seqs, const int64_t* positions,
                                int64_t n_tokens, int head_dim, cudaStream_t st) {
  const GatherParams p{c, k, v, seqs, positions, n_tokens};
  const int rows = 2 * c.n_kv, of_cta = kGaThreads / (head_dim / 8);
  const int64_t tokens = rows <= of_cta / 2 ? of_cta / rows : 1;       // of a CTA
  const dim3 grid(static_cast<unsigned>((n_tokens + tokens - 1) / tokens),
                  static_cast<unsigned>(tokens > 1 ? 1 : (rows + of_cta - 1) / of_cta));
#define QWS_GATHER(HD)                                                                        \
  case HD:                                                                                    \
    return fmt == QWS_Q4_0                                                                    \
               ? pdl_launch(paged_gather_kernel<HD, QWS_Q4_0>, grid, kGaThreads, 0, st, p)    \
               : pdl_launch(paged_gather_kernel<HD, QWS_Q8_0>, grid, kGaThreads, 0, st, p);
  switch (head_dim) {
    QWS_GATHER(32) QWS_GATHER(64) QWS_GATHER(128) QWS_GATHER(256)
  }
#undef QWS_GATHER
  return cudaErrorInvalidValue;
}

unsigned read_clear_paged_errors() {
  unsigned v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_paged, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_err_paged, &z, sizeof(z));
  return v;
}

}  // namespace qws
