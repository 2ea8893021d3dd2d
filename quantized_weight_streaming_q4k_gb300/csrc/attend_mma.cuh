// attend_mma.cuh -- attention of 128 query rows over a run of 64-key tiles on
// the 5th-generation tensor cores, to f32 accuracy.  Shared by the prompt and
// the shared-prefix kernels, which differ in where the key tiles come from.
//
// Every operand is two f16 parts, hi + lo (22 bits), and every product three:
// hi*hi + hi*lo + lo*hi, accumulated in f32.  Before the split a query row and
// a key row are each scaled by a power of two that puts their largest value in
// [2^14, 2^15), the values of a tile by one for the whole tile; the weights
// are at most 2^14.  So a value keeps 22 bits, or 2^-39 of the largest it
// is scaled with.  A key whose values would spoil its tile's scale or be spoilt by it (one
// that is not finite, or further than 2^16 from the tile's others, which may be keys that
// most rows do not even see) is left out of the tile and added at the end, in f32, by the
// rows that see it.
//
// Per tile of 64 keys, S = Q K^T (128 x 64) and O_tile = P V (128 x head_dim).
// Q and P are A operands in tensor memory; K and V come through rings in shared
// memory, both as rows (a key) of 128 bytes (64 columns), swizzled: K as a K-major B
// operand, V as an MN-major one, so neither is transposed.  O_tile is NOT accumulated
// in tensor memory: the tensor cores' f32 accumulation does not round to nearest, and
// its bias grows with the number of steps.  Each tile's O_tile (12 accumulation steps)
// is added to f32 registers with the softmax's rescaling, one multiplication and one fma
// a value, which the three products per value leave time for (256 of about 3000 cycles a
// tile at head_dim 256).  This also spares the correction pass over tensor memory.
//
// Two warps load K and V chunks into the rings, two issue the MMAs of Q K^T and of P V.
// One issuing warp would do, but a commit holds the issuing warp until its MMAs are
// done, and the tensor cores then idle for the next wait; with two, one's MMAs are
// queued behind the other's.  The chunks of O_tile alternate between two accumulators,
// so that one is drained while the next is multiplied.
#pragma once

#include <cuda_runtime.h>

#include "attend_rows.cuh"
#include "tcgen05.cuh"

namespace qws {

// waits that gave up, by who waited
enum : unsigned {
  kErrAttLoad = 1024u,     // a producer waited for a free stage
  kErrAttMma = 2048u,      // the MMA issuer
  kErrAttRows = 4096u,     // the softmax warps
};

constexpr int kTileRows = 128;
constexpr int kTileKeys = 64;
constexpr int kPShift = 14;            // weights are 2^14 exp2(s - max)

// what a key tile carries beside its values
struct __align__(16) TileMeta {
  float kscale[kTileKeys];   // 2^-e of each key row
  float vscale;              // 2^-e of the tile's values
  uint32_t left_out[2];      // keys whose values are not in the tile
  uint32_t pad;
};
static_assert(sizeof(TileMeta) == 272, "copied in 16-byte units");

// A unit: 64 keys x 64 columns of K or V, hi then lo.
// kWholeT: the units of a half tile come and go together, by their first one's barriers.
// kBufsT: buffers of S and of P in tensor memory.
template <int kHdT, int kDepthT, bool kWholeT, int kBufsT>
struct MmaCfg {
  static constexpr int kHd = kHdT;
  static constexpr bool kWhole = kWholeT;
  static constexpr int kBufs = kBufsT;
  // tiles whose meta records are there: with only two, the loads of a tile's K would wait
  // for the softmax of the tile before the last, and the ring would not run ahead
  static constexpr int kMetas = 2 * kBufs;
  static constexpr int kNC = kHd > 64 ? kHd / 64 : 1;   // chunks of head_dim
  static constexpr int kHC = kHd / kNC;                 // columns of a chunk
  static constexpr int kOC = kHC / 2;                   // of a chunk, a thread's
  static constexpr uint32_t kPart = kTileKeys * 128;    // hi or lo of a unit
  static constexpr uint32_t kUnit = 2 * kPart;
  static constexpr uint32_t kHalfTile = kNC * kUnit;    // K, or V, of a tile
  static constexpr uint32_t kTile = 2 * kHalfTile;      // a packed key tile
  // units of each of the two rings: 6, or kDepth whole tiles (a fifth unit for K at head_dim
  // 256 gained nothing)
  static constexpr int kStages = kDepthT ? kDepthT * kNC : 6;
  static constexpr uint32_t kRing = 2 * kStages * kUnit;
  // 8 warps keep the output (thread = row 32 (w % 4) + lane, w / 4 = which half of the
  // output columns); with two buffers of S and P, 8 others the softmax
  static constexpr int kRowsWarps = 8;
  static constexpr uint32_t kScratch = kRowsWarps * 32 * 36 * 4;   // in the V ring
  static_assert(kScratch <= kStages * kUnit, "the V ring holds the scratch");
  static constexpr int kSoftWarps = kBufs > 1 ? 4 : 8;    // of a tile
  static constexpr int kLoadK = kRowsWarps + (kBufs > 1 ? 8 : 0), kLoadV = kLoadK + 1;
  static constexpr int kMmaQk = kLoadK + 2, kMmaPv = kLoadK + 3;
  // Tensor memory columns (all 512 are allocated, so they start at 0): Q hi, Q lo, the
  // buffers of S, those of P (of every 16 keys hi, then lo: 16 columns, as many as their
  // scores take), and two of O_tile.  Where that is too much, Q lo
  // is in shared memory (its MMAs take 48 cycles a step in place of 32).
  static constexpr bool kQLoSmem = kBufs > 1 && kHd > 128;
  static constexpr uint32_t kQLoBytes = kQLoSmem ? kNC * kTileRows * 128 : 0;
  static constexpr uint32_t kTmQhi = 0, kTmQlo = kHd / 2;
  static constexpr uint32_t kTmS = kHd > 128 && !kQLoSmem ? 256 : 128;
  static constexpr uint32_t kTmP = kTmS + 64 * kBufs;
  static constexpr uint32_t kTmO = kTmP + 64 * kBufs;
  static_assert(kTmO + 128 <= 512, "tensor memory");
};

template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// barriers and small exchanges of one CTA
template <class Cfg>
struct MmaShared {
  uint64_t k_full[Cfg::kStages], k_empty[Cfg::kStages];
  uint64_t v_full[Cfg::kStages], v_empty[Cfg::kStages];
  uint64_t meta_full[Cfg::kMetas], meta_free[Cfg::kMetas];      // kscale
  uint64_t vmeta_full[Cfg::kMetas], vmeta_free[Cfg::kMetas];    // vscale, left_out
  uint64_t o_full[2], o_free[2];
  uint64_t s_full[Cfg::kBufs], s_free[Cfg::kBufs];
  uint64_t p_ready[Cfg::kBufs], p_free[Cfg::kBufs];
  uint64_t m_free[2];
  uint64_t q_ready, done[2];
  uint32_t tmem;
  uint32_t dead;
  float qmax[2][kTileRows];
  float x[2][2][kTileRows];
  TileMeta meta[Cfg::kMetas];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 bits2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
// a two-f32 version of split_f16x2: hi and lo of both
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(x.x, x.y);
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  const float2 r = __ffma2_rn(h, make_float2(-1.f, -1.f), x);      // exact
  lo = pack_f16x2(r.x, r.y);
}

// The softcap of a thread's scores of a tile, x in units of log 2: with c = cap log2 e and
// y = x / c, c tanh(y) = x P(y^2).  P is fitted to tanh(y) / y in y^2: with four terms, which
// hold it to 6e-9 while |y| <= 1/4 in the whole warp (scores well within the cap are), with
// eight to 1, where they leave 2.3e-8 (tanh in f32: 9e-8 and 1.2e-7 with the roundings);
// beyond, 1 - 2 / (1 + e^2|y|), which is 1.2e-7 absolute on values above 0.76.  The library's
// tanhf costs some 60 instructions a score here, four times the rest of the softmax; this 4
// or 7.  As a factor on x, P loses nothing where the cap is so far above the scores that y,
// or 1 / c, is subnormal or zero: it is 1 there.
struct SoftCap {
  float c, inv;
  __device__ __forceinline__ explicit SoftCap(float cap)
      : c(cap * kLog2e), inv(fminf(1.f / (cap * kLog2e), 3.4028235e38f)) {}   // 0 * inf is NaN
};
template <int kN>
__device__ __forceinline__ float2 tanh_ratio(float2 y, const float (&c)[kN]) {
  const float2 z = __fmul2_rn(y, y);
  float2 p = make_float2(c[kN - 1], c[kN - 1]);
#pragma unroll
  for (int i = kN - 2; i >= 0; --i) p = __ffma2_rn(p, z, make_float2(c[i], c[i]));
  return p;
}
__device__ __forceinline__ float tanh_big(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(fabsf(y) * (2.f * kLog2e))));
  return copysignf(1.f - 2.f * r, y);
}
template <int kN>
__device__ __forceinline__ void soft_caps(float (&x)[kN], SoftCap cap) {
  constexpr float kSmall[4] = {1.0f, -0.33333206f, 0.13323133f, -0.051327724f};
  constexpr float kAll[8] = {1.0f,          -0.333332777f,   0.133321598f,  -0.0538709126f,
                             0.0214648172f, -0.00791743957f, 0.00228222599f, -0.000353344454f};
  const float2 inv = make_float2(cap.inv, cap.inv);
  float a = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < kN; ++i) a = fmaxf(a, fabsf(x[i]));
  a *= cap.inv;
  if (!__any_sync(0xFFFFFFFFu, a > 0.25f)) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const float2 v = make_float2(x[i], x[i + 1]);
      const float2 r = __fmul2_rn(v, tanh_ratio(__fmul2_rn(v, inv), kSmall));
      x[i] = r.x;
      x[i + 1] = r.y;
    }
  } else {
    const bool big = __any_sync(0xFFFFFFFFu, a > 1.f);
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const float2 v = make_float2(x[i], x[i + 1]), y = __fmul2_rn(v, inv);
      float2 r = __fmul2_rn(v, tanh_ratio(y, kAll));
      if (big) {
        r.x = fabsf(y.x) > 1.f ? cap.c * tanh_big(y.x) : r.x;
        r.y = fabsf(y.y) > 1.f ? cap.c * tanh_big(y.y) : r.y;
      }
      x[i] = r.x;
      x[i + 1] = r.y;
    }
  }
}

// e with a 2^e in [2^14, 2^15) for a finite a >= 0 (0 for zero), within +-126 (a
// subnormal a stays below).
__device__ __forceinline__ int split_exp(float a) {
  const int e = 141 - static_cast<int>(__float_as_uint(a) >> 23);
  return a > 0.f ? min(126, e) : 0;
}
__device__ __forceinline__ bool finite_bits(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

template <class Cfg>
__device__ __forceinline__ void mma_init_barriers(MmaShared<Cfg>& sh, uint32_t key_count,
                                                  uint32_t value_count) {
  for (int s = 0; s < Cfg::kStages; ++s) {
    mbar_init(&sh.k_full[s], key_count);
    mbar_init(&sh.k_empty[s], 1);
    mbar_init(&sh.v_full[s], value_count);
    mbar_init(&sh.v_empty[s], 1);
  }
  for (int s = 0; s < Cfg::kMetas; ++s) {
    mbar_init(&sh.meta_full[s], key_count);
    mbar_init(&sh.meta_free[s], Cfg::kSoftWarps);
    mbar_init(&sh.vmeta_full[s], value_count);
    mbar_init(&sh.vmeta_free[s], Cfg::kRowsWarps);
  }
  for (int s = 0; s < 2; ++s) {
    mbar_init(&sh.o_full[s], 1);
    mbar_init(&sh.o_free[s], Cfg::kRowsWarps);
    mbar_init(&sh.m_free[s], Cfg::kRowsWarps);
    mbar_init(&sh.done[s], 1);
  }
  for (int s = 0; s < Cfg::kBufs; ++s) {
    mbar_init(&sh.s_full[s], 1);
    mbar_init(&sh.s_free[s], Cfg::kSoftWarps);
    mbar_init(&sh.p_ready[s], Cfg::kSoftWarps);
    mbar_init(&sh.p_free[s], 1);
  }
  mbar_init(&sh.q_ready, Cfg::kRowsWarps);
  sh.dead = 0;
  fence_barrier_init();
}

// A place in a ring of kStages: stage and the parity of its current phase.
template <int kStages>
struct RingAt {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Both phases are over, or dead: asked together, as a wait costs some 200 cycles even so.
__device__ __forceinline__ void wait2(uint64_t* a, uint32_t a_par, uint64_t* b, uint32_t b_par,
                                      bool& dead) {
  if (!__all_sync(0xFFFFFFFFu, mbar_test(a, a_par) & mbar_test(b, b_par)) && !dead)
    dead = !__all_sync(0xFFFFFFFFu, mbar_wait(a, a_par) && mbar_wait(b, b_par));
}

// ------------------------------------------------------------ the MMA issuers
// Each a whole warp.  A wait costs some 200 cycles here even if it is over, so the barriers
// of a chunk are asked together, and waited for one by one only after a no.
// S(j) = Q K(j)^T, once what was in its buffer has been read, chunk after chunk of
// head_dim: the small cross terms of all chunks, then hi * hi of all.  The tensor cores
// round each step's sum towards zero, so the fewer steps at the sum's full size the better:
// with both in one pass over the chunks the outputs' error at head_dim 256 was twice as
// large (9.8e-7 for 5.1e-7; plain f32 5.2e-7), and the second pass costs 2 %.
template <class Cfg>
__device__ __forceinline__ void mma_issue_qk(MmaShared<Cfg>& sh, uint8_t* k_ring,
                                             const uint8_t* q_lo, int n, unsigned* err) {
  constexpr uint32_t kIdesc = tc_idesc_f16(kTileRows, kTileKeys);
  constexpr int kSteps = Cfg::kHC / 16;
  const uint32_t one = elect_one();
  const uint32_t base = sw128_lo(smem_addr(k_ring));   // units of 16 bytes
  const uint32_t lo_base = sw128_lo(smem_addr(q_lo));
  RingAt<Cfg::kStages> at;
  RingAt<Cfg::kBufs> buf;
  bool ok = n <= 0 || __all_sync(0xFFFFFFFFu, mbar_wait(&sh.q_ready, 0));
  for (int j = 0; j < n && ok; ++j) {
    const uint32_t d = Cfg::kTmS + static_cast<uint32_t>(buf.stage) * 64u;
    const RingAt<Cfg::kStages> start = at;
#pragma unroll 1
    for (int c = 0; c < Cfg::kNC; ++c) {
      const bool unit = !(Cfg::kWhole && c > 0), tile = c == 0 && j >= Cfg::kBufs;
      uint64_t* const s_free = &sh.s_free[buf.stage];
      uint64_t* const k_full = &sh.k_full[at.stage];
      const bool there = (!unit || mbar_test(k_full, at.phase)) &
                         (!tile || mbar_test(s_free, buf.phase ^ 1u));
      if (!__all_sync(0xFFFFFFFFu, there))
        ok = __all_sync(0xFFFFFFFFu, (!unit || mbar_wait(k_full, at.phase)) &&
                                         (!tile || mbar_wait(s_free, buf.phase ^ 1u)));
      tc_fence_after();
      if (!ok) break;
      const uint32_t b = base + static_cast<uint32_t>(at.stage) * (Cfg::kUnit >> 4);
      at.next();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint32_t off = (t == 0 ? Cfg::kPart : 0u) + static_cast<uint32_t>(k) * 32u;
          const uint32_t add = (t | k) != 0 || c > 0 ? 1u : 0u;
          if constexpr (Cfg::kQLoSmem) {
            if (t == 1) {
              tc_mma_f16_ss(d, lo_base + static_cast<uint32_t>(c * kTileRows * 8 + k * 2),
                            b + (off >> 4), kIdesc, add, one);
              continue;
            }
          }
          const uint32_t a = (t == 1 ? Cfg::kTmQlo : Cfg::kTmQhi) +
                             static_cast<uint32_t>(c * kSteps + k) * 8u;
          tc_mma_f16_ts(d, a, b + (off >> 4), kIdesc, add, one);
        }
      }
    }
    if (!ok) break;
    at = start;
#pragma unroll 1
    for (int c = 0; c < Cfg::kNC; ++c) {
      const uint32_t b = base + static_cast<uint32_t>(at.stage) * (Cfg::kUnit >> 4);
      uint64_t* empty = &sh.k_empty[Cfg::kWhole ? at.stage - c : at.stage];
      at.next();
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        tc_mma_f16_ts(d, Cfg::kTmQhi + static_cast<uint32_t>(c * kSteps + k) * 8u,
                      b + static_cast<uint32_t>(k) * 2u, kIdesc, 1u, one);
      if (!Cfg::kWhole || c == Cfg::kNC - 1) tc_commit(empty, one);
    }
    tc_commit(&sh.s_full[buf.stage], one);
    buf.next();
  }
  if (!ok && one) atomicOr(err, kErrAttMma);
  tc_commit(&sh.done[0], one);     // arrives when every MMA above has completed
}

// O_tile(j) = P(j) V(j), a 64-column chunk at a time in one of two accumulators.
template <class Cfg>
__device__ __forceinline__ void mma_issue_pv(MmaShared<Cfg>& sh, uint8_t* v_ring, int n,
                                             unsigned* err) {
  constexpr uint32_t kIdesc = tc_idesc_f16(kTileRows, Cfg::kHC) | kIdescBMn;
  const uint32_t one = elect_one();
  const uint32_t base = sw128_lo(smem_addr(v_ring));
  RingAt<Cfg::kStages> at;
  RingAt<2> buf;
  RingAt<Cfg::kBufs> pb;
  bool ok = true;
  for (int j = 0; j < n && ok; ++j) {
#pragma unroll 1
    for (int c = 0; c < Cfg::kNC; ++c) {
      const bool unit = !(Cfg::kWhole && c > 0), tile = c == 0;
      uint64_t* const v_full = &sh.v_full[at.stage];
      uint64_t* const o_free = &sh.o_free[buf.stage];       // the first use of each passes
      uint64_t* const p_ready = &sh.p_ready[pb.stage];
      const bool there = (!unit || mbar_test(v_full, at.phase)) &
                         mbar_test(o_free, buf.phase ^ 1u) &
                         (!tile || mbar_test(p_ready, pb.phase));
      if (!__all_sync(0xFFFFFFFFu, there))
        ok = __all_sync(0xFFFFFFFFu, (!unit || mbar_wait(v_full, at.phase)) &&
                                         mbar_wait(o_free, buf.phase ^ 1u) &&
                                         (!tile || mbar_wait(p_ready, pb.phase)));
      tc_fence_after();
      if (!ok) break;
      const uint32_t b = base + static_cast<uint32_t>(at.stage) * (Cfg::kUnit >> 4);
      const uint32_t d = Cfg::kTmO + static_cast<uint32_t>(buf.stage) * 64u;
      const uint32_t hi = Cfg::kTmP + static_cast<uint32_t>(pb.stage) * 64u, lo = hi + 8u;
      uint64_t* full = &sh.o_full[buf.stage];
      uint64_t* empty = &sh.v_empty[Cfg::kWhole ? at.stage - c : at.stage];
      at.next();
      buf.next();
#pragma unroll
      for (int t = 0; t < 3; ++t) {
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; ++k) {
          const uint32_t a = (t == 1 ? lo : hi) + static_cast<uint32_t>(k) * 16u;
          const uint32_t off = (t == 0 ? Cfg::kPart : 0u) + static_cast<uint32_t>(k) * 2048u;
          tc_mma_f16_ts(d, a, b + (off >> 4), kIdesc, (t | k) != 0 ? 1u : 0u, one);
        }
      }
      tc_commit(full, one);
      if (!Cfg::kWhole || c == Cfg::kNC - 1) tc_commit(empty, one);
      if (Cfg::kBufs > 1 && c == Cfg::kNC - 1) tc_commit(&sh.p_free[pb.stage], one);
    }
    pb.next();
  }
  if (!ok && one) atomicOr(err, kErrAttMma);
  tc_commit(&sh.done[1], one);
}

// A loader: one thread.  Waits for a free stage before each of the n * kNC units;
// copy(stage, j, c) starts the copy of chunk c of tile j; before(j) comes before a
// tile's first, and returns false when it gave up.  Ends when its copies have landed.
template <class Cfg, class Before, class Copy>
__device__ __forceinline__ void mma_load(uint64_t* full, uint64_t* empty, int n, Before&& before,
                                         Copy&& copy, unsigned* err) {
  RingAt<Cfg::kStages> at;
  bool ok = true;
  int units = 0;
  for (int j = 0; j < n && ok; ++j) {
    ok = before(j);
    for (int c = 0; c < Cfg::kNC && ok; ++c) {
      ok = mbar_wait(&empty[at.stage], at.phase ^ 1u);
      if (!ok) break;
      copy(at.stage, j, c);
      at.next();
      ++units;
    }
  }
  for (int u = max(0, units - Cfg::kStages); u < units; ++u)
    ok = mbar_wait(&full[u % Cfg::kStages], static_cast<uint32_t>(u / Cfg::kStages) & 1u) && ok;
  if (!ok) atomicOr(err, kErrAttLoad);
}

// ------------------------------------------------------------ rows
template <class Cfg>
struct RowState {
  float2 o[Cfg::kNC][Cfg::kOC / 2];
  float m, l;              // of the whole row
  bool any_left_out;
};

// The 128 query rows, scaled and split into tensor memory (Q lo: into q_lo, if it is in
// shared memory), by the 8 warps that keep the output.  q: the row's head_dim values, or
// null (a row of zeros).  A lane of its own row would touch 32 lines a load: a warp reads
// its half of its 32 rows in runs of kRun columns, several lanes a row, and turns what
// goes to tensor memory through its part of scratch (kScratch bytes that nothing else
// uses until q_ready).
template <class Cfg>
__device__ __forceinline__ void store_q(MmaShared<Cfg>& sh, float* scratch, uint8_t* q_lo,
                                        const float* q) {
  constexpr int kQC = Cfg::kHd / 2, kRun = kQC < 32 ? kQC : 32, kLanes = kRun / 4;
  constexpr int kAt = 32 / kLanes, kLoads = 32 / kAt, kRuns = kQC / kRun;
  constexpr int kPitch = kRun + 4;         // hi, lo of a row
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int quad = warp & 3, part = warp >> 2;
  const int r0 = 32 * quad + lane / kLanes, at = lane % kLanes;
  float4 v[kRuns][kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const float* src = reinterpret_cast<const float*>(__shfl_sync(
        0xFFFFFFFFu, reinterpret_cast<unsigned long long>(q), k * kAt + lane / kLanes));
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      v[r][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (src) v[r][k] = *reinterpret_cast<const float4*>(src + part * kQC + r * kRun + at * 4);
    }
  }
  // the largest finite magnitude of each row; infinities, which are rare, in a second pass
  float a[kLoads];
  const auto largest = [&](bool all) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      a[k] = 0.f;
#pragma unroll
      for (int r = 0; r < kRuns; ++r) {
        const float o[4] = {v[r][k].x, v[r][k].y, v[r][k].z, v[r][k].w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (all || finite_bits(o[c])) a[k] = fmaxf(a[k], fabsf(o[c]));
      }
    }
  };
  largest(true);
  float top = a[0];
#pragma unroll
  for (int k = 1; k < kLoads; ++k) top = fmaxf(top, a[k]);
  if (__any_sync(0xFFFFFFFFu, top == INFINITY)) largest(false);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < kLoads; ++k) a[k] = fmaxf(a[k], __shfl_xor_sync(0xFFFFFFFFu, a[k], o));
#pragma unroll
  for (int k = 0; k < kLoads; ++k)
    if (at == 0) sh.qmax[part][r0 + k * kAt] = a[k];
  bar_sync(1 + quad, 64);
  uint32_t* mine = reinterpret_cast<uint32_t*>(scratch) + warp * 32 * kPitch;
  const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
#pragma unroll
  for (int k = 0; k < kLoads; ++k)
    a[k] = exp2i(split_exp(fmaxf(a[k], sh.qmax[part ^ 1][r0 + k * kAt])));
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    if (r > 0) __syncwarp();
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const float2 f = make_float2(a[k], a[k]);
      uint2 hi, lo;
      split2(__fmul2_rn(make_float2(v[r][k].x, v[r][k].y), f), hi.x, lo.x);
      split2(__fmul2_rn(make_float2(v[r][k].z, v[r][k].w), f), hi.y, lo.y);
      uint32_t* to = mine + (k * kAt + lane / kLanes) * kPitch + at * 2;
      *reinterpret_cast<uint2*>(to) = hi;
      if constexpr (Cfg::kQLoSmem) {
        const uint32_t col = static_cast<uint32_t>(part * kQC + r * kRun + at * 4);
        *reinterpret_cast<uint2*>(
            q_lo + (col / 64) * (kTileRows * 128) +
            sw128_off(static_cast<uint32_t>(r0 + k * kAt), (col % 64) / 8) + (col % 8) * 2) = lo;
      } else {
        *reinterpret_cast<uint2*>(to + kRun / 2) = lo;
      }
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < (Cfg::kQLoSmem ? 1 : 2); ++t) {
      uint32_t w[kRun / 2];
#pragma unroll
      for (int i = 0; i < kRun / 2; i += 4) {
        const uint4 y = *reinterpret_cast<const uint4*>(mine + lane * kPitch + t * (kRun / 2) + i);
        w[i] = y.x; w[i + 1] = y.y; w[i + 2] = y.z; w[i + 3] = y.w;
      }
      tc_st<kRun / 2>(lanes + (t == 0 ? Cfg::kTmQhi : Cfg::kTmQlo) +
                          static_cast<uint32_t>((part * kQC + r * kRun) / 2),
                      w);
    }
  }
  tc_wait_st();
  fence_proxy_async_smem();      // Q lo is read, and the scratch overwritten, by that proxy
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.q_ready);
}
// 2^-e of a row's split, once q_ready has been waited for (or by store_q's warps)
template <class Cfg>
__device__ __forceinline__ float q_unscale(const MmaShared<Cfg>& sh, int row) {
  return exp2i(-split_exp(fmaxf(sh.qmax[0][row], sh.qmax[1][row])));
}

// A key left out of its tile (see the head of this file): its weight from the
// row's final maximum, and its values, in f32.
template <class Cfg>
__device__ __forceinline__ void add_left_out(RowState<Cfg>& st, const float* q, const float* k,
                                          const float* v, int part, float scale, float cap) {
  float s = 0.f;
  for (int i = 0; i < Cfg::kHd; i += 4) {
    const float4 a = *reinterpret_cast<const float4*>(q + i);
    const float4 b = *reinterpret_cast<const float4*>(k + i);
    s = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
  }
  const float base = st.m == -INFINITY ? 0.f : st.m;
  const float p = ex2(soft_cap(s * scale, cap) * kLog2e - (base - static_cast<float>(kPShift)));
#pragma unroll
  for (int c = 0; c < Cfg::kNC; ++c)
#pragma unroll
    for (int i = 0; i < Cfg::kOC; i += 2) {
      const float2 x = *reinterpret_cast<const float2*>(v + c * Cfg::kHC + part * Cfg::kOC + i);
      st.o[c][i / 2] = __ffma2_rn(make_float2(p, p), x, st.o[c][i / 2]);
    }
}

// f * o into the rows at dst (null: not stored), turned through the warp's scratch so
// that a store covers whole lines
template <class Cfg>
__device__ __forceinline__ void store_rows(const RowState<Cfg>& st, float* scratch, float* dst,
                                           float f) {
  constexpr int kLanes = Cfg::kOC / 4, kAt = 32 / kLanes, kPitch = Cfg::kOC + 4;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int part = warp >> 2;
  float* mine = scratch + warp * 32 * kPitch;
#pragma unroll
  for (int c = 0; c < Cfg::kNC; ++c) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < Cfg::kOC; i += 4)
      *reinterpret_cast<float4*>(mine + lane * kPitch + i) =
          make_float4(st.o[c][i / 2].x * f, st.o[c][i / 2].y * f, st.o[c][i / 2 + 1].x * f,
                      st.o[c][i / 2 + 1].y * f);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 32 / kAt; ++k) {
      const int r = k * kAt + lane / kLanes, i = (lane % kLanes) * 4;
      float* to = reinterpret_cast<float*>(
          __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(dst), r));
      if (to)
        *reinterpret_cast<float4*>(to + c * Cfg::kHC + part * Cfg::kOC + i) =
            *reinterpret_cast<const float4*>(mine + r * kPitch + i);
    }
  }
}

// ------------------------------------------------------------ key tiles
// One key row (a lane's kPL = head_dim / 32 columns of it, times sc) as hi and lo f16 at
// the lane's place in the units: `at` for its first columns, a unit further for the
// group of columns 128 on (two units).
template <class Cfg>
__device__ __forceinline__ void store_split_at(const float (&x)[Cfg::kHd / 32], float sc, int lane,
                                               uint8_t* at) {
  constexpr int kPL = Cfg::kHd / 32;
  if constexpr (kPL >= 4) {
#pragma unroll
    for (int i = 0; i < kPL; i += 4) {
      const float2 f = make_float2(sc, sc);
      uint2 hi, lo;
      split2(__fmul2_rn(make_float2(x[i], x[i + 1]), f), hi.x, lo.x);
      split2(__fmul2_rn(make_float2(x[i + 2], x[i + 3]), f), hi.y, lo.y);
      uint8_t* u = at + (i / 4) * 2 * Cfg::kUnit;
      *reinterpret_cast<uint2*>(u) = hi;
      *reinterpret_cast<uint2*>(u + Cfg::kPart) = lo;
    }
  } else {
    float a = x[0] * sc, b;
    if constexpr (kPL == 2) b = x[1] * sc;
    else b = __shfl_xor_sync(0xFFFFFFFFu, a, 1);
    uint32_t hi, lo;
    split_f16x2(a, b, hi, lo);
    if (kPL == 2 || !(lane & 1)) {
      *reinterpret_cast<uint32_t*>(at) = hi;
      *reinterpret_cast<uint32_t*>(at + Cfg::kPart) = lo;
    }
  }
}

// the same into row r of the units at dst
template <class Cfg>
__device__ __forceinline__ void store_split_row(const float (&x)[Cfg::kHd / 32], float sc, int r,
                                                int lane, uint8_t* dst) {
  const int c = lane_col<Cfg::kHd / 32>(lane, 0);
  store_split_at<Cfg>(x, sc, lane,
                      dst + (c / 64) * Cfg::kUnit +
                          sw128_off(static_cast<uint32_t>(r), static_cast<uint32_t>(c % 64) / 8u) +
                          (c % 8) * 2);
}

// largest finite magnitude of a row over the warp; `all`: every value is finite.  The
// bits of a magnitude compare as unsigned numbers, infinities and NaN on top.
template <int kPL>
__device__ __forceinline__ float row_amax(const float (&x)[kPL], bool& all) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kPL; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  a = __reduce_max_sync(0xFFFFFFFFu, a);
  all = a < 0x7F800000u;
  if (!all) {
    a = 0;
#pragma unroll
    for (int i = 0; i < kPL; ++i)
      a = max(a, finite_bits(x[i]) ? __float_as_uint(x[i]) & 0x7FFFFFFFu : 0u);
    a = __reduce_max_sync(0xFFFFFFFFu, a);
  }
  return __uint_as_float(a);
}

// 64 keys of one kv head, n of them there (the rest zero), by a CTA of 256 threads: K as
// units at dst and the keys' scales.
template <class Cfg>
__device__ __forceinline__ void pack_keys(const float* K, int64_t stride, int n, uint8_t* dst,
                                          TileMeta* meta) {
  constexpr int kPL = Cfg::kHd / 32, kRows = kTileKeys / 8;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  float x[kRows][kPL];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + 8 * i;
#pragma unroll
    for (int c = 0; c < kPL; ++c) x[i][c] = 0.f;
    if (r < n) load_row<kPL>(K + r * stride, lane, x[i]);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + 8 * i;
    bool fin;
    const int e = split_exp(row_amax<kPL>(x[i], fin));
    store_split_row<Cfg>(x[i], exp2i(e), r, lane, dst);
    if (lane == 0) meta->kscale[r] = exp2i(-e);
  }
}

// Which of a tile's value rows share its scale: those within 2^16 of the smallest that is not
// zero, or those within 2^16 of the largest that is finite, whichever leaves out fewer.  a, b:
// the largest magnitudes of rows lane and lane + 32, infinite for a row with an infinity or
// NaN.  By a whole warp, the same in every lane.
struct ValueScale {
  uint32_t out[2];       // rows left out
  float top;             // the largest magnitude of the others
};
__device__ __forceinline__ ValueScale choose_value_scale(float a, float b) {
  float lo = fminf(a > 0.f ? a : INFINITY, b > 0.f ? b : INFINITY);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
  const float hi = warp_max(fmaxf(a == INFINITY ? 0.f : a, b == INFINITY ? 0.f : b));
  const float top = lo * 65536.0f, low = hi * (1.0f / 65536.0f);     // top: may be infinite
  const auto count = [](bool x, bool y) {
    return __popc(__ballot_sync(0xFFFFFFFFu, x)) + __popc(__ballot_sync(0xFFFFFFFFu, y));
  };
  const bool big_a = a == INFINITY || a > top, big_b = b == INFINITY || b > top;
  const bool few_a = a == INFINITY || (a > 0.f && a < low);
  const bool few_b = b == INFINITY || (b > 0.f && b < low);
  const bool large = count(big_a, big_b) <= count(few_a, few_b);
  const bool out_a = large ? big_a : few_a, out_b = large ? big_b : few_b;
  ValueScale sc;
  sc.out[0] = __ballot_sync(0xFFFFFFFFu, out_a);
  sc.out[1] = __ballot_sync(0xFFFFFFFFu, out_b);
  sc.top = warp_max(fmaxf(out_a ? 0.f : a, out_b ? 0.f : b));
  return sc;
}

// Their values, likewise, with one scale for the tile.
template <class Cfg>
__device__ __forceinline__ void pack_values(const float* V, int64_t stride, int n, uint8_t* dst,
                                            TileMeta* meta) {
  constexpr int kPL = Cfg::kHd / 32, kRows = kTileKeys / 8;
  __shared__ float vmax[kTileKeys];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  float y[kRows][kPL];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + 8 * i;
#pragma unroll
    for (int c = 0; c < kPL; ++c) y[i][c] = 0.f;
    if (r < n) load_row<kPL>(V + r * stride, lane, y[i]);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    bool fin;
    const float b = row_amax<kPL>(y[i], fin);
    if (lane == 0) vmax[warp + 8 * i] = fin ? b : INFINITY;
  }
  __syncthreads();
  const ValueScale sc = choose_value_scale(vmax[lane], vmax[lane + 32]);      // the same in all warps
  const int e = split_exp(sc.top);
  if (threadIdx.x == 0) {
    meta->vscale = exp2i(-e);
    meta->left_out[0] = sc.out[0];
    meta->left_out[1] = sc.out[1];
    meta->pad = 0;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + 8 * i;
    const bool out = ((r < 32 ? sc.out[0] : sc.out[1]) >> (r & 31)) & 1u;
#pragma unroll
    for (int c = 0; c < kPL; ++c) y[i][c] = out ? 0.f : y[i][c];
    store_split_row<Cfg>(y[i], exp2i(e), r, lane, dst);
  }
}

}  // namespace qws
