// attend_mma.cuh -- attention of 128 query rows over a run of 64-key tiles on
// the 5th-generation tensor cores, to f32 accuracy.  Shared by the prompt and
// the shared-prefix kernels, which differ in where the key tiles come from.
//
// Every operand is two f16 parts, hi + lo (22 bits), and every product three:
// hi*hi + hi*lo + lo*hi, accumulated in f32.  Before the split a query row and
// a key row are each scaled by a power of two that puts their largest value in
// [2^14, 2^15), the values of a tile by one for the whole tile; the weights
// are at most 2^14.  So a value keeps 22 bits, or 2^-40 of the largest it
// is scaled with.  A key whose values would spoil its tile's scale (one that is
// not finite, or over 2^16 times the tile's smallest: such a key may be one
// that most rows do not even see) is left out of the tile and added at the end,
// in f32, by the rows that see it.
//
// Per tile of 64 keys, S = Q K^T (128 x 64) and O_tile = P V (128 x head_dim).
// Q hi / lo and P hi / lo are A operands in tensor memory; K and V come through
// rings in shared memory, both as rows (a key) of 128 bytes (64 columns), swizzled: K
// as a K-major B operand, V as an MN-major one, so neither is transposed.  O_tile is
// NOT accumulated in tensor memory: the tensor cores' f32 accumulation does
// not round to nearest, and its bias grows with the number of steps.  Each
// tile's O_tile (12 accumulation steps) is added to f32 registers with the
// softmax's rescaling, one multiplication and one fma a value, which the three
// products per value leave time for (256 of about 3000 cycles a tile at head_dim
// 256).  This also spares the correction pass over tensor memory.
//
// TMEM columns (all 512 are allocated, so they start at 0): Q hi 0.., Q lo 128..,
// S 256.., P hi 320.., P lo 352.., O_tile 384.. and 448.. (64 columns each: the 64-column
// chunks of O_tile take turns).
//
// Roles: 4 * kSplit softmax warps (thread = row 32 (w % 4) + lane, w / 4 = which part of
// the tile's keys and of the output columns) and four helper warps: two load K and V
// chunks into their rings, two issue the MMAs of Q K^T and of P V.  One issuing warp
// would do, but a commit holds the issuing warp until its MMAs are done, and the tensor
// cores then idle for the next wait; with two, one's MMAs are queued behind the other's.
// A softmax warp turns S(j+1) into weights before it drains O_tile(j), so that Q K(j+2)^T
// and P V(j) run behind it; the chunks of O_tile alternate between two accumulators, so
// that a chunk is drained while the next is multiplied.
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
__device__ constexpr float kTanh[8] = {1.0f, -0.333332777f, 0.133321598f, -0.0538709126f, 0.0214648172f, -0.00791743957f, 0.00228222599f, -0.000353344454f};
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
template <int kHdT, int kSplitT, int kDepthT = 0, bool kWholeT = false>
struct MmaCfg {
  static constexpr int kHd = kHdT;
  static constexpr bool kWhole = kWholeT;
  static constexpr int kSplit = kSplitT;                // threads of a query row
  static constexpr int kNC = kHd > 64 ? kHd / 64 : 1;   // chunks of head_dim
  static constexpr int kHC = kHd / kNC;                 // columns of a chunk
  static constexpr int kKeys = kTileKeys / kSplit;      // of a tile, a thread's
  static constexpr int kOC = kHC / kSplit;              // of a chunk, a thread's
  static constexpr uint32_t kPart = kTileKeys * 128;    // hi or lo of a unit
  static constexpr uint32_t kUnit = 2 * kPart;
  static constexpr uint32_t kHalfTile = kNC * kUnit;    // K, or V, of a tile
  static constexpr uint32_t kTile = 2 * kHalfTile;      // a packed key tile
  // units of each of the two rings: 6, or kDepth whole tiles
  static constexpr int kStages = kDepthT ? kDepthT * kNC : 6;
  static constexpr uint32_t kRing = 2 * kStages * kUnit;
  // softmax warps, then the helpers
  static constexpr int kRowsWarps = 4 * kSplit;
  static constexpr uint32_t kScratch = kRowsWarps * 32 * 36 * 4;   // in the V ring
  static_assert(kScratch <= kStages * kUnit, "the V ring holds the scratch");
  static constexpr int kLoadK = kRowsWarps, kLoadV = kRowsWarps + 1;
  static constexpr int kMmaQk = kRowsWarps + 2, kMmaPv = kRowsWarps + 3;
  static constexpr int kThreads = 32 * (kRowsWarps + 4);
  // Registers: a scheduler's quarter of the file (16384) holds 3 (5 for kSplit = 4)
  // warps, 168 (96) a thread at launch; the helpers keep few and the softmax warps
  // take what that frees: 2 x 224 + 56 = 3 x 168, 4 x 112 + 32 = 5 x 96.
  static_assert(kSplit == 2 || kSplit == 4, "register split");
};

template <class Cfg>
__device__ __forceinline__ void regs_few() {
  if constexpr (Cfg::kSplit == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
}
template <class Cfg>
__device__ __forceinline__ void regs_many() {
  if constexpr (Cfg::kSplit == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
}

constexpr uint32_t kTmQhi = 0, kTmQlo = 128, kTmS = 256, kTmPhi = 320, kTmPlo = 352, kTmO = 384;

// barriers and small exchanges of one CTA
template <class Cfg>
struct MmaShared {
  uint64_t k_full[Cfg::kStages], k_empty[Cfg::kStages];
  uint64_t v_full[Cfg::kStages], v_empty[Cfg::kStages];
  uint64_t meta_full[2], meta_free[2];      // kscale
  uint64_t vmeta_full[2], vmeta_free[2];    // vscale, left_out
  uint64_t o_full[2], o_free[2];
  uint64_t q_ready, s_full, s_free, p_ready, done[2];
  uint32_t tmem;
  uint32_t pad;
  float xmax[2][Cfg::kSplit][kTileRows];
  TileMeta meta[2];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (d0, d1) = (a0, a1) * (b, b)
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0,
                                     float b1) {
  asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rc, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rc;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// (d0, d1) = (d0, d1) * (a, a) + (b0, b1)
__device__ __forceinline__ void scale_add2(float& d0, float& d1, float a, float b0, float b1) {
  asm("{\n\t.reg .b64 rd, ra, rb;\n\t"
      "mov.b64 rd, {%0, %1};\n\t"
      "mov.b64 ra, {%2, %2};\n\t"
      "mov.b64 rb, {%3, %4};\n\t"
      "fma.rn.f32x2 rd, rd, ra, rb;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a), "f"(b0), "f"(b1));
}

// out = scale * tanh(y) in place, for a thread's scores of a tile.  |y| <= 1 (scores
// within the cap): y P(y^2), P fitted to tanh(y) / y on [0, 1] in y^2 with a relative
// error below 5e-9, so 1e-7 with the roundings; beyond, 1 - 2 / (1 + e^2|y|), which is 1.2e-7
// absolute on values above 0.76.  The library's tanhf costs some 60 instructions a score
// here, four times the rest of the softmax; this 12.
__device__ __forceinline__ float tanh_small(float y) {
  const float z = y * y;
  float p = kTanh[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) p = fmaf(p, z, kTanh[i]);
  return y * p;
}
template <int kN>
__device__ __forceinline__ void tanh_scaled(float (&y)[kN], float scale) {
  float a = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < kN; ++i) a = fmaxf(a, fabsf(y[i]));
  if (!__any_sync(0xFFFFFFFFu, a > 1.f)) {
#pragma unroll
    for (int i = 0; i < kN; ++i) y[i] = tanh_small(y[i]) * scale;
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float b = fabsf(y[i]);
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(b * (2.f * kLog2e))));
      const float big = copysignf(1.f - 2.f * r, y[i]);
      y[i] = (b > 1.f ? big : tanh_small(y[i])) * scale;
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
__device__ __forceinline__ void mma_init_barriers(MmaShared<Cfg>& sh, uint32_t full_count) {
  for (int s = 0; s < Cfg::kStages; ++s) {
    mbar_init(&sh.k_full[s], full_count);
    mbar_init(&sh.k_empty[s], 1);
    mbar_init(&sh.v_full[s], full_count);
    mbar_init(&sh.v_empty[s], 1);
  }
  for (int s = 0; s < 2; ++s) {
    mbar_init(&sh.meta_full[s], full_count);
    mbar_init(&sh.meta_free[s], Cfg::kRowsWarps);
    mbar_init(&sh.vmeta_full[s], full_count);
    mbar_init(&sh.vmeta_free[s], Cfg::kRowsWarps);
    mbar_init(&sh.o_full[s], 1);
    mbar_init(&sh.o_free[s], Cfg::kRowsWarps);
    mbar_init(&sh.done[s], 1);
  }
  mbar_init(&sh.q_ready, Cfg::kRowsWarps);
  mbar_init(&sh.s_full, 1);
  mbar_init(&sh.s_free, Cfg::kRowsWarps);
  mbar_init(&sh.p_ready, Cfg::kRowsWarps);
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

// ------------------------------------------------------------ the MMA issuers
// Each a whole warp.  S(j) = Q K(j)^T, chunk after chunk of head_dim, once S(j-1) has
// been read; of each chunk the small cross terms first.
template <class Cfg>
__device__ __forceinline__ void mma_issue_qk(MmaShared<Cfg>& sh, uint8_t* k_ring, int n,
                                             unsigned* err) {
  constexpr uint32_t kIdesc = tc_idesc_f16(kTileRows, kTileKeys);
  constexpr int kSteps = Cfg::kHC / 16;
  const uint32_t one = elect_one();
  const uint32_t base = sw128_lo(smem_addr(k_ring));   // units of 16 bytes
  RingAt<Cfg::kStages> at;
  bool ok = true, there = false;       // there: this chunk's unit has been seen to land
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
  };
  if (n > 0) wait(&sh.q_ready, 0);
  for (int j = 0; j < n && ok; ++j) {
#pragma unroll 1
    for (int c = 0; c < Cfg::kNC; ++c) {
      if (!there && !(Cfg::kWhole && c > 0)) wait(&sh.k_full[at.stage], at.phase);
      if (c == 0 && j > 0) wait(&sh.s_free, static_cast<uint32_t>(j - 1) & 1u);
      tc_fence_after();
      if (!ok) break;
      const uint32_t b = base + static_cast<uint32_t>(at.stage) * (Cfg::kUnit >> 4);
      uint64_t* empty = &sh.k_empty[Cfg::kWhole ? at.stage - c : at.stage];
      at.next();
      const bool next = (!Cfg::kWhole || c == Cfg::kNC - 1) &&
                        mbar_test(&sh.k_full[at.stage], at.phase);
#pragma unroll
      for (int t = 0; t < 3; ++t) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint32_t a = (t == 1 ? kTmQlo : kTmQhi) + static_cast<uint32_t>(c * kSteps + k) * 8u;
          const uint32_t off = (t == 0 ? Cfg::kPart : 0u) + static_cast<uint32_t>(k) * 32u;
          tc_mma_f16_ts(kTmS, a, b + (off >> 4), kIdesc, (c | t | k) != 0 ? 1u : 0u, one);
        }
      }
      if (!Cfg::kWhole || c == Cfg::kNC - 1) tc_commit(empty, one);
      if (c == Cfg::kNC - 1) tc_commit(&sh.s_full, one);
      there = __all_sync(0xFFFFFFFFu, next);
    }
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
  bool ok = true, there = false;       // there: unit and accumulator seen to be ready
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
  };
  for (int j = 0; j < n && ok; ++j) {
#pragma unroll 1
    for (int c = 0; c < Cfg::kNC; ++c) {
      if (!there) {
        if (!(Cfg::kWhole && c > 0)) wait(&sh.v_full[at.stage], at.phase);
        wait(&sh.o_free[buf.stage], buf.phase ^ 1u);   // the first use of each passes
      }
      if (c == 0) wait(&sh.p_ready, static_cast<uint32_t>(j) & 1u);   // the last to come
      tc_fence_after();
      if (!ok) break;
      const uint32_t b = base + static_cast<uint32_t>(at.stage) * (Cfg::kUnit >> 4);
      const uint32_t d = kTmO + static_cast<uint32_t>(buf.stage) * 64u;
      uint64_t* full = &sh.o_full[buf.stage];
      uint64_t* empty = &sh.v_empty[Cfg::kWhole ? at.stage - c : at.stage];
      at.next();
      buf.next();
      const bool next = ((Cfg::kWhole && c < Cfg::kNC - 1) ||
                         mbar_test(&sh.v_full[at.stage], at.phase)) &
                        mbar_test(&sh.o_free[buf.stage], buf.phase ^ 1u);
#pragma unroll
      for (int t = 0; t < 3; ++t) {
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; ++k) {
          const uint32_t a = (t == 1 ? kTmPlo : kTmPhi) + static_cast<uint32_t>(k) * 8u;
          const uint32_t off = (t == 0 ? Cfg::kPart : 0u) + static_cast<uint32_t>(k) * 2048u;
          tc_mma_f16_ts(d, a, b + (off >> 4), kIdesc, (t | k) != 0 ? 1u : 0u, one);
        }
      }
      tc_commit(full, one);
      if (!Cfg::kWhole || c == Cfg::kNC - 1) tc_commit(empty, one);
      there = __all_sync(0xFFFFFFFFu, next);
    }
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

// ------------------------------------------------------------ softmax and output
// kSplit threads share a query row: each has its part of a tile's keys and, of
// each chunk of head_dim, its part of the output columns.
template <class Cfg>
struct RowState {
  float o[Cfg::kNC][Cfg::kOC];
  float m, l;              // of the whole row; l of this thread's keys until the end
  bool any_left_out;
};

// scratch: kScratch bytes that nothing else uses until q_ready, and again from the last
// O_tile on; q: the row's head_dim values, or null (a row of zeros); vis: it sees the keys
// below vis (relative to the first key of tile 0 of the run); all_vis: a bound
// below which every row of the CTA sees every key.  kAhead: S(j+1) is turned into weights
// before O_tile(j) is drained, which hides the softmax behind the MMAs; where the key
// tiles come slower than the MMAs take them it would only hold O_tile(j), and with it
// the V buffer, until K(j+1) is there.
template <class Cfg, bool kCap, bool kAhead>
__device__ __forceinline__ void mma_rows(MmaShared<Cfg>& sh, float* scratch, const float* q, int n, int vis, int all_vis, float scale, float cap,
                                         RowState<Cfg>& st, bool& dead) {
  constexpr int kKeys = Cfg::kKeys, kSplit = Cfg::kSplit;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int quad = warp & 3, part = warp >> 2;
  const int row = 32 * quad + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
  auto row_sync = [&]() { bar_sync(1 + quad, 32 * kSplit); };
  dead = false;
  st.m = -INFINITY;
  st.l = 0.f;
  st.any_left_out = false;
  float qscale;
  // ---- Q: this thread's part of the row, scaled and split into tensor memory.  A lane
  // of its own row would touch 32 lines a load: a warp reads its 32 rows in runs of
  // kQRun columns, several lanes a row, and turns them through its scratch
  {
    constexpr int kQC = Cfg::kHd / kSplit;
    constexpr int kQRun = kQC < 32 ? kQC : 32, kLanes = kQRun / 4, kAt = 32 / kLanes;
    constexpr int kLoads = 32 / kAt, kRuns = kQC / kQRun, kPitch = kQRun + 4;
    float* mine = scratch + warp * 32 * kPitch;
    float4 v[kRuns][kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const float* src = reinterpret_cast<const float*>(__shfl_sync(
          0xFFFFFFFFu, reinterpret_cast<unsigned long long>(q), k * kAt + lane / kLanes));
#pragma unroll
      for (int r = 0; r < kRuns; ++r) {
        v[r][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src)
          v[r][k] = *reinterpret_cast<const float4*>(src + part * kQC + r * kQRun +
                                                     (lane % kLanes) * 4);
      }
    }
    float x[kQC];
    float a = 0.f;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        *reinterpret_cast<float4*>(mine + (k * kAt + lane / kLanes) * kPitch + (lane % kLanes) * 4) =
            v[r][k];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kQRun; i += 4) {
        const float4 y = *reinterpret_cast<const float4*>(mine + lane * kPitch + i);
        float* o = x + r * kQRun + i;
        o[0] = y.x; o[1] = y.y; o[2] = y.z; o[3] = y.w;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (finite_bits(o[c])) a = fmaxf(a, fabsf(o[c]));
      }
    }
    sh.xmax[1][part][row] = a;
    row_sync();
#pragma unroll
    for (int c = 0; c < kSplit; ++c) a = fmaxf(a, sh.xmax[1][c][row]);
    const int e = split_exp(a);
    const float sc = exp2i(e);
    qscale = exp2i(-e);
    constexpr int kStep = kQC < 16 ? kQC : 16;
#pragma unroll
    for (int i = 0; i < kQC; i += kStep) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int c = 0; c < kStep / 2; ++c)
        split_f16x2(x[i + 2 * c] * sc, x[i + 2 * c + 1] * sc, hi[c], lo[c]);
      const uint32_t col = static_cast<uint32_t>((part * kQC + i) / 2);
      if constexpr (kStep == 16) {
        tc_st8(lanes + kTmQhi + col, hi);
        tc_st8(lanes + kTmQlo + col, lo);
      } else {
        tc_st4(lanes + kTmQhi + col, hi[0], hi[1], hi[2], hi[3]);
        tc_st4(lanes + kTmQlo + col, lo[0], lo[1], lo[2], lo[3]);
      }
    }
    tc_wait_st();
    fence_proxy_async_smem();      // the scratch is overwritten by copies next
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_ready);
  }
#pragma unroll
  for (int c = 0; c < Cfg::kNC; ++c)
#pragma unroll
    for (int i = 0; i < Cfg::kOC; ++i) st.o[c][i] = 0.f;
  const float rowf = kCap ? qscale * (scale / cap) : qscale * scale * kLog2e;
  const uint32_t t_o = lanes + kTmO + static_cast<uint32_t>(part * Cfg::kOC);
  float alpha = 1.f, vs = 1.f, alpha_next = 1.f;
  uint32_t hi[kKeys / 2], lo[kKeys / 2];
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
                         mbar_wait(&sh.meta_full[ph], mph) && mbar_wait(&sh.s_full, ph));
    tc_fence_after();
    float x[kKeys];
    {
      uint32_t v[kKeys];
      tc_ld<kKeys>(lanes + kTmS + static_cast<uint32_t>(kKeys * part), v);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_free);
      const float4* ks = reinterpret_cast<const float4*>(sh.meta[ph].kscale + kKeys * part);
#pragma unroll
      for (int i = 0; i < kKeys / 4; ++i) {
        const float4 f = ks[i];
        x[4 * i] = __uint_as_float(v[4 * i]) * (f.x * rowf);
        x[4 * i + 1] = __uint_as_float(v[4 * i + 1]) * (f.y * rowf);
        x[4 * i + 2] = __uint_as_float(v[4 * i + 2]) * (f.z * rowf);
        x[4 * i + 3] = __uint_as_float(v[4 * i + 3]) * (f.w * rowf);
      }
    }
    if constexpr (kCap) tanh_scaled<kKeys>(x, cap * kLog2e);
    if ((j + 1) * kTileKeys > all_vis) {
      const int left = vis - j * kTileKeys - kKeys * part;    // of this thread's keys, how many
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (i >= left) x[i] = -INFINITY;                      // a select: nothing is multiplied
    }
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < kKeys; ++i) mx = fmaxf(mx, x[i]);
    sh.xmax[ph][part][row] = mx;
    row_sync();
    // what was stored came of the scales: they have been read
    if (lane == 0) mbar_arrive(&sh.meta_free[ph]);
#pragma unroll
    for (int c = 0; c < kSplit; ++c) mx = fmaxf(mx, sh.xmax[ph][c][row]);
    const float mn = fmaxf(st.m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    alpha_next = ex2(st.m - base);
    st.m = mn;
    const float sub = base - static_cast<float>(kPShift);
    o_seen = mbar_test(&sh.o_full[buf.stage], buf.phase);   // the chunk drained next
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kKeys / 2; ++i) {
      const float a = ex2(x[2 * i] - sub), b = ex2(x[2 * i + 1] - sub);
      sum[i & 3] += a + b;
      split_f16x2(a, b, hi[i], lo[i]);
    }
    st.l = fmaf(st.l, alpha_next, (sum[0] + sum[1]) + (sum[2] + sum[3]));
  };
  auto store_p = [&](int j) {
    // S of the tile after next, meanwhile
    const uint32_t ph = static_cast<uint32_t>(j + 1) & 1u;
    s_seen = mbar_test(&sh.meta_full[ph], static_cast<uint32_t>((j + 1) >> 1) & 1u) &
             mbar_test(&sh.s_full, ph);
    tc_st<kKeys / 2>(lanes + kTmPhi + static_cast<uint32_t>(kKeys / 2 * part), hi);
    tc_st<kKeys / 2>(lanes + kTmPlo + static_cast<uint32_t>(kKeys / 2 * part), lo);
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.p_ready);
  };
  // one copy of each step: the code of a tile is read anew for every tile, and two
  // copies of it do not stay in the instruction caches
#pragma unroll 1
  for (int j = kAhead ? -1 : 0; j < n; ++j) {
    if constexpr (kAhead) {
      alpha = alpha_next;
      if (j + 1 < n) weights(j + 1);
    } else {
      weights(j);
      alpha = alpha_next;
      store_p(j);
    }
    if (j >= 0) {
      const uint32_t ph = static_cast<uint32_t>(j) & 1u;
      if (!dead)
        dead = !__all_sync(0xFFFFFFFFu,
                           mbar_wait(&sh.vmeta_full[ph], static_cast<uint32_t>(j >> 1) & 1u));
      vs = sh.meta[ph].vscale;
      const bool left = (sh.meta[ph].left_out[0] | sh.meta[ph].left_out[1]) != 0;
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
        float a, b;
        mul2(a, b, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), vs, vs);
        scale_add2(st.o[c][i], st.o[c][i + 1], alpha, a, b);
      }
    }
    }
    if constexpr (kAhead)
      if (j + 1 < n) store_p(j + 1);    // P(j) has been multiplied by now
  }
  // the row's whole sum
  row_sync();
  sh.xmax[0][part][row] = st.l;
  row_sync();
  float l = 0.f;
#pragma unroll
  for (int c = 0; c < kSplit; ++c) l += sh.xmax[0][c][row];
  st.l = l;
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
    for (int i = 0; i < Cfg::kOC; ++i)
      st.o[c][i] = fmaf(p, v[c * Cfg::kHC + part * Cfg::kOC + i], st.o[c][i]);
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
          make_float4(st.o[c][i] * f, st.o[c][i + 1] * f, st.o[c][i + 2] * f, st.o[c][i + 3] * f);
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
      float a, b, c, d;
      mul2(a, b, x[i], x[i + 1], sc, sc);
      mul2(c, d, x[i + 2], x[i + 3], sc, sc);
      uint2 hi, lo;
      split_f16x2(a, b, hi.x, lo.x);
      split_f16x2(c, d, hi.y, lo.y);
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

// 64 keys of one kv head, n of them there (the rest zero), by a CTA of 256
// threads, into dst: the units of K, then those of V, and the meta record.
template <class Cfg>
__device__ __forceinline__ void pack_tile(const float* K, const float* V, int64_t k_stride,
                                          int64_t v_stride, int n, uint8_t* dst, TileMeta* meta) {
  constexpr int kPL = Cfg::kHd / 32, kRows = kTileKeys / 8;
  __shared__ float vmax[kTileKeys];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  float y[kRows][kPL];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + 8 * i;
    float x[kPL];
#pragma unroll
    for (int c = 0; c < kPL; ++c) x[c] = y[i][c] = 0.f;
    if (r < n) {
      load_row<kPL>(K + r * k_stride, lane, x);
      load_row<kPL>(V + r * v_stride, lane, y[i]);
    }
    bool fin;
    const int e = split_exp(row_amax<kPL>(x, fin));
    store_split_row<Cfg>(x, exp2i(e), r, lane, dst);
    const float b = row_amax<kPL>(y[i], fin);
    if (lane == 0) {
      meta->kscale[r] = exp2i(-e);
      vmax[r] = fin ? b : INFINITY;
    }
  }
  __syncthreads();
  // the smallest non-zero row maximum; rows above 2^16 times it stay out
  const float a = vmax[lane], b = vmax[lane + 32];
  float lo = fminf(a > 0.f ? a : INFINITY, b > 0.f ? b : INFINITY);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
  const float top = lo * 65536.0f;                 // infinity: only what is not finite
  const bool out_a = !(a <= top) || a == INFINITY, out_b = !(b <= top) || b == INFINITY;
  const uint32_t ma = __ballot_sync(0xFFFFFFFFu, out_a), mb = __ballot_sync(0xFFFFFFFFu, out_b);
  const int e = split_exp(warp_max(fmaxf(out_a ? 0.f : a, out_b ? 0.f : b)));
  if (threadIdx.x == 0) {
    meta->vscale = exp2i(-e);
    meta->left_out[0] = ma;
    meta->left_out[1] = mb;
    meta->pad = 0;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + 8 * i;
    const bool out = ((r < 32 ? ma : mb) >> (r & 31)) & 1u;
#pragma unroll
    for (int c = 0; c < kPL; ++c) y[i][c] = out ? 0.f : y[i][c];
    store_split_row<Cfg>(y[i], exp2i(e), r, lane, dst + Cfg::kHalfTile);
  }
}

}  // namespace qws
