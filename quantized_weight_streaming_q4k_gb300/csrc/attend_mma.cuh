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
// Q hi / lo and P hi / lo are A operands in tensor memory, K and V^T come
// through a shared-memory ring in the 128-byte-swizzled K-major image.  O_tile is
// NOT accumulated in tensor memory: the tensor cores' f32 accumulation does
// not round to nearest, and its bias grows with the number of steps.  Each
// tile's O_tile (12 accumulation steps) is added to f32 registers with the
// softmax's rescaling, one multiplication and one fma a value, which the three
// products per value leave time for (256 of about 3000 cycles a tile at head_dim
// 256).  This also spares the correction pass over tensor memory.
//
// TMEM columns (all 512 are allocated, so they start at 0): Q hi 0.., Q lo 128.., S 256.., P hi 320.., P lo 352..,
// O_tile 384.. (128 columns: at head_dim 256 the two halves of O_tile take turns).
//
// Roles (12 warps, two idle): warps 0..7 softmax and output (thread = row 32 (w % 4) + lane,
// w / 4 = which half of the tile's keys and of the output columns), warp 8 loads, warp 9
// issues the MMAs in the order QK_a(j+1), PV_0(j), QK_b(j+1), PV_1(j), (a, b and
// 0, 1: halves of head_dim), so that the softmax of a tile and both drains of
// O_tile each have a segment of other MMAs to hide behind.
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
constexpr int kConsumers = 256;
constexpr int kMmaThreads = kConsumers + 128;   // whole warpgroups, for the register split
// Registers a thread: the launch gives 168 x 384 = 64512; the last warpgroup keeps 56, the
// softmax warpgroups take 224 (2 x 128 x 224 + 128 x 56 = 64512, no more than launched).
__device__ __forceinline__ void regs_few() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }
__device__ __forceinline__ void regs_many() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
}
constexpr int kPShift = 14;            // weights are 2^14 exp2(s - max)

// what a key tile carries beside its values
struct __align__(16) TileMeta {
  float kscale[kTileKeys];   // 2^-e of each key row
  float vscale;              // 2^-e of the tile's values
  uint32_t left_out[2];      // keys whose values are not in the tile
  uint32_t pad;
};
static_assert(sizeof(TileMeta) == 272, "copied in 16-byte units");

template <int kHdT>
struct MmaCfg {
  static constexpr int kHd = kHdT;
  static constexpr int kNH = kHd > 128 ? 2 : 1;         // halves of head_dim
  static constexpr int kHC = kHd / kNH;                 // columns of a half
  static constexpr int kOC = kHC / 2;                   // of these, a thread's
  static constexpr int kChunks = (kHC + 63) / 64;       // 64-column runs of a K unit
  static constexpr int kQkSteps = kHC / 16;
  static constexpr uint32_t kKPart = kChunks * 8192u;   // hi or lo of a K unit
  static constexpr uint32_t kVPart = kHC * 128u;        // hi or lo of a V unit
  static constexpr uint32_t kKUnit = 2 * kKPart, kVUnit = 2 * kVPart;
  static constexpr uint32_t kTile = kNH * (kKUnit + kVUnit);   // a packed key tile
  static constexpr uint32_t kStage = kKUnit > kVUnit ? kKUnit : kVUnit;
  static constexpr int kStages = 6;
};

constexpr uint32_t kTmQhi = 0, kTmQlo = 128, kTmS = 256, kTmPhi = 320, kTmPlo = 352, kTmO = 384;

// barriers and small exchanges of one CTA
template <int kStages>
struct MmaShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t meta_full[2], meta_free[2];
  uint64_t q_ready, s_full, s_free, p_ready, o_full, o_free, done;
  uint32_t tmem;
  uint32_t pad;
  float xmax[2][2][kTileRows];
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

// The power of two 2^e that puts a into [2^14, 2^15) (1 for zero), e in +-126.
__device__ __forceinline__ int split_exp(float a) {
  if (!(a > 0.f)) return 0;
  int E;
  frexpf(a, &E);
  return min(126, max(-126, 15 - E));
}
__device__ __forceinline__ bool finite_bits(float x) {
  return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
}

template <int kStages>
__device__ __forceinline__ void mma_init_barriers(MmaShared<kStages>& sh, uint32_t full_count) {
  for (int s = 0; s < kStages; ++s) {
    mbar_init(&sh.full[s], full_count);
    mbar_init(&sh.empty[s], 1);
  }
  for (int s = 0; s < 2; ++s) {
    mbar_init(&sh.meta_full[s], 1);
    mbar_init(&sh.meta_free[s], kConsumers / 32);
  }
  mbar_init(&sh.q_ready, kConsumers / 32);
  mbar_init(&sh.s_full, 1);
  mbar_init(&sh.s_free, kConsumers / 32);
  mbar_init(&sh.p_ready, kConsumers / 32);
  mbar_init(&sh.o_full, 1);
  mbar_init(&sh.o_free, kConsumers / 32);
  mbar_init(&sh.done, 1);
  fence_barrier_init();
}

// ------------------------------------------------------------ the MMA issuer
// A whole warp.  Units arrive in the order they are used: K halves of tile 0, then
// for every tile j and half h: K half h of tile j + 1, V half h of tile j.
template <class Cfg>
__device__ __forceinline__ void mma_issue(MmaShared<Cfg::kStages>& sh, uint8_t* stages, int n,
                                          unsigned* err) {
  constexpr uint32_t kIdescQk = tc_idesc_f16(kTileRows, kTileKeys);
  constexpr uint32_t kIdescPv = tc_idesc_f16(kTileRows, Cfg::kHC);
  const uint32_t one = elect_one();
  const uint32_t base = sw128_lo(smem_addr(stages));   // units of 16 bytes
  int unit = 0, stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
  };
  auto next = [&]() {
    ++unit;
    if (++stage == Cfg::kStages) {
      stage = 0;
      phase ^= 1u;
    }
  };
  auto qk = [&](int j, int h) {
    if (h == 0 && j > 0) wait(&sh.s_free, static_cast<uint32_t>(j - 1) & 1u);
    wait(&sh.full[stage], phase);
    tc_fence_after();
    if (!ok) return;
    const uint32_t b = base + static_cast<uint32_t>(stage) * (Cfg::kStage >> 4);
    // the small cross terms first: what is rounded off them is smaller still
#pragma unroll
    for (int t = 0; t < 3; ++t) {
#pragma unroll
      for (int k = 0; k < Cfg::kQkSteps; ++k) {
        const uint32_t a =
            (t == 1 ? kTmQlo : kTmQhi) + static_cast<uint32_t>(h * Cfg::kQkSteps + k) * 8u;
        const uint32_t off = (t == 0 ? Cfg::kKPart : 0u) + static_cast<uint32_t>(k / 4) * 8192u +
                             static_cast<uint32_t>(k % 4) * 32u;
        tc_mma_f16_ts(kTmS, a, b + (off >> 4), kIdescQk, (h | t | k) != 0 ? 1u : 0u, one);
      }
    }
    tc_commit(&sh.empty[stage], one);
    if (h == Cfg::kNH - 1) tc_commit(&sh.s_full, one);
    next();
  };
  auto pv = [&](int j, int h) {
    const int use = j * Cfg::kNH + h;
    if (h == 0) wait(&sh.p_ready, static_cast<uint32_t>(j) & 1u);
    if (use > 0) wait(&sh.o_free, static_cast<uint32_t>(use - 1) & 1u);
    wait(&sh.full[stage], phase);
    tc_fence_after();
    if (!ok) return;
    const uint32_t b = base + static_cast<uint32_t>(stage) * (Cfg::kStage >> 4);
#pragma unroll
    for (int t = 0; t < 3; ++t) {
#pragma unroll
      for (int k = 0; k < kTileKeys / 16; ++k) {
        const uint32_t a = (t == 1 ? kTmPlo : kTmPhi) + static_cast<uint32_t>(k) * 8u;
        const uint32_t off = (t == 0 ? Cfg::kVPart : 0u) + static_cast<uint32_t>(k) * 32u;
        tc_mma_f16_ts(kTmO, a, b + (off >> 4), kIdescPv, (t | k) != 0 ? 1u : 0u, one);
      }
    }
    tc_commit(&sh.empty[stage], one);
    tc_commit(&sh.o_full, one);
    next();
  };
  if (n > 0) {
    wait(&sh.q_ready, 0);
#pragma unroll
    for (int h = 0; h < Cfg::kNH; ++h) qk(0, h);
  }
  for (int j = 0; j < n && ok; ++j) {
#pragma unroll
    for (int h = 0; h < Cfg::kNH; ++h) {
      if (j + 1 < n) qk(j + 1, h);
      pv(j, h);
    }
  }
  if (!ok && one) atomicOr(err, kErrAttMma);
  tc_commit(&sh.done, one);     // arrives when every MMA above has completed
}

// ------------------------------------------------------------ softmax and output
// One query row per pair of threads.
template <class Cfg>
struct RowState {
  float o[Cfg::kNH][Cfg::kOC];
  float m, l;              // of the whole row; l of this thread's keys until finish()
  float qscale;            // 2^-e of the row
  bool any_left_out;
};

template <class Cfg>
__device__ __forceinline__ void drain_o(MmaShared<Cfg::kStages>& sh, uint32_t t_o, int use,
                                        float alpha, float vs, float (&o)[Cfg::kOC],
                                        bool& dead) {
  if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_wait(&sh.o_full, static_cast<uint32_t>(use) & 1u));
  tc_fence_after();
#pragma unroll
  for (int c = 0; c < Cfg::kOC; c += 16) {
    uint32_t v[16];
    tc_ld16(t_o + static_cast<uint32_t>(c), v);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float a, b;
      mul2(a, b, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), vs, vs);
      scale_add2(o[c + i], o[c + i + 1], alpha, a, b);
    }
  }
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.o_free);
}

// q: the row's head_dim values, or null (a row of zeros); vis: it sees the keys
// below vis (relative to the first key of tile 0 of the run); all_vis: a bound
// below which every row of the CTA sees every key.
template <class Cfg>
__device__ __forceinline__ void mma_rows(MmaShared<Cfg::kStages>& sh, const float* q, int n, int vis, int all_vis, float scale,
                                         float cap, RowState<Cfg>& st, bool& dead) {
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int quad = warp & 3, half = warp >> 2;
  const int row = 32 * quad + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
  dead = false;
  st.m = -INFINITY;
  st.l = 0.f;
  st.any_left_out = false;
#pragma unroll
  for (int h = 0; h < Cfg::kNH; ++h)
#pragma unroll
    for (int i = 0; i < Cfg::kOC; ++i) st.o[h][i] = 0.f;
  // ---- Q: this thread's half of the row, scaled and split into tensor memory
  {
    constexpr int kQC = Cfg::kHd / 2;
    float x[kQC];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kQC; i += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q) v = *reinterpret_cast<const float4*>(q + half * kQC + i);
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (finite_bits(x[i + c])) a = fmaxf(a, fabsf(x[i + c]));
    }
    sh.xmax[1][half][row] = a;
    bar_sync(1 + quad, 64);
    a = fmaxf(a, sh.xmax[1][half ^ 1][row]);
    const int e = split_exp(a);
    const float sc = exp2i(e);
    st.qscale = exp2i(-e);
#pragma unroll
    for (int i = 0; i < kQC; i += 16) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) split_f16x2(x[i + 2 * c] * sc, x[i + 2 * c + 1] * sc, hi[c], lo[c]);
      const uint32_t col = static_cast<uint32_t>((half * kQC + i) / 2);
      tc_st8(lanes + kTmQhi + col, hi);
      tc_st8(lanes + kTmQlo + col, lo);
    }
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_ready);
  }
  const float rowf = st.qscale * scale * (cap > 0.f ? 1.f : kLog2e);
  const uint32_t t_o = lanes + kTmO + static_cast<uint32_t>(half * Cfg::kOC);
  float alpha_prev = 1.f, vs_prev = 1.f;
  for (int j = 0; j < n; ++j) {
    const uint32_t ph = static_cast<uint32_t>(j) & 1u;
    const uint32_t mph = static_cast<uint32_t>(j >> 1) & 1u;
    if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_wait(&sh.meta_full[ph], mph));
    if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_wait(&sh.s_full, ph));
    tc_fence_after();
    float x[32];
    {
      uint32_t v[32];
      tc_ld32(lanes + kTmS + static_cast<uint32_t>(32 * half), v);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_free);
      const float4* ks = reinterpret_cast<const float4*>(sh.meta[ph].kscale + 32 * half);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = ks[i];
        x[4 * i] = __uint_as_float(v[4 * i]) * (f.x * rowf);
        x[4 * i + 1] = __uint_as_float(v[4 * i + 1]) * (f.y * rowf);
        x[4 * i + 2] = __uint_as_float(v[4 * i + 2]) * (f.z * rowf);
        x[4 * i + 3] = __uint_as_float(v[4 * i + 3]) * (f.w * rowf);
      }
    }
    const float vs = sh.meta[ph].vscale;
    st.any_left_out = st.any_left_out || (sh.meta[ph].left_out[0] | sh.meta[ph].left_out[1]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.meta_free[ph]);
    if (cap > 0.f) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = cap * tanhf(x[i] / cap) * kLog2e;
    }
    if ((j + 1) * kTileKeys > all_vis) {
      const int left = vis - j * kTileKeys - 32 * half;     // of this thread's keys, how many
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i >= left) x[i] = -INFINITY;                     // a select: nothing is multiplied
    }
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) mx = fmaxf(mx, x[i]);
    sh.xmax[ph][half][row] = mx;
    bar_sync(1 + quad, 64);
    mx = fmaxf(mx, sh.xmax[ph][half ^ 1][row]);
    const float mn = fmaxf(st.m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float alpha = ex2(st.m - base);
    st.m = mn;
    const float sub = base - static_cast<float>(kPShift);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = ex2(x[2 * i] - sub), b = ex2(x[2 * i + 1] - sub);
      sum[i & 3] += a + b;
      split_f16x2(a, b, hi[i], lo[i]);
    }
    st.l = fmaf(st.l, alpha, (sum[0] + sum[1]) + (sum[2] + sum[3]));
    // the last half of the tile before: after it P may be overwritten
    if (j > 0)
      drain_o<Cfg>(sh, t_o, j * Cfg::kNH - 1, alpha_prev, vs_prev, st.o[Cfg::kNH - 1], dead);
    tc_st16(lanes + kTmPhi + static_cast<uint32_t>(16 * half), hi);
    tc_st16(lanes + kTmPlo + static_cast<uint32_t>(16 * half), lo);
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.p_ready);
    if constexpr (Cfg::kNH == 2)
      drain_o<Cfg>(sh, t_o, 2 * j, alpha, vs, st.o[0], dead);
    alpha_prev = alpha;
    vs_prev = vs;
  }
  if (n > 0)
    drain_o<Cfg>(sh, t_o, n * Cfg::kNH - 1, alpha_prev, vs_prev, st.o[Cfg::kNH - 1], dead);
  // the row's whole sum
  bar_sync(1 + quad, 64);
  sh.xmax[0][half][row] = st.l;
  bar_sync(1 + quad, 64);
  st.l += sh.xmax[0][half ^ 1][row];
}

// A key left out of its tile (see the head of this file): its weight from the
// row's final maximum, and its values, in f32.
template <class Cfg>
__device__ __forceinline__ void add_left_out(RowState<Cfg>& st, const float* q, const float* k,
                                          const float* v, int half, float scale, float cap) {
  float s = 0.f;
  for (int i = 0; i < Cfg::kHd; i += 4) {
    const float4 a = *reinterpret_cast<const float4*>(q + i);
    const float4 b = *reinterpret_cast<const float4*>(k + i);
    s = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
  }
  const float base = st.m == -INFINITY ? 0.f : st.m;
  const float p = ex2(soft_cap(s * scale, cap) * kLog2e - (base - static_cast<float>(kPShift)));
#pragma unroll
  for (int h = 0; h < Cfg::kNH; ++h)
#pragma unroll
    for (int i = 0; i < Cfg::kOC; ++i)
      st.o[h][i] = fmaf(p, v[h * Cfg::kHC + half * Cfg::kOC + i], st.o[h][i]);
}

// this thread's columns of a row: f * o
template <class Cfg>
__device__ __forceinline__ void store_columns(const RowState<Cfg>& st, float* dst, int half,
                                              float f) {
#pragma unroll
  for (int h = 0; h < Cfg::kNH; ++h)
#pragma unroll
    for (int i = 0; i < Cfg::kOC; i += 4)
      *reinterpret_cast<float4*>(dst + h * Cfg::kHC + half * Cfg::kOC + i) =
          make_float4(st.o[h][i] * f, st.o[h][i + 1] * f, st.o[h][i + 2] * f, st.o[h][i + 3] * f);
}

// ------------------------------------------------------------ packing a key tile
// 64 keys of one kv head, n of them there (the rest zero), by a CTA of 256
// threads: K rows as units of [hi, lo][64-column run] x 64 rows of 128 bytes, V
// transposed as units of [hi, lo] x head_dim rows of 64 keys, into dst (the
// order K half 0, K half 1, V half 0, V half 1), and the meta record.
// smem: kTileKeys * (hd + 1) floats.
template <class Cfg>
__device__ __forceinline__ void pack_tile(const float* K, const float* V, int64_t k_stride,
                                          int64_t v_stride, int n, uint8_t* dst, TileMeta* meta,
                                          float* vt) {
  constexpr int kHd = Cfg::kHd, kPL = kHd / 32, kPitch = kHd + 1;
  __shared__ float vmax[kTileKeys];
  __shared__ uint32_t bad[2];
  __shared__ float vsc;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  for (int r = warp; r < kTileKeys; r += 8) {
    float x[kPL], y[kPL];
#pragma unroll
    for (int i = 0; i < kPL; ++i) x[i] = y[i] = 0.f;
    if (r < n) {
      load_row<kPL>(K + r * k_stride, lane, x);
      load_row<kPL>(V + r * v_stride, lane, y);
    }
    float a = 0.f, b = 0.f;
    bool fin = true;
#pragma unroll
    for (int i = 0; i < kPL; ++i) {
      if (finite_bits(x[i])) a = fmaxf(a, fabsf(x[i]));
      fin = fin && finite_bits(y[i]);
      b = fmaxf(b, fabsf(y[i]));
    }
    a = warp_max(a);
    b = warp_max(b);
    fin = __all_sync(0xFFFFFFFFu, fin);
    const int e = split_exp(a);
    const float sc = exp2i(e);
    if (lane == 0) {
      meta->kscale[r] = exp2i(-e);
      vmax[r] = fin ? b : INFINITY;
    }
    // K: neighbours in pairs (one value at head_dim 32 and 64: exchange below)
    if constexpr (kPL >= 2) {
#pragma unroll
      for (int i = 0; i < kPL; i += (kPL >= 4 ? 4 : 2)) {
        const int c = lane_col<kPL>(lane, i);
        const int h = c / Cfg::kHC, ch = c - h * Cfg::kHC;
        uint8_t* u = dst + h * Cfg::kKUnit + (ch / 64) * 8192;
        const uint32_t off = sw128_off(static_cast<uint32_t>(r), static_cast<uint32_t>(ch % 64) / 8u) +
                             static_cast<uint32_t>(ch % 8) * 2u;
        uint32_t h0, l0;
        split_f16x2(x[i] * sc, x[i + 1] * sc, h0, l0);
        if constexpr (kPL >= 4) {
          uint32_t h1, l1;
          split_f16x2(x[i + 2] * sc, x[i + 3] * sc, h1, l1);
          *reinterpret_cast<uint2*>(u + off) = make_uint2(h0, h1);
          *reinterpret_cast<uint2*>(u + Cfg::kKPart + off) = make_uint2(l0, l1);
        } else {
          *reinterpret_cast<uint32_t*>(u + off) = h0;
          *reinterpret_cast<uint32_t*>(u + Cfg::kKPart + off) = l0;
        }
      }
    } else {
      const float other = __shfl_xor_sync(0xFFFFFFFFu, x[0], 1);
      if (!(lane & 1)) {
        uint32_t h0, l0;
        split_f16x2(x[0] * sc, other * sc, h0, l0);
        const uint32_t off = sw128_off(static_cast<uint32_t>(r), static_cast<uint32_t>(lane) / 8u) +
                             static_cast<uint32_t>(lane % 8) * 2u;
        *reinterpret_cast<uint32_t*>(dst + off) = h0;
        *reinterpret_cast<uint32_t*>(dst + Cfg::kKPart + off) = l0;
      }
    }
#pragma unroll
    for (int i = 0; i < kPL; ++i) vt[r * kPitch + lane_col<kPL>(lane, i)] = y[i];
  }
  __syncthreads();
  if (warp == 0) {
    // the smallest finite non-zero row maximum; rows above 2^16 times it stay out
    const float a = vmax[lane], b = vmax[lane + 32];
    float lo = fminf(a > 0.f ? a : INFINITY, b > 0.f ? b : INFINITY);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    const float top = lo * 65536.0f;                 // infinity: only what is not finite
    const bool out_a = !(a <= top) || a == INFINITY, out_b = !(b <= top) || b == INFINITY;
    const uint32_t ma = __ballot_sync(0xFFFFFFFFu, out_a), mb = __ballot_sync(0xFFFFFFFFu, out_b);
    const float big = warp_max(fmaxf(out_a ? 0.f : a, out_b ? 0.f : b));
    if (lane == 0) {
      const int e = split_exp(big);
      bad[0] = ma;
      bad[1] = mb;
      vsc = exp2i(e);
      meta->vscale = exp2i(-e);
      meta->left_out[0] = ma;
      meta->left_out[1] = mb;
      meta->pad = 0;
    }
  }
  __syncthreads();
  const float sc = vsc;
  // a warp: 4 channels x 8 groups of 8 keys, each 16 bytes of hi and of lo
  for (int d0 = warp * 4; d0 < kHd; d0 += 32) {
    const int d = d0 + (lane >> 3), kg = lane & 7;
    const uint32_t out8 = (bad[kg >> 2] >> (8 * (kg & 3))) & 255u;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = (out8 >> i) & 1u ? 0.f : vt[(kg * 8 + i) * kPitch + d] * sc;
    uint4 hi, lo;
    split_f16x2(y[0], y[1], hi.x, lo.x);
    split_f16x2(y[2], y[3], hi.y, lo.y);
    split_f16x2(y[4], y[5], hi.z, lo.z);
    split_f16x2(y[6], y[7], hi.w, lo.w);
    const int h = d / Cfg::kHC, dh = d - h * Cfg::kHC;
    uint8_t* u = dst + Cfg::kNH * Cfg::kKUnit + h * Cfg::kVUnit;
    const uint32_t off = sw128_off(static_cast<uint32_t>(dh), static_cast<uint32_t>(kg));
    *reinterpret_cast<uint4*>(u + off) = hi;
    *reinterpret_cast<uint4*>(u + Cfg::kVPart + off) = lo;
  }
}

}  // namespace qws
