// paged_attention.cu -- attention of a batch's new tokens, each over the pages of its own
// sequence:  out = sum_j softmax_j(cap(scale q . k_j)) v_j,  j = 0 .. position of the token.
//
// Bound by the pages' bytes, which are read once: 18/32 (34/32) byte a value.  A kv head
// has one to four query rows, so a value that has been unpacked is worth two to eight
// operations, and unpacking is what the instructions go to.  The matrix instruction
// (m16n8k16) takes codes as exact f16 numbers, two to a register: masked in place in a
// half-word below the exponent of 1024 and centred by one subtraction, nine instructions for
// eight.  Its eight columns hold four rows' queries (or weights) as two f16 parts each.
// Per slab of 16 positions of a kv head, all in one warp's registers:
//   scores   K codes (16 keys, or 8 keys of two blocks) x q, summed per block of 32
//            dimensions, then times the key's f16 scale of that block in f32;
//   softmax  in f32; a weight times the value's scale is split in two f16 parts;
//   output   V codes^T x these, summed over the 16 keys, added up in f32.
// The tensor cores cut each sum towards zero, so sums there stay that short.  (Codes as
// subnormal numbers, masked in place and nothing else, need a subtraction less, but they are not
// normalised before products are aligned: errors four times those of plain f32, now the same.)
//
// q and weights times scales are f32 as hi + lo: within 2^-23 of themselves or, where lo is
// subnormal, 2^-25: at least 2^-37 of the row's largest such product (2^-38 of its largest
// query), which is brought to 2^12 and may grow to 2^15.  Weights are 2^(s - m), m within 2 of the scores' maximum so far.  For weight *
// scale to fit f16 they are multiplied by 2^k, k whole, such that s + log2(bound on the value's
// scales) - m + k <= 15 for all keys; both move rarely, and a vote decides whether they do.
// (Weights relative to one number that takes both in are less exact: s minus it is some 10.)
//
// The units of work, slabs of all (kv head, token) items one after the other, are dealt
// evenly to the CTAs of the grid, and a CTA's to its warps: a run of units each, whatever
// sequences they belong to.  A warp streams its units through a ring of its own (one bulk copy a slab), without
// a barrier with other warps.  All of that is computed in the kernel from the positions, so a
// captured launch follows them.  Items that a warp has whole are stored; the parts of the
// others meet in shared memory after the warps' last slabs, and what CTAs share is joined from
// the workspace by a second kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "attend_rows.cuh"
#include "paged.cuh"

namespace qws {

__device__ unsigned g_err_pattn;

constexpr int kPaMaxRows = 1024;             // tokens of a launch
constexpr size_t kPaSmem = 220 * 1024;

struct PagedAttnParams {
  PagedView c;
  qws_heads q, out;
  const int64_t *seqs, *positions;
  int n_tokens, group, together;             // together: tokens of a sequence in an item
  float scale, cap;
  float* parts;                              // [grid][2][rows][hd], then m and l [grid][2][rows][2]
  int4* joins;                               // [grid]: token, kv head | rows << 16, last CTA, -
};

// kRows 2: with two rows, the eight columns hold two blocks of 32 dimensions side by side
// (rows 0..7 of the instruction's 16 are one block's, 8..15 the other's): half the registers
// for queries and half the splitting of weights.
template <int kHd, int kFmt, int kRows>
struct PaCfg {
  using L = Slab<kHd, kFmt>;
  // As many as registers and the ring leave room for, two slabs a warp at least; measured with 64
  // sequences, 4 bits in two rows, in four, 8 bits in two, in four.  Heads of 256, 4096 positions:
  // 65 us with 16 (67 with 12, 72 with 14, which has no deeper ring), 69 with 12 (75 with 16, which
  // spills), 81 and 82 with 8 (84 and 95 with 10).  Heads of 128: 67 with 20 (71 with 16), 74 with 16
  // (the same with 20), 81 and 81 with 16 (84 and 82 with 20).  Heads of 64, 8192 positions: 92,
  // 96, 96, 97 with 24 (95, 99, 99, 100 with 20; 92, 97, 97, 101 with 28).
  static constexpr bool kLight = kFmt == QWS_Q4_0 && kRows == 2;
  static constexpr int kWarps = kHd == 256   ? kFmt != QWS_Q4_0 ? 8 : kLight ? 16 : 12
                                : kHd == 128 ? kLight ? 20 : 16
                                             : 24;
  static constexpr int kThreads = kWarps * 32;
  // a warp's part of an item begun before its units; that of its last item goes into its ring
  static constexpr size_t kJoin = sizeof(float) * kWarps * kRows * kHd;
  static constexpr size_t kPrefix = sizeof(unsigned long long) * (kPaMaxRows + 2);
  static constexpr size_t kTokens = 2 * sizeof(int) * kPaMaxRows;
  static constexpr int kFit = static_cast<int>((kPaSmem - kJoin - kPrefix - kTokens - 1024) /
                                               (kWarps * (L::kBytes + 16)));
  static constexpr int kDepth = kFit < 8 ? kFit : 8;
  static constexpr size_t kRing = static_cast<size_t>(kWarps) * kDepth * L::kBytes;
  static_assert(kDepth * L::kBytes >= static_cast<int>(sizeof(float)) * kRows * kHd, "ring");
  static constexpr size_t kSmem = kRing + kJoin + kPrefix + kTokens + kWarps * kDepth * 16;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same with sums that begin at zero (no registers have to be set to it)
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// step `i` of a sum
__device__ __forceinline__ void mma_step(int i, float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (i == 0) mma_f16_first(d, a0, a1, a2, a3, b0, b1);
  else mma_f16(d, a0, a1, a2, a3, b0, b1);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// Of two values rounded to f16 (keep 0), or of what that leaves of them (keep -1).
__device__ __forceinline__ uint32_t split_part(float a, float b, float keep) {
  const float2 f = __half22float2(__floats2half2_rn(a, b));
  fma2(a, b, f.x, f.y, keep, keep);
  return h2_bits(__floats2half2_rn(a, b));
}

// one lane's chunk of half a slab's codes
template <class L>
__device__ __forceinline__ void load_chunk(const uint8_t* codes, int half, int lane,
                                           uint32_t (&w)[L::kChunk / 4]) {
#pragma unroll
  for (int u = 0; u < L::kChunk / L::kUnit; ++u) {
    const uint8_t* p = codes + L::at(half, lane, u * L::kUnit);
    if constexpr (L::kUnit == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[4 * u] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
    } else if constexpr (L::kUnit == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
}

// the f16 scales of one row, two to a word
template <int kBlocks>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&w)[(kBlocks + 1) / 2]) {
  if constexpr (kBlocks == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (kBlocks == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else if constexpr (kBlocks == 2) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}

// Two codes of a word, masked in place, as f16: below the exponent of 1024 they are 1024 + code
// (bits 0..) or 1024 + 16 code (bits 4..7), and the difference to the same form of the code of
// zero is exact.
template <uint32_t kMask, uint32_t kZero>
__device__ __forceinline__ uint32_t centred(uint32_t x) {
  uint32_t y;      // (x & mask) | exponent, one instruction (two of them from plain C)
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "n"(kMask), "r"(0x64006400u));
  return h2_bits(__hsub2(bits_h2(y), bits_h2(kZero)));
}

// A warp's place among the items: the token that one begins with, its kv head, the slabs it has
struct PaItem {
  int t, head, units;
};

// a warp's part of an item: of its first one (slot 0, begun earlier) or its last (slot 1)
struct PaPart {
  int t, head, rows, ends;         // t -1: none; ends: the item ends with this part
};

template <int kHd, int kFmt, int kRows>
__global__ void __launch_bounds__(PaCfg<kHd, kFmt, kRows>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ PagedAttnParams p) {
  using C = PaCfg<kHd, kFmt, kRows>;
  using L = Slab<kHd, kFmt>;
  constexpr int kBlocks = L::kBlocks, kWords = L::kChunk / 4;
  constexpr bool kTwo = kRows == 2;
  constexpr int kSteps = kTwo ? kBlocks / 2 : kBlocks;     // B operands of a pass over head_dim
  constexpr int kWarps = C::kWarps, kDepth = C::kDepth;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  float* join = reinterpret_cast<float*>(smem + C::kRing);            // [warp][row][hd]
  auto* prefix = reinterpret_cast<unsigned long long*>(smem + C::kRing + C::kJoin);
  int* tok_seq = reinterpret_cast<int*>(smem + C::kRing + C::kJoin + C::kPrefix);
  int* tok_pos = tok_seq + kPaMaxRows;
  uint64_t* full = reinterpret_cast<uint64_t*>(tok_pos + kPaMaxRows);
  int* there = reinterpret_cast<int*>(full + kWarps * kDepth);        // the stage holds a page
  __shared__ unsigned long long scan[32];
  __shared__ int starts[32];
  __shared__ PaPart parts[2][kWarps];
  __shared__ float stat[2][kWarps][kRows][2];                         // m, l

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  for (int i = tid; i < kWarps * kDepth; i += C::kThreads) mbar_init(full + i, 1);
  fence_barrier_init();
  pdl_launch_dependents();
  pdl_wait();

  // ---- the tokens (sequence -1: padding), and the items: runs of up to `together` tokens of
  // one sequence.  A thread takes `per` neighbours; first where runs begin, then the slabs of
  // each item, summed up.
  const int T = p.n_tokens, per = (T + C::kThreads - 1) / C::kThreads;
  for (int t = tid; t < T; t += C::kThreads) {
    const int64_t s = __ldg(p.seqs + t), n = __ldg(p.positions + t);
    const TokenKind kind = token_kind(p.c, s, n);
    tok_seq[t] = kind == kTokenFine ? static_cast<int>(s) : -1;
    tok_pos[t] = kind == kTokenFine ? static_cast<int>(n) : -1;
    if (kind == kTokenOutside && blockIdx.x == 0) atomicOr(&g_err_pattn, kErrPage);
  }
  if (tid < 2 * kWarps) parts[tid / kWarps][tid % kWarps].t = -1;
  __syncthreads();
  const int t0 = min(T, tid * per), t1 = min(T, t0 + per);
  const auto begins = [&](int t) {
    return t == 0 || tok_seq[t] < 0 || tok_seq[t] != tok_seq[t - 1];
  };
  int at = -1;                               // the beginning of the run that reaches t0
  if (p.together > 1) {
    int last = -1;
    for (int t = t0; t < t1; ++t)
      if (begins(t)) last = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, last, o);
      if (lane >= o) last = max(last, y);
    }
    if (lane == 31) starts[warp] = last;
    at = __shfl_up_sync(0xFFFFFFFFu, last, 1);
    __syncthreads();
    if (lane == 0) at = -1;
    for (int w = 0; w < warp; ++w) at = max(at, starts[w]);
  }
  unsigned long long mine = 0;
  for (int t = t0; t < t1; ++t) {
    unsigned u = 0;                          // 0: not the first of its item
    if (p.together == 1 || begins(t)) at = t;
    if ((t - at) % p.together == 0) {
      int most = tok_pos[t];
      for (int i = t + 1; i < min(T, t + p.together) && !begins(i); ++i) most = max(most, tok_pos[i]);
      u = static_cast<unsigned>(max(most, 0)) / 16 + 1;
    }
    prefix[t] = u;
    mine += u;
  }
  unsigned long long sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) scan[warp] = sum;
  __syncthreads();
  unsigned long long total = 0, base = sum - mine;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += scan[w];
    total += scan[w];
  }
  for (int t = t0; t < t1; ++t) {
    const unsigned long long u = prefix[t];
    prefix[t] = base;
    base += u;
  }
  if (tid == 0) prefix[T] = total;
  __syncthreads();

  // ---- this warp's units
  const unsigned long long all = total * p.c.n_kv;
  const unsigned long long share = max((all + gridDim.x - 1) / gridDim.x, 4ull);   // a CTA's
  // (at least four: 1.2 us less than with one for a sequence of 777 positions, 98 units, which takes 8.3)
  const unsigned long long warp_share = (share + kWarps - 1) / kWarps;
  const unsigned long long cta_end = min(all, share * (blockIdx.x + 1ull));
  const unsigned long long begin = min(cta_end, share * blockIdx.x + warp_share * warp);
  const unsigned long long end = min(cta_end, begin + warp_share);
  PaItem first{0, 0, 1};
  int first_s = 0;                           // its first slab of the first item
  if (begin < end) {
    first.head = static_cast<int>(begin / total);
    const unsigned long long x = begin - first.head * total;
    int lo = 0, hi = T - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
    }
    first.t = lo;
    first.units = static_cast<int>(prefix[lo + 1] - prefix[lo]);
    first_s = static_cast<int>(x - prefix[lo]);
  }
  const auto tokens_of = [&](const PaItem& it) {
    int n = 1;
    while (n < p.together && it.t + n < T && prefix[it.t + n + 1] == prefix[it.t + n]) ++n;
    return n;
  };
  const auto next = [&](PaItem& it) {
    it.t += tokens_of(it);
    if (it.t >= T) {
      it.t = 0;
      ++it.head;
    }
    it.units = static_cast<int>(prefix[it.t + 1] - prefix[it.t]);
  };
  const int n_units = static_cast<int>(min(end - begin, 0x7FFFFFFFull));

  // ---- loads: this warp's slabs, kDepth ahead
  uint8_t* my_ring = ring + static_cast<size_t>(warp) * kDepth * L::kBytes;
  uint64_t* my_full = full + warp * kDepth;
  int* my_there = there + warp * kDepth;
  const uint64_t policy = l2_policy_evict_first();
  PaItem l_it = first;
  int l_s = first_s, l_batch = 0, l_st = 0, issued = 0;
  const uint8_t* l_addr = nullptr;           // lane i: the address of the batch's slab i
  const auto issue = [&]() {
    if (issued >= n_units) return;
    if (l_s >= l_it.units) {
      next(l_it);
      l_s = l_batch = 0;
    }
    if (l_batch % 32 == 0) {                 // the next 32 slabs' pages, one a lane
      l_addr = nullptr;
      const int s = l_s + lane, seq = tok_seq[l_it.t];
      if (seq >= 0 && s < l_it.units && lane < n_units - issued) {
        uint32_t in;
        const uint32_t pg = page_of(p.c, static_cast<uint32_t>(s), in);
        const uint8_t* a = page_head(
            p.c, __ldg(p.c.table + static_cast<int64_t>(seq) * p.c.max_pages + pg), l_it.head);
        if (a) l_addr = a + static_cast<int64_t>(in) * L::kBytes;
        else atomicOr(&g_err_pattn, kErrPage);
      }
    }
    if (lane == l_batch % 32) {
      my_there[l_st] = l_addr != nullptr;
      if (l_addr) {
        mbar_arrive_expect_tx(my_full + l_st, L::kBytes);
        bulk_copy_g2s(my_ring + l_st * L::kBytes, l_addr, L::kBytes, my_full + l_st, policy);
      } else {
        mbar_arrive(my_full + l_st);
      }
    }
    if (++l_st == kDepth) l_st = 0;
    ++issued;
    ++l_batch;
    ++l_s;
  };
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) issue();

  // ---- the items
  int used = 0, st = 0;                      // slabs done; the next one's stage and its phase
  uint32_t phase = 0;
  bool dead = false;                         // a wait ran out
  PaItem it = first;
  for (int s0 = first_s; used < n_units && !dead; s0 = 0, next(it)) {
    const int s1 = min(it.units, s0 + n_units - used);
    const int rows = tokens_of(it) * p.group;
    // the last key that a row sees; -1: none
    const auto limit = [&](int r) { return r < rows ? tok_pos[it.t + r / p.group] : -1; };
    const int row_s = kTwo ? (c & 1) : c;            // of this lane's scores and outputs
    const int row_b = kTwo ? (g >> 1) & 1 : g >> 1;  // of this lane's column as an operand
    const float lo = g & 1 ? -1.f : 0.f;
    const int par = kTwo ? g >> 2 : 0;
    const int lim = limit(row_s);
    int least = row_s < rows ? lim : INT_MAX;        // of all rows
#pragma unroll
    for (int o = 1; o < kRows; o <<= 1)
      least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));

    // queries: f32 * scale * 2^e as hi and lo columns, the row's largest in [2^13, 2^14)
    uint32_t qb[kSteps][2][2];
    float back;                                      // 2^-e of this lane's score row
    {
      const int tr = it.t + (row_b < rows ? row_b / p.group : 0);
      const float* q = p.q.data + tr * p.q.token_stride +
                       (it.head * p.group + (row_b < rows ? row_b % p.group : 0)) * p.q.head_stride;
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const float* x = q + 32 * (kTwo ? 2 * i + par : i) + 8 * c;
        const float4 a = __ldg(reinterpret_cast<const float4*>(x));
        const float4 b = __ldg(reinterpret_cast<const float4*>(x + 4));
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))));
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      if (kTwo) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 16));
      amax = fabsf(amax * p.scale);
      int e = amax > 0.f ? 127 + 13 - static_cast<int>(__float_as_uint(amax) >> 23) : 0;
      e = max(-120, min(120, e));
      if (row_b >= rows) e = 0;
      const float pw = exp2i(e);
      back = exp2i(-__shfl_sync(0xFFFFFFFFu, e, row_s * 8));   // g = 2 row, c = 0
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const float* x = q + 32 * (kTwo ? 2 * i + par : i) + 8 * c;
        const float4 a = __ldg(reinterpret_cast<const float4*>(x));
        const float4 b = __ldg(reinterpret_cast<const float4*>(x + 4));
        float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = row_b < rows ? v[j] * p.scale * pw : 0.f;
        if constexpr (kFmt == QWS_Q4_0) {
          // a word's nibbles (0, 4), (1, 5) * 16; (2, 6), (3, 7) * 16
          qb[i][0][0] = split_part(v[0], v[4], lo);
          qb[i][0][1] = split_part(v[1] * 0.0625f, v[5] * 0.0625f, lo);
          qb[i][1][0] = split_part(v[2], v[6], lo);
          qb[i][1][1] = split_part(v[3] * 0.0625f, v[7] * 0.0625f, lo);
        } else {
          // bytes (0, 2), (1, 3); (4, 6), (5, 7)
          qb[i][0][0] = split_part(v[0], v[2], lo);
          qb[i][0][1] = split_part(v[1], v[3], lo);
          qb[i][1][0] = split_part(v[4], v[6], lo);
          qb[i][1][1] = split_part(v[5], v[7], lo);
        }
      }
    }

    float o[kSteps][4] = {};
    const float back2 = back * kLog2e;
    float m = -INFINITY, k = 0.f, l = 0.f;
    for (int s = s0; s < s1; ++s) {
      const bool ok = mbar_wait(my_full + st, phase);
      if (__any_sync(0xFFFFFFFFu, !ok)) {
        dead = true;
        if (lane == 0) atomicOr(&g_err_pattn, kErrFullWait);
        break;
      }
      const uint8_t* slab = my_ring + st * L::kBytes;
      const int seen = my_there[st] ? lim : -1;
      float sc[2] = {0.f, 0.f}, ee[2];       // keys g, g + 8
      constexpr uint32_t kM0 = kFmt == QWS_Q4_0 ? 0x000F000Fu : 0x00FF00FFu;
      constexpr uint32_t kM1 = 0x00F000F0u, kZ0 = 0x64086408u, kZ1 = 0x64806480u;
      const bool odd = c >= 2;
      const int odd16 = odd ? 16 : 0;
      // ---- scores
      uint32_t kw[2][kWords], ks[2][(kBlocks + 1) / 2];
      load_chunk<L>(slab, 0, lane, kw[0]);
      load_chunk<L>(slab, 1, lane, kw[1]);
      load_scales<kBlocks>(slab + L::kKScale + 2 * kBlocks * g, ks[0]);
      load_scales<kBlocks>(slab + L::kKScale + 2 * kBlocks * (g + 8), ks[1]);
      if constexpr (kTwo) {
        // 8 keys of two blocks an instruction
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float d[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if constexpr (kFmt == QWS_Q4_0) {
                const uint32_t x = kw[h][2 * i] >> (8 * k), y = kw[h][2 * i + 1] >> (8 * k);
                mma_step(k, d, centred<kM0, kZ0>(x), centred<kM0, kZ0>(y), centred<kM1, kZ1>(x),
                        centred<kM1, kZ1>(y), qb[i][k][0], qb[i][k][1]);
              } else {
                const uint32_t x = kw[h][4 * i + k], y = kw[h][4 * i + 2 + k];
                mma_step(k, d, centred<kM0, kZ1>(x), centred<kM0, kZ1>(y),
                        centred<kM0, kZ1>(x >> 8), centred<kM0, kZ1>(y >> 8), qb[i][k][0],
                        qb[i][k][1]);
              }
            }
            const float x = d[0] + d[1], y = d[2] + d[3];
            sc[h] = fmaf(half_bits_to_float(ks[h][i] >> odd16), odd ? y : x, sc[h]);
          }
        }
        sc[0] += __shfl_xor_sync(0xFFFFFFFFu, sc[0], 2);
        sc[1] += __shfl_xor_sync(0xFFFFFFFFu, sc[1], 2);
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          float d[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if constexpr (kFmt == QWS_Q4_0) {
              const uint32_t x = kw[0][i] >> (8 * k), y = kw[1][i] >> (8 * k);
              mma_step(k, d, centred<kM0, kZ0>(x), centred<kM0, kZ0>(y), centred<kM1, kZ1>(x),
                      centred<kM1, kZ1>(y), qb[i][k][0], qb[i][k][1]);
            } else {
              const uint32_t x = kw[0][2 * i + k], y = kw[1][2 * i + k];
              mma_step(k, d, centred<kM0, kZ1>(x), centred<kM0, kZ1>(y),
                      centred<kM0, kZ1>(x >> 8), centred<kM0, kZ1>(y >> 8), qb[i][k][0],
                      qb[i][k][1]);
            }
          }
          sc[0] = fmaf(half_bits_to_float(ks[0][i / 2] >> (16 * (i & 1))), d[0] + d[1], sc[0]);
          sc[1] = fmaf(half_bits_to_float(ks[1][i / 2] >> (16 * (i & 1))), d[2] + d[3], sc[1]);
        }
      }
      // the largest f16 exponent among the value's scales of keys g and g + 8
      uint32_t x, y;
      if constexpr (kBlocks == 1) {
        x = *reinterpret_cast<const uint16_t*>(slab + L::kVScale + 2 * g);
        y = *reinterpret_cast<const uint16_t*>(slab + L::kVScale + 2 * (g + 8));
      } else {
        const uint8_t* v = slab + L::kVScale + 4 * (c % (kBlocks / 2));
        x = *reinterpret_cast<const uint32_t*>(v + 2 * kBlocks * g);
        y = *reinterpret_cast<const uint32_t*>(v + 2 * kBlocks * (g + 8));
      }
      x &= 0x7FFF7FFFu;
      y &= 0x7FFF7FFFu;
      __half2 mx = bits_h2(__byte_perm(x, y, 0x5410));
      if constexpr (kBlocks > 1) {
        mx = __hmax2(mx, bits_h2(__byte_perm(x, y, 0x7632)));
        if constexpr (kBlocks >= 4)
          mx = __hmax2(mx, bits_h2(__shfl_xor_sync(0xFFFFFFFFu, h2_bits(mx), 1)));
        if constexpr (kBlocks >= 8)
          mx = __hmax2(mx, bits_h2(__shfl_xor_sync(0xFFFFFFFFu, h2_bits(mx), 2)));
      }
      const uint32_t big = h2_bits(mx);
      if (p.cap > 0.f) {
        sc[0] = soft_cap(sc[0] * back, p.cap) * kLog2e;
        sc[1] = soft_cap(sc[1] * back, p.cap) * kLog2e;
      } else {
        sc[0] *= back2;
        sc[1] *= back2;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (s * 16 + g + 8 * h > seen) sc[h] = -INFINITY;
        const int field = static_cast<int>(h ? big >> 26 : (big >> 10) & 31u);
        ee[h] = sc[h] + static_cast<float>(field - 14);
      }
      // ---- weights
      {
        float ms = fmaxf(sc[0], sc[1]), me = fmaxf(ee[0], ee[1]);
        if (__any_sync(0xFFFFFFFFu, ms > m + 2.f || me > m - k + 15.f)) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            ms = fmaxf(ms, __shfl_xor_sync(0xFFFFFFFFu, ms, d));
            me = fmaxf(me, __shfl_xor_sync(0xFFFFFFFFu, me, d));
          }
          if (ms > m + 2.f || me > m - k + 15.f) {
            const float mn = fmaxf(m, ms);
            const float kn = floorf(mn - fmaxf(m - k, me - 12.f));    // some -6 to 26
            const float f = ex2(m - mn), fo = f * ex2(kn - k);
            m = mn;
            k = kn;
            l *= f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[i][j] *= fo;
          }
        }
      }
      const float pk = ex2(k);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (nothing seen yet: m is -inf too)
        sc[h] = sc[h] == -INFINITY ? 0.f : ex2(sc[h] - m);
        l += sc[h];
        sc[h] *= pk;
      }
      // ---- as operands: this lane's column, keys 2c, 2c + 1, 2c + 8, 2c + 9
      float w[4];
      uint32_t vs[4][(kBlocks + 1) / 2], vw[2][kWords];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = __shfl_sync(0xFFFFFFFFu, sc[j / 2], 8 * c + 4 * (j & 1) + row_b);
        load_scales<kBlocks>(slab + L::kVScale + 2 * kBlocks * (2 * c + (j & 1) + 4 * (j & 2)),
                             vs[j]);
      }
      load_chunk<L>(slab + L::kV, 0, lane, vw[0]);
      load_chunk<L>(slab + L::kV, 1, lane, vw[1]);
      if (s * 16 + 15 > least || seen < 0) {
        // keys that some row does not see: their scales may be anything
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < (kBlocks + 1) / 2; ++i) vs[j][i] = w[j] == 0.f ? 0u : vs[j][i];
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int wi = kTwo ? i : i / 2;
        const uint32_t sel = (kTwo ? par : i & 1) ? 0x7632u : 0x5410u;
        uint32_t vb[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 d =
              __half22float2(bits_h2(__byte_perm(vs[2 * j][wi], vs[2 * j + 1][wi], sel)));
          vb[j] = split_part(w[2 * j] * d.x, w[2 * j + 1] * d.y, lo);
        }
        if constexpr (kTwo) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float d[4];
            if constexpr (kFmt == QWS_Q4_0) {
              const auto code = [&](uint32_t x) {
                x >>= j & 2 ? 8 : 0;
                return j & 1 ? centred<kM1, kZ1>(x) : centred<kM0, kZ0>(x);
              };
              mma_f16_first(d, code(vw[0][2 * i]), code(vw[0][2 * i + 1]),
                       code(vw[1][2 * i]), code(vw[1][2 * i + 1]), vb[0], vb[1]);
            } else {
              const int k = j / 2, sh = j & 1 ? 8 : 0;
              mma_f16_first(d, centred<kM0, kZ1>(vw[0][4 * i + k] >> sh),
                      centred<kM0, kZ1>(vw[0][4 * i + 2 + k] >> sh),
                      centred<kM0, kZ1>(vw[1][4 * i + k] >> sh),
                      centred<kM0, kZ1>(vw[1][4 * i + 2 + k] >> sh), vb[0], vb[1]);
            }
            const float x = d[0] + d[1], y = d[2] + d[3];
            o[i][j] += odd ? y : x;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            float d[4];
            if constexpr (kFmt == QWS_Q4_0) {
              const int sh = j ? 8 : 0;
              const uint32_t x = vw[0][i] >> sh, y = vw[1][i] >> sh;
              mma_f16_first(d, centred<kM0, kZ0>(x), centred<kM1, kZ1>(x), centred<kM0, kZ0>(y),
                      centred<kM1, kZ1>(y), vb[0], vb[1]);
            } else {
              const uint32_t x = vw[0][2 * i + j / 2], y = vw[1][2 * i + j / 2];
              mma_f16_first(d, centred<kM0, kZ1>(x), centred<kM0, kZ1>(x >> 8),
                      centred<kM0, kZ1>(y), centred<kM0, kZ1>(y >> 8), vb[0], vb[1]);
            }
            o[i][j] += d[0] + d[1];
            o[i][j + 1] += d[2] + d[3];
          }
        }
      }
      ++used;
      if (++st == kDepth) {
        st = 0;
        phase ^= 1;
      }
      __syncwarp();
      issue();
    }
    // ---- the item, or this warp's part of it
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    const bool whole = s0 == 0 && s1 == it.units;
    const int slot = s0 == 0;
    float* to = p.out.data + (it.t + row_s / p.group) * p.out.token_stride +
                (it.head * p.group + row_s % p.group) * p.out.head_stride;
    float y = ex2(-k);
    if (whole) {
      y = l == 0.f ? 0.f : y / l;
    } else {
      // its last item's part goes where the slabs were: all of them have been read
      to = (slot ? reinterpret_cast<float*>(my_ring) : join + warp * kRows * kHd) + row_s * kHd;
      if (g == 0 && c < kRows) {
        stat[slot][warp][c][0] = m;
        stat[slot][warp][c][1] = l;
      }
      if (lane == 0) parts[slot][warp] = PaPart{it.t, it.head, rows, s1 == it.units};
    }
    const float x = kFmt == QWS_Q4_0 ? 0.0625f * y : y;
    if (row_s < rows) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        *reinterpret_cast<float4*>(to + 32 * (kTwo ? 2 * i + (c >> 1) : i) + 4 * g) =
            make_float4(o[i][0] * y, o[i][1] * x, o[i][2] * y, o[i][3] * x);
    }
  }
  // copies still in flight after a wait that ran out
  for (; used < issued; ++used) {
    mbar_wait(my_full + st, phase);
    if (++st == kDepth) {
      st = 0;
      phase ^= 1;
    }
  }
  __syncthreads();

  // ---- parts of one item in neighbouring warps: the first is a slot 1, or slot 0 of warp 0
  // for an item begun by an earlier CTA; slots 0 follow until the item ends.  A warp takes a row of
  // an item at a time, a part's m and l to a lane.  (All threads going through the items one
  // after the other took 5000 to 9000 cycles.)
  const bool has = lane < kWarps;
  const uint32_t has0 = __ballot_sync(0xFFFFFFFFu, has && parts[0][has ? lane : 0].t >= 0);
  const uint32_t has1 = __ballot_sync(0xFFFFFFFFu, has && parts[1][has ? lane : 0].t >= 0);
  const uint32_t end0 = has0 & __ballot_sync(0xFFFFFFFFu, has && parts[0][has ? lane : 0].ends);
  static_assert(kWarps < 31, "a bit a warp, one more for the first lead");
  const uint32_t leads = has1 << 1 | (has0 & 1u);
  for (int task = warp; task < __popc(leads) * kRows; task += kWarps) {
    uint32_t lead = leads;
    for (int i = task / kRows; i > 0; --i) lead &= lead - 1;
    const int at = __ffs(static_cast<int>(lead)) - 1, slot = at > 0, w0 = max(at - 1, 0);
    const int r = task % kRows;
    const PaPart a = parts[slot][w0];
    if (r >= a.rows) continue;
    int n = 1;
    bool ends = a.ends;
    if (!ends) {
      const int run = __ffs(static_cast<int>(~(has0 >> (w0 + 1)))) - 1;
      const int e = __ffs(static_cast<int>(end0 >> (w0 + 1)));
      ends = e > 0 && e <= run;
      n += ends ? e : run;
    }
    float mi = -INFINITY, li = 0.f;
    if (lane < n) {
      const float* ml = stat[slot && lane == 0][w0 + lane][r];
      mi = ml[0];
      li = ml[1];
    }
    float mx = mi;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    const float f = mi == -INFINITY ? 0.f : ex2(mi - mx);
    float ls = f * li;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) ls += __shfl_xor_sync(0xFFFFFFFFu, ls, d);
    constexpr int kCols = kHd / 4, kPer = (kCols + 31) / 32;
    const bool in = kCols >= 32 || lane < kCols;
    float4 v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float fi = __shfl_sync(0xFFFFFFFFu, f, i);
      const float* part = (i == 0 && slot ? reinterpret_cast<const float*>(
                                                ring + static_cast<size_t>(w0) * kDepth * L::kBytes)
                                          : join + (w0 + i) * kRows * kHd) + r * kHd;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (in) {
          const float4 z = *reinterpret_cast<const float4*>(part + 4 * (lane + 32 * j));
          v[j].x = fmaf(fi, z.x, v[j].x); v[j].y = fmaf(fi, z.y, v[j].y);
          v[j].z = fmaf(fi, z.z, v[j].z); v[j].w = fmaf(fi, z.w, v[j].w);
        }
      }
    }
    const bool whole = slot && ends;
    const size_t place = (static_cast<size_t>(blockIdx.x) * 2 + slot) * kRows + r;
    const float y = !whole ? 1.f : ls == 0.f ? 0.f : 1.f / ls;
    float* to = whole ? p.out.data + (a.t + r / p.group) * p.out.token_stride +
                            (a.head * p.group + r % p.group) * p.out.head_stride
                      : p.parts + place * kHd;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (in)
        *reinterpret_cast<float4*>(to + 4 * (lane + 32 * j)) =
            make_float4(v[j].x * y, v[j].y * y, v[j].z * y, v[j].w * y);
    if (!whole && lane == 0) {
      float* ml = p.parts + static_cast<size_t>(gridDim.x) * 2 * kRows * kHd + place * 2;
      *reinterpret_cast<float2*>(ml) = make_float2(mx, ls);
    }
  }
  if (tid == 0) {
    // the item that goes on in the next CTA: the last one begun, unless it ends here
    int4 join_of = make_int4(-1, 0, 0, 0);
    const int w = 31 - __clz(static_cast<int>(has1));
    if (has1 && end0 >> (w + 1) == 0) {
      const PaPart a = parts[1][w];
      const unsigned long long last = a.head * total + prefix[a.t + 1] - 1;
      join_of = make_int4(a.t, a.head | a.rows << 16, static_cast<int>(last / share), 0);
    }
    p.joins[blockIdx.x] = join_of;
  }
}

// Joins an item that CTAs blockIdx.x .. last computed parts of: slot 1 of the first, slot 0 of
// the others.
constexpr int kPjThreads = 256;

template <int kHd>
__global__ void __launch_bounds__(kPjThreads)
    paged_join_kernel(const __grid_constant__ PagedAttnParams p, int n_ctas, int max_rows) {
  __shared__ float4 part[kPjThreads];
  __shared__ float lsum[kPjThreads];
  pdl_launch_dependents();
  pdl_wait();
  const int first = blockIdx.x, r = blockIdx.y;
  const int4 j = p.joins[first];
  const int rows = j.y >> 16, head = j.y & 0xFFFF;
  if (j.x < 0 || r >= rows) return;
  const int n = j.z - first + 1;
  const float2* ml =
      reinterpret_cast<const float2*>(p.parts + static_cast<size_t>(n_ctas) * 2 * max_rows * kHd);
  const auto slot = [&](int i) {
    return (static_cast<size_t>(first + i) * 2 + (i == 0)) * max_rows + r;
  };
  constexpr int kCols = kHd / 4, kLanes = kPjThreads / kCols;
  const int d = threadIdx.x % kCols, k = threadIdx.x / kCols;
  // the first part's load is on its way before the maximum is known
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float2 s = make_float2(0.f, 0.f);
  const auto load = [&](int i) {
    if (i >= n) return;
    v = *reinterpret_cast<const float4*>(p.parts + slot(i) * kHd + 4 * d);
    s = ml[slot(i)];
  };
  load(k);
  float mx = -INFINITY;
  for (int i = threadIdx.x % 32; i < n; i += 32) mx = fmaxf(mx, ml[slot(i)].x);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float ls = 0.f;
  for (int i = k; i < n; i += kLanes) {
    const float f = s.x == -INFINITY ? 0.f : ex2(s.x - mx);
    a.x = fmaf(f, v.x, a.x); a.y = fmaf(f, v.y, a.y);
    a.z = fmaf(f, v.z, a.z); a.w = fmaf(f, v.w, a.w);
    ls = fmaf(f, s.y, ls);
    load(i + kLanes);
  }
  part[threadIdx.x] = a;
  lsum[threadIdx.x] = ls;
  __syncthreads();
  if (k) return;
  for (int i = 1; i < kLanes; ++i) {
    const float4 z = part[i * kCols + d];
    a.x += z.x; a.y += z.y; a.z += z.z; a.w += z.w;
    ls += lsum[i * kCols + d];
  }
  const float f = ls == 0.f ? 0.f : 1.f / ls;
  float* to = p.out.data + (j.x + r / p.group) * p.out.token_stride +
              (head * p.group + r % p.group) * p.out.head_stride + 4 * d;
  *reinterpret_cast<float4*>(to) = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
}

// Rows of an item: the query rows that a kv head's codes are unpacked for, group times the
// neighbouring tokens of a sequence, if they are two and head_dim is more than one block (see kRows), else
// four.  12 sequences of up to 4099 positions, Q4_0, heads of 256, two query heads a kv head, in four rows
// and in two: four tokens each 21.5 and 29.0 us, two 17.3 and 18.9; one query head, heads of 128:
// 16.0 and 22.2, 16.0 and 14.8.  How many there are only the caller knows, the table may have
// rows to spare; without a word from it, more tokens than rows must mean some.
static int rows_of(int64_t n_tokens, int64_t n_seqs, int tokens_per_seq, int group, int head_dim) {
  const int64_t tokens = tokens_per_seq ? tokens_per_seq : n_tokens > n_seqs ? 4 : 1;
  return head_dim == 32 || group * tokens > 2 ? 4 : 2;
}

size_t paged_attention_workspace_bytes(int64_t, int, int, int head_dim) {
  const size_t slots = static_cast<size_t>(device_sms()) * 2 * 4;
  return (slots * (head_dim + 2) * sizeof(float) + device_sms() * sizeof(int4) + 255) / 256 * 256;
}

template <int kHd, int kFmt, int kRows>
cudaError_t launch_paged_rows(const PagedAttnParams& p, int grid, cudaStream_t st) {
  using C = PaCfg<kHd, kFmt, kRows>;
  const auto kernel = paged_attention_kernel<kHd, kFmt, kRows>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_once(kernel, C::kSmem, false, done);
  if (e != cudaSuccess) return e;
  e = pdl_launch(kernel, dim3(static_cast<unsigned>(grid)), C::kThreads, C::kSmem, st, p);
  if (e != cudaSuccess) return e;
  return pdl_launch(paged_join_kernel<kHd>, dim3(static_cast<unsigned>(grid), kRows), kPjThreads, 0,
                    st, p, grid, kRows);
}

template <int kHd, int kFmt>
cudaError_t launch_paged_fmt(const PagedAttnParams& p, int rows, int grid, cudaStream_t st) {
  if constexpr (kHd > 32)
    if (rows == 2) return launch_paged_rows<kHd, kFmt, 2>(p, grid, st);
  return launch_paged_rows<kHd, kFmt, 4>(p, grid, st);
}

cudaError_t launch_paged_attention(const PagedView& c, int fmt, const qws_heads& q,
                                   const qws_heads& out, const int64_t* seqs,
                                   const int64_t* positions, int64_t n_tokens,
                                   int tokens_per_seq, int group, int head_dim, float scale,
                                   float cap, void* ws, cudaStream_t st) {
  const int grid = device_sms();
  const int rows = rows_of(n_tokens, c.n_seqs, tokens_per_seq, group, head_dim);
  PagedAttnParams p{c, q, out, seqs, positions, 0, group, rows / group, scale, cap, nullptr, nullptr};
  p.parts = static_cast<float*>(ws);
  p.joins = reinterpret_cast<int4*>(p.parts + static_cast<size_t>(grid) * 2 * 4 * (head_dim + 2));
  for (int64_t t = 0; t < n_tokens; t += kPaMaxRows) {
    p.n_tokens = static_cast<int>(std::min<int64_t>(kPaMaxRows, n_tokens - t));
    p.seqs = seqs + t;
    p.positions = positions + t;
    p.q.data = q.data + t * q.token_stride;
    p.out.data = out.data + t * out.token_stride;
    cudaError_t e = cudaErrorInvalidValue;
#define QWS_PATTN(HD)                                                       \
  case HD:                                                                  \
    e = fmt == QWS_Q4_0 ? launch_paged_fmt<HD, QWS_Q4_0>(p, rows, grid, st) \
                        : launch_paged_fmt<HD, QWS_Q8_0>(p, rows, grid, st); \
    break;
    switch (head_dim) {
      QWS_PATTN(32) QWS_PATTN(64) QWS_PATTN(128) QWS_PATTN(256)
    }
#undef QWS_PATTN
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

unsigned read_clear_pattn_errors() {
  unsigned v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_pattn, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_err_pattn, &z, sizeof(z));
  return v;
}

}  // namespace qws
