// sample.cu -- the next token of every row of logits, from a given random number.
//
// Order of the tokens: larger logits first, equal ones by index.  w_i = exp((x_i - max) / T).
// Kept is a prefix of that order, the shortest of
//   top_k   the first k;
//   top_p   as few as reach top_p of the sum over the first k;
//   min_p   those with w >= min_p.
// The token is the smallest index i with sum_{j <= i, kept} w_j > u * (sum of the kept).
//
// Sums over a vocabulary decide between neighbours, so they have to be better than f32: a
// weight is a whole number of 2^-44 of the largest, and sums of whole numbers are exact and the
// same in any order.  The exponential is 2^-t, t = (max - x) log2(e) / T as a pair of f32
// (value and remainder); 2^-t = 2^-n 2^(-k/1024) 2^-r with the middle factor from a table and
// |r| <= 2^-11 by series: about 2^-42 of the weight.
//
// The vocabulary is not sorted: top_k and top_p are a border among the f32 values, found by a
// histogram of the keys (counts, or weights) in linear steps from the largest down.  With at most
// 256 tokens above the border's bin one CTA puts these in order and does the rest; with at most 1024
// in the bin it finds the border among those; else further histograms narrow the bin down.
// Up to 256 are put in order by counting who comes before (5 us less than a sort), more by a sort.
//
// Bound by latency: a row's logits are read once, into the shared memory of a cluster of CTAs, and
// the rest is passes over these and barriers of the cluster: 262144 logits take 6.7 us greedily,
// 8.2 with min_p, 11.6 with all their weights, 13.6 with top_k 64 and top_p, 29 with top_p alone
// where thousands of tokens are kept; 9 rows of 50257 with top_p 20; 64 rows of 262144 with mixed
// filters 68.  512 threads a CTA, two of them on an SM, were slower for many rows (104 for those
// 64, of 78 then).  A warp's word for all (sums over the CTAs) saves 1.6 us of each of these.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "launch.h"
#include "sample_plan.h"

namespace qws {

constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaBins = 2048;
constexpr int kSaFew = kSaThreads;           // candidates that one CTA puts in order
constexpr int kSaRank = kSaThreads / 4;      // of which it orders by counting, a quarter a thread
static_assert(kSaWarps == 32 && kSaFew * 8 <= kSaBins * 4, "a list in place of a histogram");

// 2^(-k/1024) in units of 2^-45, by the exponential's power series at compile time
struct ExpTable {
  unsigned long long v[1024];
};
constexpr ExpTable make_exp_table() {
  ExpTable t{};
  for (int k = 0; k < 1024; ++k) {
    // by squares of exp(y / 8)
    const double y = -0.693147180559945309 * k / 1024 / 8;
    double term = 1, s = 1;
    for (int i = 1; i < 14; ++i) {
      term *= y / i;
      s += term;
    }
    s *= s;
    s *= s;
    s *= s;
    t.v[k] = static_cast<unsigned long long>(s * 35184372088832.0 + 0.5);
  }
  return t;
}
__device__ const ExpTable kExp = make_exp_table();

// How a cluster adds up its CTAs' histograms: CTA r has bins r * bins on; where there are more
// threads than bins, `groups` of them share out the CTAs, `ctas` each (two or three).
struct BinShare {
  int bins, groups, ctas, per_bin;    // per_bin: 2^20 / bins, rounded up
};

struct SampleParams {
  const float* logits;
  int64_t stride;
  int vocab, slice, vec;           // slice: logits of a CTA; vec: rows are 16-byte aligned
  BinShare share;
  const float *u, *temperature, *top_p, *min_p;
  const int64_t* top_k;
  int64_t* out;
};

typedef unsigned long long u64;

// u32 in the order of the floats; NaN counts as -inf, -0 as 0
__device__ __forceinline__ uint32_t order_key(float x) {
  x = x != x ? -INFINITY : x + 0.0f;
  const uint32_t b = __float_as_uint(x);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kKeyNone = 0x007FFFFFu;   // of -inf

struct Weigher {
  float top, ch, cl;      // the row's largest; log2(e) / T as a pair
  const u64* table;

  __device__ __forceinline__ u64 operator()(float x) const {
    // top - x and its remainder; no branches, so that several run side by side
    const float dh = __fsub_rn(top, x);
    const float bb = __fsub_rn(dh, top);
    const float dl = __fsub_rn(__fsub_rn(top, __fsub_rn(dh, bb)), __fadd_rn(x, bb));
    // beyond 2^-46 the shift below leaves nothing, whatever the rest comes to (infinities too)
    const float th = fminf(__fmul_rn(dh, ch), 50.f);
    const float tl = __fmaf_rn(dl, ch, __fmaf_rn(dh, cl, __fmaf_rn(dh, ch, -th)));
    constexpr float kRound = 12288.f;                      // 1.5 * 2^23 / 2^10
    const float tk = __fadd_rn(th, kRound);                // th * 1024, rounded, in its last bits
    const uint32_t k = __float_as_uint(tk);
    const float rh = __fsub_rn(th, __fsub_rn(tk, kRound));
    // v = r ln 2;  2^-r - 1 = -v + v^2 / 2 - v^3 / 6
    constexpr float kLn2 = 0.69314718f, kLn2Low = -1.9046542e-9f;
    const float vh = __fmul_rn(rh, kLn2);
    const float vl = __fmaf_rn(tl, kLn2, __fmaf_rn(rh, kLn2Low, __fmaf_rn(rh, kLn2, -vh)));
    // -vh - vl + (vh + vl)^2 / 2 - ...; vl is below 2^-17
    const float v = vh + vl;
    const float pl = __fmaf_rn(v * v, __fmaf_rn(v, -1.f / 6, 0.5f), -vl);
    const int P = static_cast<int>(static_cast<uint32_t>(__float2int_rn(pl * 0x1p42f)) -
                                   static_cast<uint32_t>(__float2int_rn(vh * 0x1p42f)));
    const u64 t = table[k & 1023];                         // in units of 2^-45
    const int t31 = static_cast<int>((t - (t >> 45)) >> 14);
    const u64 w = t + static_cast<u64>((static_cast<long long>(t31) * P) >> 28);
    const u64 r = ((w >> (k >> 10 & 63)) + 1) >> 1;
    return x == top ? 1ull << 44 : r;                      // (the top may be infinite)
  }
};

// ------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// the address of p, a place in this CTA's shared memory, in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void remote_store(uint32_t a, u64 v, u64 w) {
  asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(a), "l"(v), "l"(w) : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_load(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t remote_add(uint32_t a, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
  return old;
}

struct SampleShared {
  alignas(16) uint32_t hist[4][kSaBins];   // counts in the first; weights by digits of 15 bits
  u64 table[1024];
  u64 fold[kSaThreads];                    // a bin's mass in two CTAs, and its number
  uint32_t fold_n[kSaThreads];
  alignas(16) u64 box[2][kSaMaxCluster][2];   // [turn][from rank]: what the CTAs tell one another
  alignas(16) u64 cut[2][2];       // [turn]: the bin that a round found (+ whole), the mass above it
  u64 part[2][kSaWarps + 1];       // sums of the warps before, and of all
  u64 told[2][2];                  // [word]: sums over the CTAs before this one, and over all
  float low[2];                    // T ln min_p, as a pair
  uint32_t n_few[2];               // candidates: all of the row's (rank 0), this CTA's

  // lists of candidates, when the histograms are done with
  __device__ u64* few(int i) { return reinterpret_cast<u64*>(hist[i]); }
  uint32_t part32[3][kSaWarps];
};

// One CTA's view of its cluster.  Every call of a member function is made by all threads of all
// CTAs of the cluster.
struct Team {
  SampleShared& s;
  const BinShare& share;
  uint32_t rank, size;
  int turn;

  // two words of every CTA to all; read them with box(word, rank) until the next tell()
  __device__ __forceinline__ void tell(u64 a, u64 b) {
    turn ^= 1;
    if (threadIdx.x < size) {
      remote_store(remote(&s.box[turn][rank][0], threadIdx.x), a, b);
    }
    cluster_sync();
  }
  __device__ __forceinline__ u64 box(int word, uint32_t r) const { return s.box[turn][r][word]; }

  // Sums of the words told: over the CTAs before this one, and over all.  A warp a word: all
  // warps adding up sixteen numbers each took 3000 cycles.
  __device__ __forceinline__ void sums(u64 (&before)[2], u64 (&total)[2]) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < 2) {
      const u64 own = lane < static_cast<int>(size) ? box(warp, lane) : 0ull;
      u64 x = own;
#pragma unroll
      for (int o = 1; o < kSaMaxCluster; o <<= 1) {
        const u64 y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == static_cast<int>(rank)) s.told[warp][0] = x - own;
      if (lane == static_cast<int>(size) - 1) s.told[warp][1] = x;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      before[i] = s.told[i][0];
      total[i] = s.told[i][1];
    }
  }
  // What the one thread for which `mine` is true found, to all CTAs; they have it after the next
  // cluster_sync.
  __device__ __forceinline__ void publish(bool mine, u64 a, u64 b) const {
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine);
    if (!who) return;
    const int from = __ffs(static_cast<int>(who)) - 1;
    a = __shfl_sync(0xFFFFFFFFu, a, from);
    b = __shfl_sync(0xFFFFFFFFu, b, from);
    const uint32_t to = threadIdx.x & 31;
    if (to < size) remote_store(remote(&s.cut[turn][0], to), a, b);
  }
};

// Sums over the CTA's threads before this one, and over all, of one or two values.
template <int kN>
__device__ __forceinline__ void block_scan(SampleShared& s, const u64 (&v)[kN], u64 (&before)[kN],
                                           u64 (&total)[kN]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    x[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xFFFFFFFFu, x[i], o);
      if (lane >= o) x[i] += y;
    }
  }
  __syncthreads();
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < kN; ++i) s.part[i][warp] = x[i];
  __syncthreads();
  // one warp for the warps' sums: shuffles of 64 bits by all of them take longer than the barrier
  if (warp < kN) {
    u64 w = s.part[warp][lane];
    const u64 own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    s.part[warp][lane] = w - own;
    if (lane == 31) s.part[warp][kSaWarps] = w;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    before[i] = s.part[i][warp] + x[i] - v[i];
    total[i] = s.part[i][kSaWarps];
  }
}

struct Steps {
  float top, scale;       // bins of 1 / scale from the largest logit down

  // higher for larger keys (every operation keeps the order)
  __device__ __forceinline__ uint32_t operator()(uint32_t key) const {
    const int b = __float2int_rz(__fmul_rn(__fsub_rn(top, key_value(key)), scale));
    return static_cast<uint32_t>(kSaBins - 1 - max(0, min(kSaBins - 1, b)));
  }
  // the smallest key in [lo, hi] whose bin is b or above, hi + 1 without one; by a whole warp
  __device__ __forceinline__ u64 first_of(uint32_t b, uint32_t lo, uint32_t hi) const {
    u64 from = lo, to = static_cast<u64>(hi) + 1;              // the answer is in [from, to]
    while (from < to) {
      const u64 step = (to - from + 31) / 32, k = from + (threadIdx.x & 31) * step;
      const uint32_t yes = __ballot_sync(0xFFFFFFFFu, k >= to || (*this)(static_cast<uint32_t>(k)) >= b);
      const int f = yes ? __ffs(static_cast<int>(yes)) - 1 : 32;
      if (f < 32) to = min(to, from + f * step);
      if (f > 0) from = min(to, from + (f - 1) * step + 1);
    }
    return from;
  }
};

// The values of the first n threads (others have ~0) in rising order over the threads; n2: a
// power of two, n <= n2 <= kSaThreads.  Neighbours of up to 32 trade in registers, others through
// two buffers of kSaThreads in turn: one barrier a step.
__device__ __forceinline__ u64 block_sort(u64 v, int n2, u64* buf) {
  const int tid = threadIdx.x;
  const bool in = (tid & ~31) < n2;                // other warps only take the barriers
  u64* b = buf;
  for (int k = 2; k <= n2; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      u64 o = v;
      if (j >= 32) {
        if (in) b[tid] = v;
        __syncthreads();
        if (in) o = b[tid ^ j];
        b = b == buf ? buf + kSaThreads : buf;
      } else if (in) {
        o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
      }
      v = ((tid & k) == 0) == ((tid & j) == 0) ? min(v, o) : max(v, o);
    }
  return v;
}

__device__ __forceinline__ int power_of_two(int n) { return n < 2 ? 1 : 1 << (32 - __clz(n - 1)); }

// Candidates, the logits whose keys `take` accepts, to the list of the cluster's first CTA, at most
// kSaFew; returns their number there.  A candidate is ~key, then its number from i0 on.
template <class Take>
__device__ __forceinline__ int collect(Team& t, const uint32_t* keys, int n, int i0, Take take) {
  SampleShared& s = t.s;
  const int tid = threadIdx.x;
  if (tid == 0) s.n_few[1] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kSaThreads) {
    const uint32_t k = keys[i];
    if (take(k)) {
      const uint32_t at = atomicAdd(&s.n_few[1], 1u);
      if (at < kSaFew)
        s.few(1)[at] = static_cast<u64>(~k) << 32 | static_cast<uint32_t>(i0 + i);
    }
  }
  __syncthreads();
  const uint32_t mine = s.n_few[1];
  if (tid == 0) s.part32[0][0] = mine ? remote_add(remote(&s.n_few[0], 0), mine) : 0u;
  __syncthreads();
  const uint32_t base = s.part32[0][0];
  if (tid < mine && base + tid < kSaFew)
    remote_store(remote(&s.few(0)[base + tid], 0), s.few(1)[tid]);
  cluster_sync();
  return min(static_cast<int>(s.n_few[0]), kSaFew);
}

// The list's m candidates in order over the threads, ~0 behind them.  Up to 256 by counting who
// comes before, a quarter of the others a thread; more are sorted.
__device__ __forceinline__ u64 in_order(SampleShared& s, int m) {
  const int tid = threadIdx.x;
  u64* list = s.few(0);
  if (m > kSaRank) return block_sort(tid < m ? list[tid] : ~0ull, power_of_two(m), s.few(1));
  const int other = tid % kSaRank, j0 = tid / kSaRank * (kSaRank / 4);
  const int j1 = min(m, j0 + kSaRank / 4);
  uint32_t* place = s.hist[2];
  if (tid < kSaRank) place[tid] = 0;
  const u64 x = other < m ? list[other] : 0ull;
  uint32_t before = 0;
  for (int j = j0; j < j1; ++j) before += list[j] < x;
  __syncthreads();
  if (other < m && before) atomicAdd(&place[other], before);
  __syncthreads();
  if (tid < m) s.few(1)[place[tid]] = x;
  __syncthreads();
  return tid < m ? s.few(1)[tid] : ~0ull;
}

// The border within a bin that holds at most kSaFew logits: the key at which the mass from
// `above` on reaches `want`; above: the mass of larger keys then.
template <class Take, class Mass>
__device__ __forceinline__ uint32_t border_of(Team& t, const uint32_t* keys, int n, u64& above,
                                              u64 want, Take take, Mass mass) {
  SampleShared& s = t.s;
  const int tid = threadIdx.x;
  const int m = collect(t, keys, n, static_cast<int>(t.rank) * kSaMaxSlice, take);
  if (t.rank == 0) {
    const u64 v = in_order(s, m);
    const uint32_t key = ~static_cast<uint32_t>(v >> 32);
    const u64 x[1] = {tid < m ? mass(key) : 0ull};
    u64 before[1], all[1];
    block_scan(s, x, before, all);
    s.fold_n[tid] = key;
    if (tid == 0) s.n_few[0] = 0;
    if (above + before[0] < want && want <= above + before[0] + x[0]) s.part32[0][0] = key;
    __syncthreads();
    t.publish(tid < m && key == s.part32[0][0] && (tid == 0 || s.fold_n[tid - 1] != key), key,
              above + before[0]);
  }
  cluster_sync();
  above = s.cut[t.turn][1];
  return static_cast<uint32_t>(s.cut[t.turn][0]);
}

template <bool kWeights, class Mass, class Want>
__device__ __forceinline__ uint32_t find_cut(Team& t, const uint32_t* keys, int n, uint32_t lo,
                                             uint32_t hi, const Steps& steps, u64& above,
                                             bool& whole, int& few, Mass mass, Want want_of) {
  SampleShared& s = t.s;
  constexpr int kDigits = kWeights ? 3 : 0;
  static_assert(kSaMaxSlice <= 1 << 16, "sums of digits of 15 bits in 32");
  const int tid = threadIdx.x, size = static_cast<int>(t.size);
  // a thread a bin, the highest with the first thread; two where one CTA has all 2048
  const int bins = t.share.bins, per = bins > kSaThreads ? 2 : 1;
  const int first_bin = (static_cast<int>(t.rank) + 1) * bins - 1 - tid * per;
  u64 want = 0;
  whole = false;
  const u64 most = static_cast<u64>(few);
  few = 0;
  for (bool first = true; first || (lo < hi && !whole); first = false) {
    const uint32_t width = hi - lo;
    const int sh = max(0, 32 - __clz(static_cast<int>(width)) - 11);
    for (int i = tid; i < (kDigits + 1) * kSaBins; i += kSaThreads) s.hist[0][i] = 0;
    if (tid == 0) s.cut[t.turn ^ 1][0] = ~0ull;    // nobody's border: the same for all CTAs then
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kSaThreads) {
      const uint32_t k = keys[i];
      if (k >= lo && k <= hi) {
        const uint32_t b = first ? steps(k) : (k - lo) >> sh;
        if constexpr (kWeights) {
          const u64 m = mass(k);
          if (m) {
            atomicAdd(&s.hist[0][b], 1u);
            atomicAdd(&s.hist[1][b], static_cast<uint32_t>(m) & 0x7FFFu);
            atomicAdd(&s.hist[2][b], static_cast<uint32_t>(m >> 15) & 0x7FFFu);
            atomicAdd(&s.hist[3][b], static_cast<uint32_t>(m >> 30));
          }
        } else {
          atomicAdd(&s.hist[0][b], 1u);
        }
      }
    }
    cluster_sync();
    const auto mass_of = [&](const uint32_t (&h)[kDigits + 1]) {
      u64 m = h[0];
      if constexpr (kWeights)
        m = h[1] + (static_cast<u64>(h[2]) << 15) + (static_cast<u64>(h[3]) << 30);
      return m;
    };
    u64 m[2] = {0, 0};
    uint32_t cnt[2] = {0, 0};
    const bool holds = tid * per < bins;
    if (size == 1) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h[kDigits + 1];
#pragma unroll
        for (int d = 0; d <= kDigits; ++d) h[d] = s.hist[d][first_bin - j];
        m[j] = mass_of(h);
        cnt[j] = h[0];
      }
    } else {
      // a bin's counts in two or three CTAs a thread, neighbouring bins side by side, then all
      const int ctas = t.share.ctas, group = (tid * t.share.per_bin) >> 20;     // tid / bins
      const int bin = static_cast<int>(t.rank) * bins + tid - group * bins, from = group * ctas;
      const auto load = [&](int cta, uint32_t (&h)[kDigits + 1]) {
#pragma unroll
        for (int d = 0; d <= kDigits; ++d)
          h[d] = cta < size && bin < kSaBins ? remote_load(remote(&s.hist[d][bin], cta)) : 0u;
      };
      uint32_t h0[kDigits + 1], h1[kDigits + 1];
      load(from, h0);
      load(from + 1, h1);
      u64 mass_in = mass_of(h0) + mass_of(h1);
      uint32_t n_in = h0[0] + h1[0];
      if (ctas == 3) {
        load(from + 2, h0);
        mass_in += mass_of(h0);
        n_in += h0[0];
      }
      s.fold[tid] = mass_in;
      s.fold_n[tid] = n_in;
      __syncthreads();
      if (holds)
        for (int j = bins - 1 - tid; j < t.share.groups * bins; j += bins) {
          m[0] += s.fold[j];
          cnt[0] += s.fold_n[j];
        }
    }
    u64 more = 0, higher;                          // the logits above by number, their mass
    if (kWeights && first && most) {
      const u64 v[2] = {m[0] + m[1], cnt[0] + cnt[1]};
      u64 before[2], mine[2];
      block_scan(s, v, before, mine);
      higher = before[0];
      more = before[1];
      t.tell(mine[0], mine[1]);
    } else {
      const u64 v[1] = {m[0] + m[1]};
      u64 before[1], mine[1];
      block_scan(s, v, before, mine);
      higher = before[0];
      t.tell(mine[0], 0);
    }
    u64 lower[2], all[2];
    t.sums(lower, all);
    higher += above + all[0] - lower[0] - t.box(0, t.rank);
    more += all[1] - lower[1] - t.box(1, t.rank);
    if (first) want = want_of(above + all[0]);
    bool found = false;
    u64 which = 0, over = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (holds && higher < want && want <= higher + m[j]) {
        const u64 exact = kWeights ? cnt[j] == 1 : higher + m[j] == want;
        const u64 number = kWeights ? more + cnt[j] : higher + m[j];
        const u64 list = first && cnt[j] <= kSaFew;
        found = true;
        which = static_cast<u64>(first_bin - j) | exact << 32 | list << 33 |
                (first && number <= most ? number << 34 : 0);
        over = higher;
      }
      higher += m[j];
      more += cnt[j];
    }
    t.publish(found, which, over);
    cluster_sync();
    if (s.cut[t.turn][0] == ~0ull) break;
    const uint32_t bin = static_cast<uint32_t>(s.cut[t.turn][0]);
    whole = s.cut[t.turn][0] >> 32 & 1;
    few = static_cast<int>(s.cut[t.turn][0] >> 34);
    above = s.cut[t.turn][1];
    if (few) return bin;
    if (s.cut[t.turn][0] >> 33 & 1) {
      whole = false;
      return border_of(
          t, keys, n, above, want,
          [&](uint32_t k) { return k >= lo && k <= hi && steps(k) == bin && mass(k) != 0; }, mass);
    }
    if (first) {
      if (tid < 64) {
        const u64 k = steps.first_of(bin + tid / 32, lo, hi);
        if (tid % 32 == 0) s.part[0][tid / 32] = k;
      }
      __syncthreads();
      lo = static_cast<uint32_t>(s.part[0][0]);
      hi = static_cast<uint32_t>(s.part[0][1] - 1);
      __syncthreads();
    } else {
      lo += bin << sh;
      hi = min(hi, lo + ((1u << sh) - 1u));
    }
  }
  return lo;
}

// z f for f >= 0 (z from 1 on), a whole number: rounded up or down, in integers.  FP64 runs at
// 1/64 of the f32 rate here, and a few operations by all threads of a CTA take microseconds.
__device__ __forceinline__ u64 part_of(u64 z, float f, bool up) {
  if (f >= 1.f) return z;
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const u64 m = e ? (bits & 0x7FFFFFu) | 0x800000u : bits;      // f = m 2^-s
  const uint32_t s = 150 - max(e, 1u);                          // 24 to 149
  const u64 lo = z * m, hi = __umul64hi(z, m);
  if (s >= 128) return up && (hi | lo) ? 1 : 0;
  if (s >= 64) {
    const u64 q = hi >> (s - 64);
    return q + (up && ((q << (s - 64)) != hi || lo) ? 1 : 0);
  }
  const u64 q = hi << (64 - s) | lo >> s;
  return q + (up && (lo << (64 - s)) ? 1 : 0);
}

// What the filters and the draw need of a row.
struct Draw {
  u64 k, z;               // first k (if any is set: use_k); else the sum that top_p is a part of
  float top_p, u;
  uint32_t least;         // min_p's smallest key
  bool use_k, use_p;

  __device__ __forceinline__ u64 wanted(u64 sum) const { return part_of(sum, top_p, true); }
  // the place among the sum of the kept weights
  __device__ __forceinline__ u64 target(u64 sum) const {
    return min(part_of(sum, u, false), sum - 1);
  }
};

// The whole choice among few candidates, the logits from bin `from` of `steps` on that have a
// weight, by one CTA.
__device__ __forceinline__ void choose_few(Team& t, const uint32_t* keys, int n, int i0,
                                           uint32_t from, uint32_t least, const Steps& steps,
                                           const Weigher& w, const Draw& d, int64_t* out) {
  SampleShared& s = t.s;
  const int tid = threadIdx.x;
  const int m = collect(t, keys, n, i0, [&](uint32_t k) {
    return k >= least && steps(k) >= from && (d.use_k || w(key_value(k)));
  });
  if (t.rank) return;
  u64* list = s.few(0);
  const u64 v = in_order(s, m);
  const uint32_t key = ~static_cast<uint32_t>(v >> 32);
  const bool first = tid < m && (!d.use_k || static_cast<u64>(tid) < d.k);
  const u64 weight[1] = {first ? w(key_value(key)) : 0ull};
  u64 before[1], sum[1];
  block_scan(s, weight, before, sum);
  const u64 want = d.wanted(d.use_k ? sum[0] : d.z);
  const bool keep =
      first && key >= d.least && (tid == 0 || !d.use_p || (d.top_p > 0.f && before[0] < want));
  const int kept = __syncthreads_count(keep);      // they are the first ones
  // by index: index and weight, 19 and 45 bits
  constexpr u64 kWeight = (1ull << 45) - 1;
  const u64 y = keep ? (v & 0xFFFFFFFFull) << 45 | weight[0] : ~0ull;
  if (kept > kSaRank) {
    const u64 z = block_sort(y, power_of_two(kept), s.few(1));
    const u64 x[1] = {tid < kept ? z & kWeight : 0ull};
    block_scan(s, x, before, sum);
    const u64 goal = d.target(sum[0]);
    if (before[0] <= goal && goal < before[0] + x[0]) *out = static_cast<int64_t>(z >> 45);
    return;
  }
  // the kept weights' sum is what the last of them has before it, and its own
  if (tid == kept - 1) s.fold[0] = before[0] + weight[0];
  if (keep) list[tid] = y;
  __syncthreads();
  const u64 goal = d.target(s.fold[0]);
  u64* part = reinterpret_cast<u64*>(s.hist[3]);
  const int other = tid % kSaRank, j0 = tid / kSaRank * (kSaRank / 4);
  const u64 x = other < kept ? list[other] : 0ull;
  u64 ahead = 0;
  for (int j = j0; j < min(kept, j0 + kSaRank / 4); ++j) {
    const u64 z = list[j];
    ahead += z < x ? z & kWeight : 0ull;
  }
  part[tid] = ahead;
  __syncthreads();
  if (tid < kept) {
    ahead = part[tid] + part[kSaRank + tid] + part[2 * kSaRank + tid] + part[3 * kSaRank + tid];
    if (ahead <= goal && goal < ahead + (x & kWeight)) *out = static_cast<int64_t>(x >> 45);
  }
}

__global__ void __launch_bounds__(kSaThreads) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SampleShared sh;
  pdl_launch_dependents();
  cluster_arrive();                                // "this CTA has started"
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < 1024; i += kSaThreads) sh.table[i] = kExp.v[i];
  if (tid == 0) sh.n_few[0] = 0;
  pdl_wait();
  Team team{sh, p.share, cluster_rank(), cluster_size(), 0};
  const int row = blockIdx.x / team.size;
  const int i0 = static_cast<int>(team.rank) * p.slice;
  const int n = max(0, min(p.vocab - i0, p.slice));
  const float* x = p.logits + row * p.stride + i0;
  const float T = p.temperature ? __ldg(p.temperature + row) : 1.f;
  const float mp = p.min_p ? __ldg(p.min_p + row) : 0.f;
  if (warp == kSaWarps - 1 && mp > 0.f && T > 0.f) {      // while the logits come
    const double low = static_cast<double>(T) * log(static_cast<double>(mp));
    sh.low[0] = static_cast<float>(low);
    sh.low[1] = static_cast<float>(low - static_cast<double>(sh.low[0]));
  }
  uint32_t hi = kKeyNone, lo = 0xFFFFFFFFu, some = 0;      // of those above -inf
  const auto take = [&](int i, float v) {
    const uint32_t k = order_key(v);
    keys[i] = k;
    hi = max(hi, k);
    if (k != kKeyNone) {
      lo = min(lo, k);
      ++some;
    }
  };
  int done = 0;
  if (p.vec) {
    done = n / 4 * 4;
#pragma unroll 4
    for (int i = 4 * tid; i < done; i += 4 * kSaThreads) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(x + i));
      take(i, v.x);
      take(i + 1, v.y);
      take(i + 2, v.z);
      take(i + 3, v.w);
    }
  }
#pragma unroll 4
  for (int i = done + tid; i < n; i += kSaThreads) take(i, __ldg(x + i));
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  some = __reduce_add_sync(0xFFFFFFFFu, some);
  if (lane == 0) {
    sh.part32[0][warp] = hi;
    sh.part32[1][warp] = lo;
    sh.part32[2][warp] = some;
  }
  __syncthreads();
  hi = __reduce_max_sync(0xFFFFFFFFu, sh.part32[0][lane]);
  lo = __reduce_min_sync(0xFFFFFFFFu, sh.part32[1][lane]);
  some = __reduce_add_sync(0xFFFFFFFFu, sh.part32[2][lane]);
  cluster_wait();                                  // the others' shared memory exists from here on
  team.tell(static_cast<u64>(hi) << 32 | lo, some);
  const bool told = lane < static_cast<int>(team.size);
  const u64 range = told ? team.box(0, lane) : static_cast<u64>(kKeyNone) << 32 | 0xFFFFFFFFu;
  hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(range >> 32));
  lo = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(range));
  const uint32_t finite =
      __reduce_add_sync(0xFFFFFFFFu, told ? static_cast<uint32_t>(team.box(1, lane)) : 0u);
  // from here on every decision is the same in all CTAs of the cluster
  if (finite == 0) {
    if (team.rank == 0 && tid == 0) p.out[row] = -1;
    return;
  }
  const uint32_t top_key = hi;
  const float top = key_value(top_key);
  Draw d{0, 0, 1.f, __ldg(p.u + row), 0, false, false};
  if (!(d.u > 0.f)) d.u = 0.f;
  uint32_t cut = 0;                                // kept: keys above, and `ties` of those equal
  u64 ties = ~0ull;
  Weigher w{top, 0.f, 0.f, sh.table};
  if (!(T > 0.f)) {
    cut = top_key;
    ties = 1;
  } else {
    // log2(e) / T as a pair
    constexpr float kL = 1.4426950216293335f, kLLow = 1.9259629e-8f;
    w.ch = kL / T;
    w.cl = (__fmaf_rn(-w.ch, T, kL) + kLLow) / T;
    // (a top_k beyond the finite logits leaves out nothing that has a weight)
    const long long k = p.top_k ? __ldg(p.top_k + row) : 0;
    d.use_k = k > 0 && static_cast<u64>(k) < finite;
    d.k = static_cast<u64>(k);
    d.top_p = p.top_p ? __ldg(p.top_p + row) : 1.f;
    d.use_p = d.top_p < 1.f;
    if (mp > 0.f) {
      // the smallest f32 that is not below max + T ln min_p
      const float t = __fadd_rn(top, sh.low[0]), tt = __fsub_rn(t, top);
      const float rest = __fadd_rn(__fsub_rn(top, __fsub_rn(t, tt)), __fsub_rn(sh.low[0], tt)) + sh.low[1];
      d.least = min(order_key(t) + (rest > 0.f ? 1u : 0u), top_key);
    }
    if (d.use_k) {
      u64 above = 0;
      bool whole;
      // More than kSaRank candidates are two sorts for one CTA.  With top_p they still take less
      // than a second search, by weights (9 rows of 262144, top_k 1000: 43 us for 59); without
      // it the border alone and the draw by all CTAs are sooner done (18 for 31 us, a row; 64: 84 for 97).
      int few = d.use_p ? kSaFew : kSaRank;
      // Steps no lower than 128 max(T, 1) below the largest, where weights end at 32 T: a mask's
      // -1e4, -1e9 or lowest f32 would have all other logits in one bin (a row of 262144 with nine in
      // ten masked so, top_k 64 and top_p: 14 us, and 33 with steps down to the smallest).
      const float low = __fsub_rd(top, 128.f * fmaxf(T, 1.f));
      const uint32_t from = min(max(lo, order_key(low)), top_key);
      const Steps steps{top, (kSaBins - 1) / (top - key_value(from))};
      cut = find_cut<false>(team, keys, n, lo, top_key, steps, above, whole, few,
                            [](uint32_t) { return 1ull; }, [&](u64) { return d.k; });
      if (few) return choose_few(team, keys, n, i0, cut, lo, steps, w, d, p.out + row);
      if (!whole) ties = d.k - above;
    }
    if (d.use_p && !(d.top_p > 0.f)) {
      cut = top_key;
      ties = 1;
    } else if (d.use_p) {
      // the keys above the cut first, then the equal ones that top_k keeps, known by number
      const u64 one_cut = ties != ~0ull ? w(key_value(cut)) : 0ull;
      const u64 last = ties != ~0ull ? ties * one_cut : 0ull;
      u64 above = 0, want = 0;
      const auto wanted = [&](u64 sum) {
        d.z = sum;
        want = d.wanted(sum + last);
        return min(want, sum);
      };
      uint32_t at = cut;
      bool whole = false;
      const uint32_t next = ties == ~0ull ? cut : cut + 1;       // the lowest of the keys above
      if (next <= top_key) {
        // (weights below 2^-46 are zero, and 32 is above 46 ln 2)
        const float low = __fsub_rd(top, __fmul_ru(32.f, T));
        const uint32_t from = min(max(max(lo, next), order_key(low)), top_key);
        const Steps steps{top, (kSaBins - 1) / (top - key_value(from))};
        int few = d.use_k ? 0 : kSaRank;
        at = find_cut<true>(team, keys, n, from, top_key, steps, above, whole, few,
                            [&](uint32_t q) { return w(key_value(q)); }, wanted);
        if (few) return choose_few(team, keys, n, i0, at, from, steps, w, d, p.out + row);
      } else {
        wanted(0);
      }
      if (want <= d.z) {
        cut = at;
        const u64 one = w(key_value(at));
        ties = whole ? ~0ull : (want - above + one - 1) / one;
      } else {
        ties = min(ties, (want - d.z + one_cut - 1) / one_cut);
      }
    }
    if (d.least > cut) {
      cut = d.least;
      ties = ~0ull;
    }
  }
  // A thread a run of neighbours, of odd length: no bank conflicts.  Its weight above the cut, and
  // how many are equal to it: of those the first `ties` count, one weight each.
  const int run = ((p.slice + kSaThreads - 1) / kSaThreads) | 1;
  const int r0 = min(n, tid * run), r1 = min(n, r0 + run);
  const u64 one = w(key_value(cut));               // (cut may be no key: then none is equal)
  u64 mine = 0, equal = 0;
#pragma unroll 4
  for (int i = r0; i < r1; ++i) {
    const uint32_t k = keys[i];
    if (k > cut) mine += w(key_value(k));
    equal += k == cut;
  }
  const u64 sums[2] = {mine, equal};
  u64 before[2], all[2];
  block_scan(sh, sums, before, all);
  team.tell(all[0], all[1]);
  u64 lower[2];
  team.sums(lower, all);
  u64 z = all[0];
  const u64 z_equal = all[1], ahead = before[0] + lower[0];
  u64 met = before[1] + lower[1];
  z += min(ties, z_equal) * one;
  const u64 target = d.target(z);
  u64 cum = ahead + min(ties, met) * one;
  if (cum <= target && target < ahead + mine + min(ties, met + equal) * one) {
    for (int i = r0; i < r1; ++i) {
      const uint32_t k = keys[i];
      if (k > cut) cum += w(key_value(k));
      else if (k == cut && met++ < ties) cum += one;
      if (cum > target) {
        p.out[row] = i0 + i;
        break;
      }
    }
  }
}

static cudaLaunchConfig_t sample_config(int n_rows, int size, size_t smem, cudaStream_t st,
                                        cudaLaunchAttribute (&attr)[2]) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(size);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_rows * size));
  cfg.blockDim = dim3(kSaThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of that size that the device runs at once: 152 SMs hold 76 of 2, 23 of 6, but 15 of 8
// and 7 of 16, whose SMs have to be neighbours; none of a size for which too few are in reach.  Asked
// once a device and size (some microseconds); a question that fails is not an answer and is not kept.
static cudaError_t clusters_at_once(int size, int* n) {
  static std::atomic<int> known[64][kSaMaxCluster + 1];      // 0: not asked; else the answer + 1
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int k = dev < 64 ? known[dev][size].load(std::memory_order_relaxed) : 0;
  if (k) {
    *n = k - 1;
    return cudaSuccess;
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = sample_config(1, size, kSaMaxSlice * 4, nullptr, attr);
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, sample_kernel, &cfg);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  if (dev < 64) known[dev][size].store(*n + 1, std::memory_order_relaxed);
  return cudaSuccess;
}

cudaError_t launch_sample(const float* logits, int64_t stride, int vocab, int n_rows,
                          const float* u, const float* temperature, const int64_t* top_k,
                          const float* top_p, const float* min_p, int64_t* out, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_once(sample_kernel, kSaMaxSlice * 4, true, done);
  if (e != cudaSuccess) return e;
  cudaError_t asked = cudaSuccess;
  const int size = sample_cluster_size(vocab, n_rows, [&](int i) {
    int n = 0;
    const cudaError_t a = clusters_at_once(i, &n);
    if (a != cudaSuccess) {
      asked = a;
      return 0;
    }
    return n;
  });
  if (size == 0) return asked != cudaSuccess ? asked : cudaErrorInvalidClusterSize;
  SampleParams p{logits, stride, vocab, 0, 0, {}, u, temperature, top_p, min_p, top_k, out};
  p.slice = ((vocab + size - 1) / size + 3) / 4 * 4;
  p.vec = reinterpret_cast<uintptr_t>(logits) % 16 == 0 && (stride % 4 == 0 || n_rows == 1);
  p.share.bins = (kSaBins + size - 1) / size;
  p.share.groups = std::max(1, kSaThreads / p.share.bins);
  p.share.ctas = (size + p.share.groups - 1) / p.share.groups;
  p.share.per_bin = ((1 << 20) + p.share.bins - 1) / p.share.bins;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      sample_config(n_rows, size, static_cast<size_t>(p.slice) * 4, st, attr);
  return cudaLaunchKernelEx(&cfg, sample_kernel, p);
}

}  // namespace qws
