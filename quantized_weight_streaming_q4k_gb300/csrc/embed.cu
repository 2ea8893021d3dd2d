// embed.cu -- rows of a quantised embedding table, scaled (the input of a
// decode step or of a prompt; the table is the one the lm_head multiplies
// when the two are tied):
//   out[t][i] = scale * dequant(W)[token[t]][i].
//
// One thread writes runs of four consecutive values with 16-byte stores and reads
// the 2 to 4 bytes of codes behind each, the block's f16 scale(s) and its
// sub-block scale; the reads of a block's scales hit L1 for all but the first
// thread.  Bound by writing out (4 bytes written per 0.56 to 1.06 read) for many
// tokens, behind two dependent reads, the token and its row: 4001 rows of 2560 Q6_K
// values take 13.2 us (3.7 TB/s; 49 MB at the copy rate: 7.3 us).  160 threads x 4 runs
// were best there; 128 x 5 took 14.1, 320 x 2 13.4, 64 x 10 17.6 us.
//
// Rounding: a Q4_0, Q8_0 or Q6_K weight d * sc * q is exact in f32 (11 + 7 + 6
// bits at most); a Q4_K weight d * sc * q - dmin * m is one fma of two exact
// products; the multiplication by scale rounds once.
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"

namespace qws {

__device__ unsigned g_err_embed;

constexpr int kEmbThreads = 160;
constexpr int kEmbRuns = 4;

__device__ __forceinline__ uint32_t ld_u16(const uint8_t* p) {
  return __ldg(reinterpret_cast<const unsigned short*>(p));
}
// four bytes at a 2-byte boundary
__device__ __forceinline__ uint32_t ld_u32_at2(const uint8_t* p) {
  return ld_u16(p) | (ld_u16(p + 2) << 16);
}

// Byte i of q, minus bias, as f32: put below 2^23's exponent and taken off again, both
// exact.  The conversion instruction runs at a quarter of this rate; with it, and 64-bit
// column arithmetic, the case above took 16.0 us (issue slots 63 % busy).
template <int kBias>
__device__ __forceinline__ float byte_float(uint32_t q, int i) {
  return __uint_as_float(__byte_perm(q, 0x4B000000u, 0x7440u + static_cast<uint32_t>(i))) -
         static_cast<float>(8388608 + kBias);
}

// values c .. c + 3 of a row (c % 4 == 0), before the scale
template <int kFmt>
__device__ __forceinline__ float4 embed_four(const uint8_t* row, uint32_t c) {
  float v[4];
  if constexpr (kFmt == QWS_Q4_0) {
    const uint8_t* b = row + c / 32 * 18;
    const uint32_t j = c % 32;
    const float d = half_bits_to_float(ld_u16(b));
    const uint32_t q = (ld_u32_at2(b + 2 + j % 16) >> (j >= 16 ? 4 : 0)) & 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = d * byte_float<8>(q, i);
  } else if constexpr (kFmt == QWS_Q8_0) {
    const uint8_t* b = row + c / 32 * 34;
    const float d = half_bits_to_float(ld_u16(b));
    const uint32_t q = ld_u32_at2(b + 2 + c % 32) ^ 0x80808080u;      // + 128
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = d * byte_float<128>(q, i);
  } else if constexpr (kFmt == QWS_Q4_K) {
    const uint8_t* b = row + c / 256 * 144;
    const uint32_t r = c % 256, s = r / 32;   // sub-block
    const uint4 hd = __ldg(reinterpret_cast<const uint4*>(b));
    const uint32_t sh = 8u * (s & 3u);
    const uint32_t a = (hd.y >> sh) & 255u, m = (hd.z >> sh) & 255u, h = (hd.w >> sh) & 255u;
    const uint32_t sc = s < 4 ? (a & 63u) : ((h & 15u) | ((a >> 6) << 4));
    const uint32_t mn = s < 4 ? (m & 63u) : ((h >> 4) | ((m >> 6) << 4));
    const float ds = half_bits_to_float(hd.x) * byte_float<0>(sc, 0);
    const float dm = half_bits_to_float(hd.x >> 16) * byte_float<0>(mn, 0);
    const uint32_t q = (__ldg(reinterpret_cast<const uint32_t*>(b + 16 + r / 64 * 32 + r % 32)) >>
                        ((s & 1u) ? 4 : 0)) & 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(ds, byte_float<0>(q, i), -dm);
  } else {
    const uint8_t* b = row + c / 256 * 210;
    const uint32_t r = c % 256, h = r / 128, l = r % 32, qt = r % 128 / 32;
    const float ds =
        half_bits_to_float(ld_u16(b + 208)) * byte_float<128>(__ldg(b + 192 + r / 16) ^ 0x80u, 0);
    const uint32_t lo = ld_u32_at2(b + 64 * h + 32 * (qt & 1u) + l) >> (4 * (qt >> 1));
    const uint32_t hi = ld_u32_at2(b + 128 + 32 * h + l) >> (2 * qt);
    const uint32_t q = (lo & 0x0F0F0F0Fu) | ((hi & 0x03030303u) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ds * byte_float<32>(q, i);
  }
  return make_float4(v[0], v[1], v[2], v[3]);
}

// grid.x = n_tokens * segs: a CTA covers 4 * kEmbThreads * kEmbRuns values of a row
template <int kFmt>
__global__ void __launch_bounds__(kEmbThreads)
    embed_kernel(const uint8_t* __restrict__ W, const int64_t* __restrict__ tokens,
                 float* __restrict__ out, int64_t vocab, uint32_t hidden, int64_t row_bytes,
                 uint32_t segs, float scale) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t t = blockIdx.x / segs, seg = blockIdx.x - t * segs;
  const int64_t tok = __ldg(tokens + t);
  const uint32_t c0 = (seg * kEmbRuns * kEmbThreads + threadIdx.x) * 4;     // hidden <= 2^24
  const bool known = tok >= 0 && tok < vocab;
  if (!known && threadIdx.x == 0) atomicOr(&g_err_embed, kErrTokenRange);
  float4 v[kEmbRuns];
#pragma unroll
  for (int r = 0; r < kEmbRuns; ++r) {
    const uint32_t c = c0 + static_cast<uint32_t>(r) * kEmbThreads * 4;
    v[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (known && c < hidden) v[r] = embed_four<kFmt>(W + tok * row_bytes, c);
  }
#pragma unroll
  for (int r = 0; r < kEmbRuns; ++r) {
    const uint32_t c = c0 + static_cast<uint32_t>(r) * kEmbThreads * 4;
    if (c < hidden)
      *reinterpret_cast<float4*>(out + static_cast<int64_t>(t) * hidden + c) =
          make_float4(v[r].x * scale, v[r].y * scale, v[r].z * scale, v[r].w * scale);
  }
}

cudaError_t launch_embed(int fmt, const uint8_t* W, const int64_t* tokens, float* out,
                         int64_t vocab, int64_t hidden, int64_t n_tokens, float scale,
                         cudaStream_t st) {
  const uint32_t segs = static_cast<uint32_t>((hidden / 4 + kEmbThreads * kEmbRuns - 1) /
                                              (kEmbThreads * kEmbRuns));
  const int64_t rb = row_bytes_of(fmt, hidden);
  const dim3 grid(static_cast<unsigned>(n_tokens * segs));
  switch (fmt) {
#define QWS_EMB_CASE(F)                                                                       \
  case F:                                                                                     \
    return pdl_launch(embed_kernel<F>, grid, kEmbThreads, 0, st, W, tokens, out, vocab,       \
                      static_cast<uint32_t>(hidden), rb, segs, scale);
    QWS_EMB_CASE(QWS_Q4_0) QWS_EMB_CASE(QWS_Q8_0) QWS_EMB_CASE(QWS_Q4_K) QWS_EMB_CASE(QWS_Q6_K)
#undef QWS_EMB_CASE
  }
  return cudaErrorInvalidValue;
}

unsigned read_clear_embed_errors() {
  unsigned v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_embed, sizeof(v)) != cudaSuccess) return 0;
  cudaMemcpyToSymbol(g_err_embed, &z, sizeof(z));
  return v;
}

}  // namespace qws
