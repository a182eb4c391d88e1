// Device helpers of the one-kind paged caches: spans of new tokens, page
// lookups, the pieces of the 4-bit layout (include/oscar.h) and the 128-point
// Hadamard transform on the tensor cores.
#pragma once

#include "oscar_device.cuh"
#include "oscar_internal.h"
#include "oscar_paged.h"

namespace oscar {
namespace {

// Request b's tokens: the first one's position, how many, and their first row.
__device__ __forceinline__ bool token_span(const TokenRefs& t, int b, int& p0, int& n, int& row0, unsigned* err,
                                           bool report) {
  p0 = t.pos[b];
  row0 = b;
  n = 1;
  if (t.cu != nullptr) {
    const int lo = t.cu[b], hi = t.cu[b + 1];
    if (lo < 0 || hi < lo || hi > t.n_tokens || hi - lo > t.max_tokens) {
      if (report) set_error(err, kErrTokens);
      return false;
    }
    row0 = lo;
    n = hi - lo;
  }
  return true;
}

// Physical page of logical page lp (known to be inside the table) of request b, -1 with an error bit if bad.
__device__ __forceinline__ int page_of(const PageRefs& p, int b, int lp, unsigned* err, bool report) {
  const int phys = p.table[(size_t)b * p.max_pages + lp];
  if (phys >= 0 && phys < p.num_pages) return phys;
  if (report) set_error(err, kErrPage);
  return -1;
}

// Asynchronous copies to shared memory; zeros where `real` is false (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const unsigned n = real ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool real) {
  const unsigned n = real ? 8u : 0u;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(p) : "memory");
  return v;
}

// The codes of a 4-bit word as 16-bit floats without exponent bits, whole numbers of their smallest subnormals
// (fp16: 2^-24; bf16: 2^-133, on into the first binade): pairs (2 h, 2 h + 1) of a word, x = w >> 8 h, as c and 16 c
__device__ __forceinline__ void code_pairs(uint32_t x, uint32_t& lo, uint32_t& hi) {
  lo = x & 0x000F000Fu;
  hi = x & 0x00F000F0u;
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ uint32_t& word_of(uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// (x c - y s, y c + x s) for two pairs at once, each product and sum rounded once, as written: a fused product would
// round the two terms differently, and its bits would not be those of the formula in elementary operations.
__device__ __forceinline__ void turn2(float2& x, float2& y, float2 c, float2 s) {
  const float2 z = make_float2(-y.x, -y.y), u = fadd2(fmul2(x, c), fmul2(z, s));
  y = fadd2(fmul2(y, c), fmul2(x, s));
  x = u;
}

// Turn eight pairs: a = (x0..x7), b = (y0..y7) as bf16, c and s their cosines and sines.
__device__ __forceinline__ void turn8(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = make_float2(bf16_lo(word_of(a, i)), bf16_hi(word_of(a, i)));
    float2 y = make_float2(bf16_lo(word_of(b, i)), bf16_hi(word_of(b, i)));
    turn2(x, y, make_float2(c[2 * i], c[2 * i + 1]), make_float2(s[2 * i], s[2 * i + 1]));
    word_of(a, i) = pack_bf16x2(x.x, x.y);
    word_of(b, i) = pack_bf16x2(y.x, y.y);
  }
}

// Turn four adjacent pairs held in one 16-byte piece.
__device__ __forceinline__ void turn4(uint4& a, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    float2 x = make_float2(bf16_lo(word_of(a, i)), bf16_lo(word_of(a, i + 1)));
    float2 y = make_float2(bf16_hi(word_of(a, i)), bf16_hi(word_of(a, i + 1)));
    turn2(x, y, make_float2(c[i], c[i + 1]), make_float2(s[i], s[i + 1]));
    word_of(a, i) = pack_bf16x2(x.x, y.x);
    word_of(a, i + 1) = pack_bf16x2(x.y, y.y);
  }
}

__device__ __forceinline__ void load8(float (&v)[8], const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void load4(float* v, const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}

__device__ __forceinline__ int odd_bits(int x) { return __popc((unsigned)x) & 1; }

// Two bf16 signs: +-1 with the low half's sign bit lo and the high half's hi.
__device__ __forceinline__ uint32_t signs_bf16(int lo, int hi) {
  return 0x3F803F80u ^ ((uint32_t)lo << 15) ^ ((uint32_t)hi << 31);
}

// The add/subtract stages over bits 2, 5, 6: d[2 M + b2] is combination (M = bits 5, 6; b2 = bit 2).
template <int N>
__device__ __forceinline__ void butterfly(float2 (&d)[8][N], int stage) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!(i & stage))
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float2 x = d[i][j], y = d[i | stage][j];
        d[i][j] = fadd2(x, y);
        d[i | stage][j] = ffma2(y, make_float2(-1.f, -1.f), x);
      }
}

}  // namespace
}  // namespace oscar
