// Position-rotated appends into BF16 pages and into the 4-bit cache, and the
// read-back of the 4-bit cache (include/oscar.h gives the definitions).

#include "oscar_paged.cuh"

namespace oscar {
namespace {

// One row of cosines and sines; the angle and its functions in fp64 (a far
// position times a frequency needs more than fp32's 24 bits), rounded once.
__global__ void __launch_bounds__(256) rope_table_kernel(float* table, int n_positions, int half, double log_theta) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)n_positions * half) return;
  const int p = (int)(i / half), f = (int)(i % half);
  double s, c;
  sincos((double)p * exp(-log_theta * (double)f / (double)half), &s, &c);
  table[(size_t)p * 2 * half + f] = (float)c;
  table[(size_t)p * 2 * half + half + f] = (float)s;
}

// How a kernel of this file turns a row.
enum { kTurnNone = 0, kTurnHalves = 1, kTurnPairs = 2 };

// ---------------------------------------------------------------- rows of 128 channels (BF16 in, BF16 out)
// Bound by the copies: four prompts of up to 8192 tokens (64 + 16 heads, 1.13 GB) in 171 us, 97% of the copy bandwidth.
// Eight threads take a row, two 16-byte pieces each, so that a piece and the
// one it turns with (64 / 32 channels on) sit in one thread.  A group of eight
// threads keeps its token's cosines and sines in registers and goes through
// `split`-th of the token's rows (q heads, then k, then v), four at a time.
template <int TURN, bool KV, int THREADS>
__device__ __forceinline__ void rope_rows(const RopeLaunch& a, int block, int b, int split) {
  const int t = threadIdx.x & 7;
  const int unit = block * (THREADS / 8) + (threadIdx.x >> 3);
  const int i = unit / split, sub = unit % split;
  int p0, n, row0;
  if (!token_span(a.tok, b, p0, n, row0, a.err, threadIdx.x == 0) || i >= n) return;
  const long long p = (long long)p0 + i;
  if (p < 0 || p >= (long long)a.pages.max_pages * kPage || (TURN != kTurnNone && p >= a.rope_positions)) {
    if (t == 0) set_error(a.err, kErrLength);
    return;
  }
  int phys = -1;
  if constexpr (KV) phys = page_of(a.pages, b, (int)(p >> 6), a.err, t == 0);
  const int np = TURN == kTurnNone ? 8 : a.rotary >> 4;  // threads that turn channels
  const bool turns = TURN != kTurnNone && t < np;
  const int c0 = t < np ? t : 2 * t, c1 = t < np ? t + np : 2 * t + 1;  // the thread's two pieces (np + 2 (t - np) + np = 2 t)
  float c[8], s[8];
  if (turns) {
    const float* row = a.rope + (size_t)p * a.rotary;
    const int half = a.rotary >> 1;
    if constexpr (TURN == kTurnHalves) {
      load8(c, row + 8 * t);
      load8(s, row + half + 8 * t);
    } else {
      load4(c, row + 4 * c0);
      load4(c + 4, row + 4 * c1);
      load4(s, row + half + 4 * c0);
      load4(s + 4, row + half + 4 * c1);
    }
  }
  const size_t tok = (size_t)row0 + i;
  const int R = a.Hq + (KV && phys >= 0 ? 2 * a.Hkv : 0);
  for (int r0 = sub; r0 < R; r0 += 4 * split) {
    uint4 x0[4], x1[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * split;
      if (r < R) {
        const uint16_t* src = r < a.Hq ? a.q + tok * a.q_stride + (size_t)r * kD
                              : r < a.Hq + a.Hkv ? a.k + tok * a.k_stride + (size_t)(r - a.Hq) * kD
                                                 : a.v + tok * a.v_stride + (size_t)(r - a.Hq - a.Hkv) * kD;
        x0[u] = reinterpret_cast<const uint4*>(src)[c0];
        x1[u] = reinterpret_cast<const uint4*>(src)[c1];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * split;
      if (r < R) {
        if (turns && r < a.Hq + a.Hkv) {
          if constexpr (TURN == kTurnHalves) {
            turn8(x0[u], x1[u], c, s);
          } else {
            turn4(x0[u], c, s);
            turn4(x1[u], c + 4, s + 4);
          }
        }
        const int h = r - a.Hq;
        uint16_t* dst = r < a.Hq ? a.q_out + tok * a.qo_stride + (size_t)r * kD
                                 : (h < a.Hkv ? a.k_pages : a.v_pages) +
                                       (((size_t)phys * a.Hkv + (h < a.Hkv ? h : h - a.Hkv)) * kPage + (p & 63)) * kD;
        reinterpret_cast<uint4*>(dst)[c0] = x0[u];
        reinterpret_cast<uint4*>(dst)[c1] = x1[u];
      }
    }
  }
}

template <int TURN>
__global__ void __launch_bounds__(256) rope_append_bf16_kernel(const __grid_constant__ RopeLaunch a, int split) {
  // (no early launch of what comes next: it gained nothing)
  griddep_wait();
  rope_rows<TURN, true, 256>(a, blockIdx.x, blockIdx.y, split);
}

// ---------------------------------------------------------------- the 4-bit cache
// x' = x H / sqrt(128) runs as H = H_16 (x) H_8: the factor over channel bits
// 0, 1, 3, 4 as m16n8k16 MMAs with a matrix of +-1 (exact products of bf16,
// fp32 sums), the factor over bits 2, 5, 6 as three add/subtract stages on a
// lane's own sums.  A warp takes 16 tokens of one head, the tile of the 4-bit
// layout, and the layout is such that each lane ends up with whole words of it.
//
// K: D = x H_16 with tokens as the MMA's rows: lane (r, tq) = (lane / 4,
// lane % 4) loads pieces tq + 4 M (M < 4) of rows r and r + 8 and holds the
// same rotated channels of the same rows.
// V: D = H_16 x^T with the channels as rows: the same loads, as the other
// operand, leave lane (c, tq) with channels of residue c of tokens 2 tq,
// 2 tq + 1, 2 tq + 8, 2 tq + 9, which is how the attention's P V reads them.
struct Tile4 {
  uint4 x[2][4];  // [row r, row r + 8][piece tq + 4 M]
};

template <int TURN>
__device__ __forceinline__ void turn_tile(Tile4& t, const RopeLaunch& a, int p_r, bool v0, bool v1, int tq) {
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    if (!(rh ? v1 : v0)) continue;
    const float* row = a.rope + (size_t)(p_r + 8 * rh) * a.rotary;
    const int half = a.rotary >> 1;
    if constexpr (TURN == kTurnHalves) {
      float c[8], s[8];
      load8(c, row + 8 * tq);
      load8(s, row + half + 8 * tq);
      if (a.rotary == 64) {
        turn8(t.x[rh][0], t.x[rh][1], c, s);
      } else {
        turn8(t.x[rh][0], t.x[rh][2], c, s);
        load8(c, row + 8 * tq + 32);
        load8(s, row + half + 8 * tq + 32);
        turn8(t.x[rh][1], t.x[rh][3], c, s);
      }
    } else {
#pragma unroll
      for (int M = 0; M < 4; ++M) {
        if (M >= 2 && a.rotary == 64) continue;
        float c[4], s[4];
        load4(c, row + 4 * (tq + 4 * M));
        load4(s, row + half + 4 * (tq + 4 * M));
        turn4(t.x[rh][M], c, s);
      }
    }
  }
}

constexpr float kMaxScale4 = 65504.0f;           // fp16's largest, the scale of a group that overflows it
constexpr float kMagic4 = 12582912.0f + 8.0f;    // 1.5 2^23 + 8: the sum's low bits are floor(x' / s) + 8
constexpr uint32_t kMagic4Bits = 0x4B400000u;

// Scale and multiplier of a group with maximum m of |sum| (before the 1 / sqrt(128)); `clips`: a
// quotient may leave 0..15 (a subnormal scale's rounding, or a scale cut at fp16's largest).
__device__ __forceinline__ __half scale4(float m, float& inv, bool& clips) {
  const float a = fminf(m * kInvSqrt128, kMaxScale4 * 7.5f);
  // a / 7.5: the product with 1 / 7.5, and what it lacks once more (the quotient to half a step of fp32)
  float q = a * (1.f / 7.5f);
  q = fmaf(fmaf(-7.5f, q, a), 1.f / 7.5f, q);
  const __half h = __float2half_rn(q);
  const float s = __half2float(h);
  inv = s > 0.f ? __fdividef(kInvSqrt128, s) : 0.f;  // (two steps of fp32, as the sums' own roundings)
  clips = clips || s < 6.2e-5f || m * kInvSqrt128 > kMaxScale4 * 7.5f;
  return h;
}

// Two codes' float sums 1.5 2^23 + code: one fma rounding down in place of a division, floor and conversion.
template <bool CLIP>
__device__ __forceinline__ float2 code4(float2 y, float2 inv) {
  float2 f = ffma2_rd(y, inv, make_float2(kMagic4, kMagic4));
  if constexpr (CLIP) {
    f.x = fminf(fmaxf(f.x, 12582912.0f), 12582927.0f);
    f.y = fminf(fmaxf(f.y, 12582912.0f), 12582927.0f);
  }
  return f;
}

// K words of rows r (rh 0) and r + 8: word M = nibbles n = 4 j0 + 2 j2 + j1 of channels with bits 5, 6 = M.
// d[2 M + b2][2 nt + rh] = channels (j1 = nt, j0 = x / y) of row r + 8 rh.
template <bool CLIP>
__device__ __forceinline__ void pack_k(const float2 (&d)[8][4], const float (&inv)[2][2], uint4 (&w)[2]) {
#pragma unroll
  for (int rh = 0; rh < 2; ++rh)
#pragma unroll
    for (int M = 0; M < 4; ++M) {
      uint32_t acc = 0u - kMagic4Bits * 0x11111111u;
      const float iv = inv[rh][M >> 1];
#pragma unroll
      for (int b2 = 0; b2 < 2; ++b2)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float2 f = code4<CLIP>(d[2 * M + b2][2 * nt + rh], make_float2(iv, iv));
          acc += __float_as_uint(f.x) << (4 * (2 * b2 + nt));
          acc += __float_as_uint(f.y) << (4 * (4 + 2 * b2 + nt));
        }
      word_of(w[rh], M) = acc;
    }
}

// V words m = 2 M + b2 of a lane: byte 2 (u % 2) + u / 8, nibble = channel bit 4.
// d[m][2 th + half] = tokens (2 tq, 2 tq + 1) + 8 th of the channel with bit 4 = half; inv[th][g] by token.
template <bool CLIP>
__device__ __forceinline__ void pack_v(const float2 (&d)[8][4], const float2 (&inv)[2][2], uint32_t (&w)[8]) {
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    uint32_t acc = 0u - kMagic4Bits * 0x11111111u;
#pragma unroll
    for (int th = 0; th < 2; ++th)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float2 f = code4<CLIP>(d[m][2 * th + hf], inv[th][m >> 2]);
        acc += __float_as_uint(f.x) << (4 * (2 * th + hf));
        acc += __float_as_uint(f.y) << (4 * (4 + 2 * th + hf));
      }
    w[m] = acc;
  }
}

__device__ __forceinline__ float max4(float m, float2 a, float2 b) {
  return fmaxf(fmaxf(m, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
}

// A warp's `per` heads (of K's, then V's) of one tile: the next head's rows are on their way while one is turned and
// rounded.  `sm`: 8 KB of the warp's own, two heads' rows, each lane's 16-byte pieces read by that lane alone.
constexpr int kAhead4 = 2;  // heads of a warp in shared memory
template <int TURN>
__device__ __forceinline__ void append_tiles4(const RopeLaunch& a, int unit, int b, int per, uint32_t sm) {
  const int lane = threadIdx.x & 31, r = lane >> 2, tq = lane & 3;
  const int groups = (2 * a.Hkv + per - 1) / per, tile = unit / groups;
  const int first = (unit - tile * groups) * per, last = min(first + per, 2 * a.Hkv);
  int p0, n, row0;
  if (!token_span(a.tok, b, p0, n, row0, a.err, lane == 0)) return;
  const int T = (max(p0, 0) >> 4) + tile;
  // the tile's new tokens [lo, hi), of those inside the tables
  const long long end = (long long)p0 + n;
  long long limit = (long long)a.pages.max_pages * kPage;
  if (TURN != kTurnNone && a.rope_positions < limit) limit = a.rope_positions;
  if (n > 0 && (p0 < 0 || end > limit) && lane == 0) set_error(a.err, kErrLength);
  const long long base = (long long)T * kTile4;
  const int lo = (int)max((long long)max(p0, 0) - base, 0ll);
  const int hi = (int)min(min(end, limit) - base, (long long)kTile4);
  if (hi <= lo || base >= limit) return;
  const int phys = page_of(a.pages, b, T >> 2, a.err, lane == 0);
  if (phys < 0) return;
  const bool v0 = r >= lo && r < hi, v1 = r + 8 >= lo && r + 8 < hi;
  const long long tok = (long long)row0 + (base - p0) + r;
  sm += 16 * lane;
  auto load = [&](int head) {
    const bool is_v = head >= a.Hkv;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const uint16_t* x = (is_v ? a.v + (size_t)(head - a.Hkv) * kD : a.k + (size_t)head * kD) + 8 * tq;
    const uint16_t* x0 = v0 ? x + tok * stride : x;
    const uint16_t* x1 = v1 ? x + (tok + 8) * stride : x;
    const uint32_t dst = sm + 4096 * (head % kAhead4);
#pragma unroll
    for (int M = 0; M < 4; ++M) {
      cp_async16(dst + 512 * M, x0 + 32 * M, v0);
      cp_async16(dst + 512 * (4 + M), x1 + 32 * M, v1);
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead4 - 1; ++i) {
    if (first + i < last) load(first + i);
    cp_async_commit();
  }
#pragma unroll 1
  for (int head = first; head < last; ++head) {
  if (head + kAhead4 - 1 < last) load(head + kAhead4 - 1);
  cp_async_commit();
  cp_async_wait<kAhead4 - 1>();
  const bool is_v = head >= a.Hkv;
  const int h = is_v ? head - a.Hkv : head;
  Tile4 t;
#pragma unroll
  for (int i = 0; i < 8; ++i) t.x[i >> 2][i & 3] = lds128(sm + 4096 * (head % kAhead4) + 512 * i);
  if constexpr (TURN != kTurnNone)
    if (!is_v) turn_tile<TURN>(t, a, (int)base + r, v0, v1, tq);
  uint8_t* blk = a.pages4 + ((size_t)phys * a.Hkv + h) * kBlock4Bytes + (size_t)(T & 3) * kTile4Bytes;
  float2 d[8][4];
  bool clips = false;
  if (!is_v) {
    // B[k][n]: k bit 0 = e, bits 1, 2 = tq, bit 3 = kh (channel bits 0, 3, 4, 1), n the same of the result
    const uint32_t s = signs_bf16(odd_bits(2 * tq & r), odd_bits((2 * tq + 1) & r));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int M = i >> 1, b2 = i & 1;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        mma_bf16_acc(acc, word_of(t.x[0][M], 2 * b2), word_of(t.x[1][M], 2 * b2), word_of(t.x[0][M], 2 * b2 + 1),
                     word_of(t.x[1][M], 2 * b2 + 1), s, nt ? s ^ 0x80008000u : s);
        d[i][2 * nt] = make_float2(acc[0], acc[1]);
        d[i][2 * nt + 1] = make_float2(acc[2], acc[3]);
      }
    }
    butterfly(d, 1);
    butterfly(d, 2);
    butterfly(d, 4);
    float inv[2][2];
    __half sc[2][2];
#pragma unroll
    for (int rh = 0; rh < 2; ++rh)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float m = 0.f;
#pragma unroll
        for (int i = 4 * g; i < 4 * g + 4; ++i) m = max4(m, d[i][rh], d[i][2 + rh]);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        sc[rh][g] = scale4(m, inv[rh][g], clips);
      }
    uint4 w[2];
    if (__any_sync(0xffffffffu, clips))
      pack_k<true>(d, inv, w);
    else
      pack_k<false>(d, inv, w);
#pragma unroll
    for (int rh = 0; rh < 2; ++rh)
      if (rh ? v1 : v0) {
        *reinterpret_cast<uint4*>(blk + 64 * (r + 8 * rh) + 16 * tq) = w[rh];
        if (tq == 0)
          *reinterpret_cast<__half2*>(blk + kTile4Scales + 4 * (r + 8 * rh)) = __halves2half2(sc[rh][0], sc[rh][1]);
      }
  } else {
    // A[row][k]: row bits = channel bits 0, 1, 3, 4; k bits = channel bits 0, 3, 4, 1
    const int c = r, base_s = ((c >> 2) & tq) & 1;
    const uint32_t s0 = signs_bf16(base_s, base_s ^ (c & 1));
    const uint32_t f1 = (tq >> 1) ? 0x80008000u : 0u, f2 = ((c >> 1) & 1) ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int M = i >> 1, b2 = i & 1;
#pragma unroll
      for (int th = 0; th < 2; ++th) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        mma_bf16_acc(acc, s0, s0 ^ f1, s0 ^ f2, s0 ^ f1 ^ f2, word_of(t.x[th][M], 2 * b2), word_of(t.x[th][M], 2 * b2 + 1));
        d[i][2 * th] = make_float2(acc[0], acc[1]);
        d[i][2 * th + 1] = make_float2(acc[2], acc[3]);
      }
    }
    butterfly(d, 1);
    butterfly(d, 2);
    butterfly(d, 4);
    float2 inv[2][2];
    __half2 sc[2][2];  // [th][even, odd token]: both groups
    __half hx[2][2], hy[2][2];
#pragma unroll
    for (int th = 0; th < 2; ++th)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float mx = 0.f, my = 0.f;
#pragma unroll
        for (int i = 4 * g; i < 4 * g + 4; ++i) {
          mx = fmaxf(mx, fmaxf(fabsf(d[i][2 * th].x), fabsf(d[i][2 * th + 1].x)));
          my = fmaxf(my, fmaxf(fabsf(d[i][2 * th].y), fabsf(d[i][2 * th + 1].y)));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, o));
        }
        hx[th][g] = scale4(mx, inv[th][g].x, clips);
        hy[th][g] = scale4(my, inv[th][g].y, clips);
      }
#pragma unroll
    for (int th = 0; th < 2; ++th) {
      sc[th][0] = __halves2half2(hx[th][0], hx[th][1]);
      sc[th][1] = __halves2half2(hy[th][0], hy[th][1]);
    }
    uint32_t w[8];
    if (__any_sync(0xffffffffu, clips))
      pack_v<true>(d, inv, w);
    else
      pack_v<false>(d, inv, w);
    uint8_t* vb = blk + kTile4V + 16 * lane;
    if (lo == 0 && hi == kTile4) {
      *reinterpret_cast<uint4*>(vb) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(vb + 512) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      // byte 2 (u % 2) + u / 8 of every word belongs to token u alone
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = 2 * tq + (q >> 1) + 8 * (q & 1);
        if (u >= lo && u < hi)
#pragma unroll
          for (int m = 0; m < 8; ++m) vb[512 * (m >> 2) + 4 * (m & 3) + q] = (uint8_t)(w[m] >> (8 * q));
      }
    }
    if (c == 0)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = 2 * tq + (q >> 1) + 8 * (q & 1);
        if (u >= lo && u < hi) *reinterpret_cast<__half2*>(blk + kTile4Scales + 64 + 4 * u) = sc[q & 1][q >> 1];
      }
  }
  }
}

// (128 registers and 16 warps an SM: with 96 and 20 warps the spills cost 331 us for 306, 131,072 tokens in and out.
// 147 us of it are the append's, 680 MB and 67 MB of the rope table; half of the issue slots are used: what is left
// is the latency of the table's rows and of the exchanges that find a group's maximum.)
template <int TURN>
__global__ void __launch_bounds__(128, 4) rope_append_int4_kernel(const __grid_constant__ RopeLaunch a, int kv_blocks,
                                                               int units, int per, int split) {
  extern __shared__ __align__(16) uint8_t sm[];
  griddep_wait();  // (and no early launch of what comes next, as above)
  if ((int)blockIdx.x >= kv_blocks) {  // the queries' rows
    rope_rows<TURN, false, 128>(a, blockIdx.x - kv_blocks, blockIdx.y, split);
    return;
  }
  const int warp = threadIdx.x >> 5, unit = blockIdx.x * 4 + warp;
  if (unit < units) append_tiles4<TURN>(a, unit, blockIdx.y, per, smem_u32(sm) + kAhead4 * 4096 * warp);
}

// ---------------------------------------------------------------- reading the 4-bit cache back
// The codes of a word as fp16 numbers c 2^-24 (pairs 0, 2: nibbles i and i + 4) and 16 c 2^-24 (pairs 1, 3).
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&v)[4]) {
  code_pairs(w, v[0], v[1]);
  code_pairs(w >> 8, v[2], v[3]);
}

__device__ __forceinline__ uint32_t signs_f16(int lo, int hi) {
  return 0x3C003C00u ^ ((uint32_t)lo << 15) ^ ((uint32_t)hi << 31);
}

// The transform back: the codes of 16 tokens as the MMA's rows (the signs of the ones that are 16 times larger are
// +-1/16; the levels' -7.5 add up to -7.5 x 16 in the column of ones alone, where the sum starts: all of it exact),
// the stages over bits 2 and 5 inside each group of 64, each group's scale, then the stage over bit 6.
// A warp takes `per` heads (of K's, then V's) of one tile in turn, the codes of the next ones on their way meanwhile.
// (131,072 tokens x 8 heads of K and V: 107 us, 93% of the copy bandwidth; 82 us, 93%, at 100,000.)
constexpr int kAheadRead = 4;
__global__ void __launch_bounds__(128, 4) int4_to_bf16_kernel(const __grid_constant__ Read4Launch a, int units, int per) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, r = lane >> 2, tq = lane & 3, b = blockIdx.y;
  const int unit = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int groups = (2 * a.Hkv + per - 1) / per, tile = unit / groups;
  const int first = (unit - tile * groups) * per, last = min(first + per, 2 * a.Hkv);
  const int p0 = a.pos[b], n = a.count[b];
  if (n <= 0) return;
  if (n > a.max_count) {
    if (lane == 0) set_error(a.err, kErrTokens);
    return;
  }
  const int T = (max(p0, 0) >> 4) + tile;
  const long long end = (long long)p0 + n, limit = (long long)min(a.from.max_pages, a.to.max_pages) * kPage;
  if ((p0 < 0 || end > limit) && lane == 0) set_error(a.err, kErrLength);
  const long long base = (long long)T * kTile4;
  const int lo = (int)max((long long)max(p0, 0) - base, 0ll);
  const int hi = (int)min(min(end, limit) - base, (long long)kTile4);
  if (hi <= lo || base >= limit) return;
  const int from = page_of(a.from, b, T >> 2, a.err, lane == 0), to = page_of(a.to, b, T >> 2, a.err, lane == 0);
  if (from < 0 || to < 0) return;
  const uint8_t* page = a.pages4 + (size_t)from * a.Hkv * kBlock4Bytes + (size_t)(T & 3) * kTile4Bytes;
  extern __shared__ __align__(16) uint8_t sm[];  // the heads ahead: [warp][kAheadRead] codes, scales
  const uint32_t ring = smem_u32(sm) + (threadIdx.x >> 5) * (kAheadRead * 1088);
  auto load = [&](int head) {
    if (head < last) {
      const bool is_v = head >= a.Hkv;
      const uint8_t* blk = page + (size_t)(is_v ? head - a.Hkv : head) * kBlock4Bytes;
      const uint8_t* cb = blk + (is_v ? kTile4V : 0) + 16 * lane;
      const uint32_t dst = ring + 1088 * (head % kAheadRead) + 16 * lane;
      cp_async16(dst, cb, true);
      cp_async16(dst + 512, cb + 512, true);
      if (lane < 4) cp_async16(dst + 1024, blk + kTile4Scales + (is_v ? 64 : 0) + 16 * lane, true);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kAheadRead - 1; ++i) load(first + i);
#pragma unroll 1
  for (int head = first; head < last; ++head) {
  const bool is_v = head >= a.Hkv;
  const int h = is_v ? head - a.Hkv : head;
  __syncwarp();
  load(head + kAheadRead - 1);
  cp_async_wait<kAheadRead - 1>();
  __syncwarp();
  const uint32_t stage = ring + 1088 * (head % kAheadRead);
  const uint4 w0 = lds128(stage + 16 * lane), w1 = lds128(stage + 512 + 16 * lane);
  float2 sc[2];
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    const uint32_t u = lds32(stage + 1024 + 4 * (r + 8 * rh));
    sc[rh] = __half22float2(*reinterpret_cast<const __half2*>(&u));
    sc[rh].x *= kInvSqrt128 * 16777216.f;
    sc[rh].y *= kInvSqrt128 * 16777216.f;
  }
  float2 d[8][4];  // [2 M + b2][2 nt + rh]
  // B[k][n] with n bits = channel bits 0, 3, 4 and nt = bit 1; k bits = bits 0, 3, 4, 1 (K) or 0, 1, 3, 4 (V)
  const int e0 = is_v ? ((tq >> 1) & (r >> 1)) & 1 : odd_bits(2 * tq & r);
  const uint32_t s = signs_f16(e0, e0 ^ (r & 1));
  const uint32_t flip_hi = is_v && ((r >> 2) & 1) ? 0x80008000u : 0u;           // k bit 3 against n (V)
  const uint32_t nt_lo = is_v && (tq & 1) ? 0x80008000u : 0u;                   // k bits against nt
  const uint32_t nt_hi = is_v ? nt_lo : 0x80008000u;
  uint32_t lev[2][4][4];  // K: [row half][word M][pair]
  if (!is_v) {
#pragma unroll
    for (int M = 0; M < 4; ++M) {
      codes4(word_of(w0, M), lev[0][M]);
      codes4(word_of(w1, M), lev[1][M]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t a0, a1, a2, a3;
    if (!is_v) {
      const int M = i >> 1, b2 = i & 1;
      a0 = lev[0][M][2 * b2], a1 = lev[1][M][2 * b2], a2 = lev[0][M][2 * b2 + 1], a3 = lev[1][M][2 * b2 + 1];
    } else {  // a word holds a 16-channel x 16-token block with the channels as rows: transpose its quarters
      uint32_t v[4];
      codes4(i < 4 ? word_of(w0, i) : word_of(w1, i - 4), v);
      a0 = movmatrix_trans(v[0]), a1 = movmatrix_trans(v[2]), a2 = movmatrix_trans(v[1]), a3 = movmatrix_trans(v[3]);
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const float first = nt == 0 && tq == 0 ? -7.5f * 16.f / 16777216.f : 0.f;
      float acc[4] = {first, 0.f, first, 0.f};
      mma_f16(acc, a0, a1, a2, a3, nt ? s ^ nt_lo : s, ((nt ? s ^ nt_hi : s) ^ flip_hi) - 0x10001000u);
      d[i][2 * nt] = make_float2(acc[0], acc[1]);
      d[i][2 * nt + 1] = make_float2(acc[2], acc[3]);
    }
  }
  butterfly(d, 1);
  butterfly(d, 2);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = i < 4 ? sc[j & 1].x : sc[j & 1].y;
      d[i][j] = fmul2(d[i][j], make_float2(f, f));
    }
  butterfly(d, 4);
  uint16_t* dst = (is_v ? a.v_pages : a.k_pages) + (((size_t)to * a.Hkv + h) * kPage + 16 * (T & 3)) * kD;
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    const int u = r + 8 * rh;
    if (u >= lo && u < hi)
#pragma unroll
      for (int M = 0; M < 4; ++M) {
        uint4 y;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // channels 2 q, 2 q + 1 of the piece: j1 = q % 2, j2 = q / 2
          const float2 f = d[2 * M + (q >> 1)][2 * (q & 1) + rh];
          word_of(y, q) = pack_bf16x2(f.x, f.y);
        }
        reinterpret_cast<uint4*>(dst + (size_t)u * kD)[tq + 4 * M] = y;
      }
  }
  }
}

int turn_of(const RopeLaunch& a) { return a.rotary == 0 ? kTurnNone : a.interleaved ? kTurnPairs : kTurnHalves; }

// Groups of eight threads that share a token's rows: enough of them to fill the GPU (256 groups per SM
// are resident), but not more, since each reads the token's cosines and sines again.
int split_of(const RopeLaunch& a, int rows) {
  int split = 1;
  while (split < 32 && 2 * split <= rows && (long long)a.tok.n_tokens * split < 256ll * a.num_sms) split *= 2;
  return split;
}

// Heads of a tile that a warp takes in turn, the next one's loads under the work on one: as many, up to eight, as
// leave a group for each of the 16 warps that an SM holds (131,072 tokens of 8 heads in and out, with one head ahead:
// 385 us with one head a warp, 298 with two, 274 with four, 268 with eight; a short call needs every warp).
int heads_of(long long tiles, int num_sms) {
  int per = 1;
  while (per < 8 && tiles >= 2 * per * 16ll * num_sms) per *= 2;
  return per;
}

}  // namespace

cudaError_t launch_rope_table(float* table, int32_t n_positions, int32_t rotary, double theta, cudaStream_t stream) {
  const long long n = (long long)n_positions * (rotary / 2);
  rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(table, n_positions, rotary / 2, log(theta));
  return cudaGetLastError();
}

cudaError_t launch_rope_append_bf16(const RopeLaunch& a, cudaStream_t stream) {
  const int split = split_of(a, a.Hq + 2 * a.Hkv);
  const dim3 grid((unsigned)(((long long)a.tok.max_tokens * split + 31) / 32), a.pages.batch);
  const void* fn[3] = {reinterpret_cast<const void*>(rope_append_bf16_kernel<kTurnNone>),
                       reinterpret_cast<const void*>(rope_append_bf16_kernel<kTurnHalves>),
                       reinterpret_cast<const void*>(rope_append_bf16_kernel<kTurnPairs>)};
  RopeLaunch la = a;
  int sp = split;
  void* args[] = {&la, &sp};
  return launch_pdl(fn[turn_of(a)], grid, dim3(256), 0, stream, args);
}

cudaError_t launch_rope_append_int4(const RopeLaunch& a, cudaStream_t stream) {
  const int split = a.Hq ? split_of(a, a.Hq) : 1;
  const long long tiles = ((long long)a.tok.max_tokens + 2 * kTile4 - 2) / kTile4;
  const int per = heads_of(tiles * a.pages.batch * 2 * a.Hkv, a.num_sms);
  const long long units = tiles * ((2 * a.Hkv + per - 1) / per);
  const long long kv = (units + 3) / 4, qb = a.Hq ? ((long long)a.tok.max_tokens * split + 15) / 16 : 0;
  if (kv + qb > INT32_MAX || units > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(kv + qb), a.pages.batch);
  const void* fn[3] = {reinterpret_cast<const void*>(rope_append_int4_kernel<kTurnNone>),
                       reinterpret_cast<const void*>(rope_append_int4_kernel<kTurnHalves>),
                       reinterpret_cast<const void*>(rope_append_int4_kernel<kTurnPairs>)};
  RopeLaunch la = a;
  int kv_blocks = (int)kv, n_units = (int)units, pr = per, sp = split;
  void* args[] = {&la, &kv_blocks, &n_units, &pr, &sp};
  return launch_pdl(fn[turn_of(a)], grid, dim3(128), 4 * kAhead4 * 4096, stream, args);
}

cudaError_t launch_int4_to_bf16(const Read4Launch& a, cudaStream_t stream) {
  const long long tiles = ((long long)a.max_count + 2 * kTile4 - 2) / kTile4;
  int per = heads_of(tiles * a.from.batch * 2 * a.Hkv, a.num_sms);
  const long long units = tiles * ((2 * a.Hkv + per - 1) / per);
  if (units > INT32_MAX - 8) return cudaErrorInvalidValue;
  Read4Launch la = a;
  int n_units = (int)units;
  void* args[] = {&la, &n_units, &per};
  return launch_pdl(reinterpret_cast<const void*>(int4_to_bf16_kernel), dim3((unsigned)((units + 3) / 4), a.from.batch),
                    dim3(128), 4 * kAheadRead * 1088, stream, args);
}

}  // namespace oscar
