// Read-back of the mixed cache into BF16 pages (include/oscar.h gives the
// definition): sink and recent rows as they are, history rows from their 2-bit
// codes back in the original basis, x = x' R^T.
//
// x'_j = (c_j - 1.5) s_g for a channel j of group g, so with the levels
// l = c - 1.5 (exact in fp16)
//   x_i = s_0 sum_(j < 64) l_j R_ij + s_1 sum_(j >= 64) l_j R_ij:
// two products over 64 channels on the tensor cores, whose sums the scales meet
// in fp32.  R enters as two fp16 terms (off by at most 2^-24; one alone, by up
// to 2^-12 of an entry, would add an eighth of the result's own rounding), the
// products are exact, and x is rounded once, to bf16.
//
// A tile is 128 rows (two pages) of one (request, KV head) and one matrix: D_g
// [128 rows][128 channels] = L_g [128][64] R_g^T as tcgen05 MMAs (M 128, N 128,
// K 16).  Persistent blocks, one per SM, every other one for V:
//   warps 0-7, 8-15   results, of every other tile: half a row of both sums a
//                thread, scaled and added; whole pages of history rows go out by
//                TMA, the rows of others one by one
//   warps 16-19  unpack 32 bytes of codes a thread into the next tile's operand
//   warp 20      looks up the tiles that there are, 32 at a time, and copies their codes and
//                scales (one bulk copy a page) into a ring of kRdStages
//   warp 21      one thread issues the products
// with two operands, two pairs of sums in tensor memory and two results, so that
// a tile is unpacked while the one before is multiplied and the one before that
// is written.
// R's image (64 KB, the channels in the order in which the codes unpack) is laid
// out by oscar_load_rotation and copied once a block.

#include "oscar_paged.cuh"
#include "oscar_prompt.h"

#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

namespace oscar {
namespace {

constexpr int kRdThreads = 22 * 32;
constexpr int kRdUnpack = 16, kRdCopy = 20, kRdMma = 21;  // warps
constexpr int kRdStages = 6;
constexpr int kRdPart = 2304;  // a page's codes and scales of one matrix
constexpr uint32_t kRdR = 0;                        // [group of channels][term][128 rows][128 B]
constexpr uint32_t kRdA = 65536;                    // operands: [two in turn][group of channels][128 rows][128 B]
constexpr uint32_t kRdO = kRdA + 65536;             // results: [two in turn][64 channels][128 rows][128 B]
constexpr uint32_t kRdStage = kRdO + 65536;         // [stage][2 pages][codes, scales]
constexpr uint32_t kRdBars = kRdStage + kRdStages * 2 * kRdPart;
constexpr uint32_t kRdDesc = kRdBars + 256;
constexpr size_t kRdSmem = kRdDesc + kRdStages * 64 + 1024;  // + slack to align
static_assert(kBlockBytes == 2 * kRdPart && kVCodes == kRdPart && kKScales == 2048, "a block's halves");

struct ReadTile {
  int b, h;      // b < 0: no more tiles
  int p0;        // position of the tile's first row
  int lo, hi;    // positions that are written
  int hlo, hhi;  // positions that lie in the history
  int dst[2];    // BF16 page of either half (-1: none)
  int src;       // bit i: the codes of page i are there
  const uint16_t* rows[2];  // where either half's first row would lie in the sink or recent pool (null: not read)
};
static_assert(sizeof(ReadTile) <= 64, "a ring slot");

// A request's rows, and how many tiles (per head) they touch.
struct ReadSpan {
  int pos, len;  // of its first row; the cache's
  int end;       // behind its last row that is written
  int tiles;
};
__device__ __forceinline__ ReadSpan read_span(const Read2Launch& a, int b, bool report) {
  ReadSpan s;
  s.pos = a.pos[b];
  const int n = a.count[b];
  s.len = max(a.ctx_len[b], 0);
  s.end = s.tiles = 0;
  if (n <= 0) return s;
  if (n > a.max_count) {
    if (report) set_error(a.err, kErrTokens);
    return s;
  }
  const long long end = (long long)s.pos + n, limit = min((long long)s.len, (long long)a.to.max_pages * kPage);
  if (report && (s.pos < 0 || end > limit)) set_error(a.err, kErrLength);
  const int first = max(s.pos, 0) & ~(kPage - 1);
  s.end = (int)max(min(end, limit), 0ll);
  s.tiles = s.end > first ? (s.end - first - 1) / (2 * kPage) + 1 : 0;
  return s;
}

// What the k-th tile of request b and head h reads and writes.  Loads first, so that they travel together.
__device__ __forceinline__ void read_tile(const Read2Launch& a, int b, int h, int k, const ReadSpan& s, bool is_v, ReadTile& t,
                                          int (&blk)[2]) {
  const CacheRefs& c = a.from;
  const unsigned Hkv = (unsigned)c.num_kv_heads;
  t.b = b;
  t.h = h;
  const int pos = s.pos, len = s.len;
  const int sink = c.sink_page[t.b], slot = c.recent_table == nullptr ? c.ring_slot[t.b] : -1;
  const long long first = ((max(pos, 0) >> 6) + 2ll * k) * kPage;
  t.p0 = (int)first;
  t.lo = max(pos, t.p0);
  t.hi = (int)min((long long)s.end, first + 2 * kPage);
  t.hlo = kSink;
  t.hhi = len - kRecent;
  t.src = 0;
  const int lp0 = t.p0 >> 6;
  int to[2] = {-1, -1}, from[2] = {-1, -1}, recent[2] = {-1, -1};  // the tables' entries
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (lp0 + i < a.to.max_pages) to[i] = a.to.table[(size_t)t.b * a.to.max_pages + lp0 + i];
    if (lp0 + i < c.max_pages) {
      from[i] = c.page_table[(size_t)t.b * c.max_pages + lp0 + i];
      if (c.recent_table != nullptr) recent[i] = c.recent_table[(size_t)t.b * c.max_pages + lp0 + i];
    }
  }
  unsigned errors = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int lp = lp0 + i;
    const int p0 = max(lp * kPage, t.lo), p1 = (int)min(first + (i + 1) * kPage, (long long)t.hi);
    t.dst[i] = blk[i] = -1;
    t.rows[i] = nullptr;
    if (p0 >= p1) continue;
    if (to[i] < 0 || to[i] >= a.to.num_pages) {
      errors |= kErrPage;
      continue;
    }
    t.dst[i] = to[i];
    const bool history = max(p0, t.hlo) < min(p1, t.hhi), table = lp != 0 && (history || c.recent_table != nullptr);
    if (table && lp >= c.max_pages) {
      errors |= kErrLength;
      continue;
    }
    if (lp == 0) {
      if (sink < 0 || sink >= c.num_sink)
        errors |= kErrSink;
      else
        t.rows[i] = (is_v ? c.v_sink : c.k_sink) + ((size_t)sink * Hkv + t.h) * kSink * kD;
    } else if (p1 > t.hhi) {  // in the recent window: row p % 64 of its page, or (p - 64) % 256 of the ring
      const int place = c.recent_table != nullptr ? recent[i] : slot;
      if (place < 0 || place >= c.num_ring)
        errors |= kErrRing;
      else
        t.rows[i] = (is_v ? c.v_ring : c.k_ring) +
                    (c.recent_table != nullptr ? ((size_t)place * Hkv + t.h) * kPage
                                               : ((size_t)place * Hkv + t.h) * kRecent + (lp * kPage - kSink) % kRecent) * kD;
    }
    if (!history) continue;
    if (from[i] < 0 || from[i] >= c.num_pages) {
      errors |= kErrPage;
      continue;
    }
    blk[i] = from[i];
    t.src |= 1 << i;
  }
  if (errors != 0) set_error(a.err, errors);
}

// The 16 codes of a word as levels c - 1.5: pair n is the fields at bits 2 n and 2 n + 16.  Three of a word's fields
// and the first of the next byte lie within the mantissa of 1024 (0x6400) as they are.
__device__ __forceinline__ void levels16(uint32_t w, uint32_t (&h)[8]) {
  auto part = [](uint32_t x, uint32_t mask, float scale, float base) {
    const uint32_t y = (x & mask) | 0x64006400u;
    return h2_as_u32(__hfma2(*reinterpret_cast<const __half2*>(&y), __float2half2_rn(scale), __float2half2_rn(base)));
  };
  const uint32_t v = w >> 8;
  h[0] = part(w << 2, 0x000C000Cu, 0.25f, -257.5f);
  h[1] = part(w, 0x000C000Cu, 0.25f, -257.5f);
  h[2] = part(w, 0x00300030u, 0.0625f, -65.5f);
  h[3] = part(w, 0x00C000C0u, 0.015625f, -17.5f);
  h[4] = part(w, 0x03000300u, 0.00390625f, -5.5f);
  h[5] = part(v, 0x000C000Cu, 0.25f, -257.5f);
  h[6] = part(v, 0x00300030u, 0.0625f, -65.5f);
  h[7] = part(v, 0x00C000C0u, 0.015625f, -17.5f);
}

// Chunk c (16 bytes) of row r of an operand or result in the 128-byte swizzle.
__device__ __forceinline__ uint4* sw128_chunk(uint8_t* base, int r, int c) {
  return reinterpret_cast<uint4*>(base + r * 128 + ((c ^ (r & 7)) << 4));
}

// Thread u of 256: its 16 bytes of the tile's codes into the operand (both groups of channels).  Within a group the
// channels go in the order in which a word's pairs come out: K 16 tq + 2 n + hi for channel 16 (n % 4) + 4 tq + n / 4 + 2 hi,
// V 8 jl + 2 n + hi for channel 16 n + 8 hi + jl.
template <bool IS_V>
__device__ __forceinline__ void unpack(const uint8_t* stage, uint8_t* op, int u) {
  const int T = u >> 5, lane = u & 31, x = lane >> 2, y = lane & 3;
  const uint4 w = *reinterpret_cast<const uint4*>(stage + (T >> 2) * kRdPart + (T & 3) * 512 + 16 * lane);
#pragma unroll
  for (int u3 = 0; u3 < 2; ++u3) {
    const uint32_t w0 = word_of(w, 2 * u3), w1 = word_of(w, 2 * u3 + 1);
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (!IS_V) {  // words of one row: its two groups
        levels16(k ? w1 : w0, h);
        const int row = 16 * T + 8 * u3 + x;
        *sw128_chunk(op + 16384 * k, row, 2 * y) = make_uint4(h[0], h[1], h[2], h[3]);
        *sw128_chunk(op + 16384 * k, row, 2 * y + 1) = make_uint4(h[4], h[5], h[6], h[7]);
      } else {  // halves of two words: a row's eight fields, the low ones of group 0
        levels16(__byte_perm(w0, w1, k ? 0x7632 : 0x5410), h);
        const int row = 16 * T + 8 * u3 + 2 * y + k;
        *sw128_chunk(op, row, x) = make_uint4(h[0], h[1], h[2], h[3]);
        *sw128_chunk(op + 16384, row, x) = make_uint4(h[4], h[5], h[6], h[7]);
      }
    }
  }
}

// 16 columns of this thread's lane from each of two places, one wait (32 at once spill).
__device__ __forceinline__ void tmem_ld16x2(uint32_t tx, uint32_t ty, float (&x)[16], float (&y)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3]), "=f"(y[4]), "=f"(y[5]), "=f"(y[6]), "=f"(y[7]), "=f"(y[8]), "=f"(y[9]), "=f"(y[10]), "=f"(y[11]), "=f"(y[12]), "=f"(y[13]), "=f"(y[14]), "=f"(y[15])
      : "r"(tx), "r"(ty)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const void* tmap, int c0, int c1, int c2, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }

__device__ __forceinline__ void bulk_copy_s2g(void* dst, const void* src, unsigned bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}

// f(row, rows, place) for the pieces of the BF16 rows [first, end) of a tile's half i, as they pass through the result's
// place for that half: 32 rows in either of its two parts.
template <typename F>
__device__ __forceinline__ void bf16_pieces(int i, int first, int end, F f) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r0 = max(first, 32 * k), r1 = min(end, 32 * k + 32);
    if (r0 < r1) f(r0, r1 - r0, (uint32_t)(16384 * k + 8192 * i + (r0 - 32 * k) * 256));
  }
}

__global__ void __launch_bounds__(kRdThreads, 1)
    int2_to_bf16_kernel(const __grid_constant__ Read2Launch a, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
  extern __shared__ uint8_t rd_raw[];
  const uint32_t raw = smem_u32(rd_raw);
  uint8_t* sm = rd_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kRdBars);  // [stages] a tile's description and codes are there
  uint64_t* empty = full + kRdStages;                           // [stages] they are read
  uint64_t* afull = empty + kRdStages;                          // [2] an operand is unpacked
  uint64_t* aempty = afull + 2;                                 // [2] it is read
  uint64_t* tfull = aempty + 2;                                 // [2] a tile's sums are complete
  uint64_t* tempty = tfull + 2;                                 // [2] they are read
  uint64_t* rfull = tempty + 2;                                 // R's image is there
  uint64_t* brows = rfull + 1;                                  // [2] a tile's BF16 rows are there
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(brows + 2);
  volatile unsigned* dead = reinterpret_cast<volatile unsigned*>(tmem_at + 1);  // [2] the tile in front of which a result warp gave up
  ReadTile* desc = reinterpret_cast<ReadTile*>(sm + kRdDesc);
  static_assert((2 * kRdStages + 11) * 8 + 12 <= 256, "the barriers' place");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool is_v = (blockIdx.x & 1) != 0;
  const unsigned cta = blockIdx.x >> 1, n_cta = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRdStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4 + 8);  // unpacking and result warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&afull[i], 4);
      mbar_init(&aempty[i], 1);
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
      mbar_init(&brows[i], 1);
    }
    mbar_init(rfull, 1);
    dead[0] = dead[1] = 0;
    fence_mbar_init();
  }
  if (warp == kRdMma) tmem_alloc(tmem_at, 512);  // all of it, so its base is column 0
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  bool ok = true;

  if (warp == kRdCopy) {
    if (lane == 0) {  // (R does not depend on the work ahead in the stream: oscar_load_rotation returns with its copies complete)
      mbar_arrive_expect_tx(rfull, 65536);
      bulk_copy_g2s(sm + kRdR, a.r_image + (is_v ? 32768 : 0), 65536, rfull);
    }
    griddep_wait();
    griddep_launch_dependents();
    unsigned it = 0;
    // The tiles that there are, request by request (32 at a time, a lane each), and of these every n_cta-th: shares of a
    // ragged batch differ by a tile (28 requests of 100 to 4096, each with as many numbers as the longest has tiles: 44
    // for the busiest block, 39 on average, and 54.0 us for 52.7).
    unsigned idx = cta + (unsigned)lane * n_cta, before = 0;  // this lane's next tile; tiles of the requests before
    ReadSpan span = {0, 0, 0, 0};
    unsigned upto = 0, window = 0;
    for (int from = -32; ok;) {
      if (__all_sync(0xffffffffu, idx >= before + window)) {
        before += window;
        from += 32;
        if (from >= a.from.batch) break;
        span.tiles = 0;
        if (from + lane < a.from.batch) span = read_span(a, from + lane, blockIdx.x == 0);
        upto = (unsigned)span.tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        window = __shfl_sync(0xffffffffu, upto, 31) * (unsigned)a.from.num_kv_heads;
        continue;
      }
      ReadTile t;
      int blk[2];
      const bool some = idx < before + window;
      const unsigned r = some ? idx - before : 0u, q = r / (unsigned)a.from.num_kv_heads;
      int owner = 0;  // the first lane whose requests, up to its own, have more than q tiles
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (__shfl_sync(0xffffffffu, upto, owner + o - 1) <= q) owner += o;
      ReadSpan s;
      s.pos = __shfl_sync(0xffffffffu, span.pos, owner);
      s.len = __shfl_sync(0xffffffffu, span.len, owner);
      s.end = __shfl_sync(0xffffffffu, span.end, owner);
      const unsigned first = __shfl_sync(0xffffffffu, upto - (unsigned)span.tiles, owner);
      if (some) {
        read_tile(a, from + owner, (int)(r % (unsigned)a.from.num_kv_heads), (int)(q - first), s, is_v, t, blk);
        idx += 32u * n_cta;
      }
      unsigned left = __ballot_sync(0xffffffffu, some);
      for (; left != 0u && ok; left &= left - 1u, ++it) {
        const unsigned stage = it % kRdStages;
        ok = __all_sync(0xffffffffu, mbar_wait_timed(&empty[stage], ((it / kRdStages) & 1) ^ 1, kWaitNs));
        if (ok && lane == __ffs(left) - 1) {  // (the lane that looked the tile up)
          desc[stage] = t;
          mbar_arrive_expect_tx(&full[stage], (unsigned)kRdPart * __popc(t.src));
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (t.src >> i & 1)
              bulk_copy_g2s(sm + kRdStage + (stage * 2 + i) * kRdPart,
                            a.from.pages + ((size_t)blk[i] * a.from.num_kv_heads + t.h) * kBlockBytes + (is_v ? kRdPart : 0),
                            kRdPart, &full[stage]);
        }
        __syncwarp();
      }
    }
    for (int k = 0; k < 2 && ok; ++k, ++it) {  // the end, for the warps of either result
      const unsigned stage = it % kRdStages;
      ok = __all_sync(0xffffffffu, mbar_wait_timed(&empty[stage], ((it / kRdStages) & 1) ^ 1, kWaitNs));
      if (ok && lane == 0) {
        desc[stage].b = -1;
        desc[stage].src = 0;
        mbar_arrive(&full[stage]);
      }
      __syncwarp();
    }
    if (!ok) {
      if (lane == 0) set_error(a.err, kErrTimeout);
      for (unsigned i = it > kRdStages ? it - kRdStages : 0; i < it; ++i)  // copies in flight land before the block ends
        mbar_wait_timed(&full[i % kRdStages], (i / kRdStages) & 1, kWaitNs);
    }
    mbar_wait_timed(rfull, 0, kWaitNs);
  } else if (warp == kRdMma) {
    constexpr uint32_t idesc = umma_idesc_f16_f32(128, 128);
    const uint64_t ad = umma_desc_sw128(smem_u32(sm + kRdA)), rd = umma_desc_sw128(smem_u32(sm + kRdR));
    ok = __all_sync(0xffffffffu, mbar_wait_timed(rfull, 0, kWaitNs));
    unsigned it = 0;
    for (; ok; ++it) {
      const unsigned buf = it & 1, stage = it % kRdStages;
      ok = __all_sync(0xffffffffu, mbar_wait_timed(&afull[buf], (it >> 1) & 1, kWaitNs));
      if (!ok || desc[stage].b < 0) break;  // (the stage is given back behind the products)
      ok = __all_sync(0xffffffffu, mbar_wait_timed(&tempty[buf], ((it >> 1) & 1) ^ 1, kWaitNs));
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        if (desc[stage].src) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f16(256 * buf + 128 * g, ad + (32768 * buf + 16384 * g + 32 * k) / 16,
                         rd + (32768 * g + 16384 * term + 32 * k) / 16, idesc, term > 0 || k > 0);
        }
        umma_commit(&aempty[buf]);
        umma_commit(&tfull[buf]);
      }
      __syncwarp();
    }
    if (!ok) {
      if (lane == 0) set_error(a.err, kErrTimeout);
      if (it > 0) mbar_wait_timed(&tfull[(it - 1) & 1], ((it - 1) >> 1) & 1, kWaitNs);  // products in flight end first
    }
  } else if (warp >= kRdUnpack) {
    const int u = threadIdx.x - 32 * kRdUnpack;
    for (unsigned it = 0; ok; ++it) {
      const unsigned buf = it & 1, stage = it % kRdStages;
      ok = __all_sync(0xffffffffu, mbar_wait_timed(&full[stage], (it / kRdStages) & 1, kWaitNs) &&
                                       mbar_wait_timed(&aempty[buf], ((it >> 1) & 1) ^ 1, kWaitNs));
      if (!ok) break;
      const bool end = desc[stage].b < 0;
      if (!end && desc[stage].src != 0) {
        const uint8_t* codes = sm + kRdStage + stage * 2 * kRdPart;
        uint8_t* op = sm + kRdA + buf * 32768;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (is_v)
            unpack<true>(codes, op, u + 128 * k);
          else
            unpack<false>(codes, op, u + 128 * k);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&empty[stage]);
        mbar_arrive(&afull[buf]);
      }
      if (end) break;
    }
    if (!ok && lane == 0) set_error(a.err, kErrTimeout);
  } else {
    griddep_wait();
    const int buf = warp >> 3, q = warp & 3, hf = (warp >> 2) & 1, row = 32 * q + lane, pg = q >> 1;
    const bool issuer = (warp & 7) == 0 && lane == 0;
    uint16_t* pool = is_v ? a.v_pages : a.k_pages;
    unsigned phase = 0;  // (issuer) of the BF16 rows
    for (unsigned it = buf;; it += 2) {
      const unsigned stage = it % kRdStages;
      ok = __all_sync(0xffffffffu, mbar_wait_timed(&full[stage], (it / kRdStages) & 1, kWaitNs));
      const ReadTile& d = desc[stage];
      const bool end = ok && d.b < 0;
      ok = ok && (end || __all_sync(0xffffffffu, mbar_wait_timed(&tfull[buf], (it >> 1) & 1, kWaitNs)));
      tc_fence_after();
      // (a stage is held until its products are complete)
      const int h = d.h, lo = d.lo, hi = d.hi, hlo = d.hlo, hhi = d.hhi, p0 = d.p0, src = d.src;
      const int dst0 = d.dst[0], dst1 = d.dst[1];
      const uint16_t *const rows0 = d.rows[0], *const rows1 = d.rows[1];
      const __half2 scale = *reinterpret_cast<const __half2*>(sm + kRdStage + (stage * 2 + pg) * kRdPart + 2048 + 4 * (row & 63));
      __syncwarp();
      if (lane == 0) {
        if (!ok)
          dead[buf] = it + 1;
        else if (!end)
          mbar_arrive(&empty[stage]);
      }
      if (issuer) bulk_wait_read();  // the result of this buffer's tile before is read
      group_sync(1 + buf, 256);
      if ((dead[buf] != 0 && dead[buf] <= it + 1) || end) break;  // all of the tile's warps, or none
      // BF16 rows of either half, on their way while the others are worked out: f(half, row, rows, place)
      const int held = (rows0 != nullptr) | (rows1 != nullptr) << 1;
      auto bf16_rows_of = [&](auto f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pp = p0 + i * kPage, first = max(pp == 0 ? lo : max(lo, hhi), pp) - pp;
          if (held >> i & 1)
            bf16_pieces(i, first, min(hi - pp, kPage), [&](int r, int n, uint32_t place) { f(i, r, n, place); });
        }
      };
      if (issuer && held != 0) {
        unsigned bytes = 0;
        bf16_rows_of([&](int, int, int n, uint32_t) { bytes += n * 256; });
        mbar_arrive_expect_tx(&brows[buf], bytes);
        bf16_rows_of([&](int i, int r, int n, uint32_t place) {
          bulk_copy_g2s(sm + kRdO + buf * 32768 + place, (i ? rows1 : rows0) + (size_t)r * kD, n * 256, &brows[buf]);
        });
      }
      const float s0 = __low2float(scale), s1 = __high2float(scale);
      // pages of which every row is written from codes leave by TMA
      auto whole_page = [&](int i) {
        const int p = p0 + i * kPage;
        return (src >> i & 1) && p >= lo && p + kPage <= hi && p >= hlo && p + kPage <= hhi;
      };
      const bool whole = whole_page(pg);
      const int p = p0 + row, page = pg ? dst1 : dst0;
      const bool mine = p >= lo && p < hi && page >= 0, history = p >= hlo && p < hhi;
      uint8_t* res = sm + kRdO + buf * 32768 + hf * 16384;
      uint4* dst = reinterpret_cast<uint4*>(pool + (((size_t)max(page, 0) * a.from.num_kv_heads + h) * kPage + (row & 63)) * kD + 64 * hf);
      if (src) {
        const uint32_t tm = ((uint32_t)(32 * q) << 16) + 256 * buf + 64 * hf;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          float x[16], y[16];
          tmem_ld16x2(tm + 16 * cc, tm + 128 + 16 * cc, x, y);
          if (cc == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 8 * c + 2 * e;
              const float2 z = ffma2(make_float2(x[i], x[i + 1]), make_float2(s0, s0),
                                     fmul2(make_float2(y[i], y[i + 1]), make_float2(s1, s1)));
              o[e] = pack_bf16x2(z.x, z.y);
            }
            const uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
            if (whole)
              *sw128_chunk(res, row, 2 * cc + c) = v;
            else if (mine && history && (src >> pg & 1))
              dst[2 * cc + c] = v;
          }
        }
      } else if (lane == 0) {
        mbar_arrive(&tempty[buf]);
      }
      fence_proxy_async_smem();
      group_sync(1 + buf, 256);
      if (issuer) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (whole_page(i))
#pragma unroll
            for (int half = 0; half < 2; ++half)
              tma_store_3d(is_v ? &tmv : &tmk, 64 * half, h * kPage, i ? dst1 : dst0,
                           sm + kRdO + buf * 32768 + 16384 * half + 8192 * i);
        if (held != 0) {
          if (mbar_wait_timed(&brows[buf], phase, kWaitNs))
            bf16_rows_of([&](int i, int r, int n, uint32_t place) {
              bulk_copy_s2g(pool + (((size_t)(i ? dst1 : dst0) * a.from.num_kv_heads + h) * kPage + r) * kD,
                            sm + kRdO + buf * 32768 + place, n * 256);
            });
          else
            dead[buf] = it + 3;
          phase ^= 1u;
        }
        bulk_commit();
      }
    }
    if (dead[buf] != 0 && issuer) set_error(a.err, kErrTimeout);
    if (issuer) bulk_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kRdMma) {
    tc_fence_after();
    tmem_dealloc(0, 512);
  }
}

}  // namespace

cudaError_t launch_int2_to_bf16(const Read2Launch& a, cudaStream_t stream) {
  static std::atomic<uint64_t> set;
  const void* fn = reinterpret_cast<const void*>(int2_to_bf16_kernel);
  const cudaError_t e = smem_attr_once(fn, kRdSmem, set);
  if (e != cudaSuccess) return e;
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t r = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (r != cudaSuccess || q != cudaDriverEntryPointSuccess) return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  // the BF16 pools as [num_pages][Hkv 64 rows][128 channels], boxes of 64 channels x one head's page
  const int Hkv = a.from.num_kv_heads;
  CUtensorMap tm[2];
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)Hkv * kPage, (cuuint64_t)a.to.num_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)Hkv * kPage * kD * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)kPage, 1}, estride[3] = {1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (encode(&tm[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i ? a.v_pages : a.k_pages, dims, strides, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  // at most: a request's rows touch (max_count + 126) / 64 pages, and no more than its table has (a loose bound is no error)
  const long long pages = std::min(((long long)a.max_count + 126) / kPage, (long long)a.to.max_pages), pairs = (pages + 1) / 2;
  const long long tiles = pairs * Hkv * a.from.batch;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  Read2Launch la = a;
  void* args[] = {&la, &tm[0], &tm[1]};
  const unsigned blocks = 2 * (unsigned)std::min<long long>(tiles, std::max(a.num_sms / 2, 1));
  return launch_pdl(fn, dim3(blocks), dim3(kRdThreads), kRdSmem, stream, args);
}

}  // namespace oscar
