// Windowed attention of chunks and prompts over BF16 pages, and of whole prompts
// in packed rows, on the 5th-generation tensor cores.
//
// One thread block per SM goes through work items (in steps of the grid); an
// item is two tiles of 128 rows of one (request, KV head): row r of a tile is
// query r / g of the tile and query head r % g, so the g heads that share the
// keys share each of their copies.  For a block of 128 keys (two pages)
//   S = Q K^T   M 128 (rows), N 128 (keys), K 16 a step; both from shared memory
//   P = exp2(c S - m), rounded to bf16 (one term, at most 2^-8 of a weight, as
//       the result is; c = sm_scale log2 e, m the row's reference, below)
//   O += P V    P from tensor memory (over S's columns), V as it lies in
//       the page: keys along K, channels contiguous (an "MN-major" operand)
// with S, O and the sums in fp32.  Tensor memory: S of both tiles (2 x 128
// columns), O of both (2 x 128).
//
//   warps 0-15   softmax: tile w / 8, keys 64 (w / 4 % 2) .. + 63 of a block; a
//                thread is half a row (its TMEM lane), so that the time from S to
//                P, which the products wait for, is that of 64 exponentials
//   warp 16      copies the queries (TMA, 64 channels x g heads x the tile's
//                queries) and K and V blocks (64 channels x 64 rows; 128-byte
//                swizzle) into a ring of five 32 KB slots, in the order of use:
//                K_0, V_0, K_1, V_1, ...; it runs ahead into the next item
//   warp 17      one thread issues the MMAs, tile by tile: S_t(j + 1) right
//                behind P_t V(j), so that one tile's softmax runs under the other
//                tile's products
//   warps 18, 19 (relays) of tile 0, 1: wait for the copies that the next products
//                read and clear the V rows that no query sees; work out the next
//                item under the result of the one before.  (The softmax warps poll
//                for their products themselves: with a relay that polled and met
//                them at a hardware barrier 467 us, now 454, 48 ragged prompts.)
// The next item's first logits are computed while the last weights and the
// result of the one before are still under way (a block per item: 25,000 of
// 105,000 cycles an item were its beginning and its end).  An item sees only
// the pages that some of its queries see.  With few (tile pair, KV head) groups
// their keys are split over several items, whose records (m, l, O) a second
// kernel joins in item order.
//
// What bounds it: the way from a block's logits to its weights (TMEM loads, 64
// exponentials a thread at 4 cycles a warp, the vote on the maximum, TMEM store),
// about 1340 cycles, behind 1030 of the tile's own products, which the other tile's
// share: a pair of blocks takes 2400 cycles, its products 2060; and an item's last
// and first blocks 6200, with the result on its way to memory (2700) in between.
// For seconds on end, the board's power limit (1.7 to 1.8 GHz instead of 2.05).
// Three prompts of up to 12K tokens over pages (window 4096, 32 query heads):
// 0.98 ms, 1.58 PFLOP/s; 256 tokens at 100,000: 257 us.  In packed rows: one
// prompt of 24,001 tokens 2.5 to 2.8 ms, 1.66 to 1.92 PFLOP/s, 48 prompts of 1 to
// 2048 tokens 437 us (490 to 500 for seconds).
// Tried when the first took 1.19: all sixteen warps on one tile at a time (a
// quarter of a row a thread), 1.32 ms, since the loads and votes then lie bare;
// the next logits' loads under the exponentials, 1.22 ms.  When the 48 prompts took
// 436: 64 keys a product, so that half of the weights could begin earlier, 481 (the
// queries are read twice as often); an item's result behind the next one's first
// weights, 543 for 481 (both tiles' weights then fall into step).
// Nothing may spill: the block's shared memory leaves the SM no first-level cache,
// so a register in local memory is an L2 access, 600 cycles, wherever it is read
// (nine a warp in the result's way out cost 4,000 cycles an item).
//
// Packed rows (ROWS): a "page" is 64 rows of a request's keys, copied by the same
// boxes from a map of [heads][rows][128]; the blocks take items by ticket, which
// the copying warp hands to the others through a ring of two.

#include "oscar_paged.cuh"
#include "oscar_prompt.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

namespace oscar {
namespace {

constexpr float kLog2eT = 1.4426950408889634f;
constexpr int kTcwThreads = 20 * 32;
constexpr int kTcwCopy = 16, kTcwMma = 17, kTcwRelay = 18;  // warps
constexpr int kTcwSlots = 5;
constexpr uint32_t kTcwQ = 0;                    // queries: [tile][2 x 64 channels][128 rows][128 B]
constexpr uint32_t kTcwRing = 65536;             // slots: [2 x 64 channels][128 keys][128 B]
constexpr uint32_t kTcwBars = kTcwRing + kTcwSlots * 32768;
constexpr uint32_t kTcwItems = kTcwBars + 256;  // the softmax warps' items: [tile][two in turn]
constexpr uint32_t kTcwX = kTcwBars + 1024;      // what the two halves of a row tell each other: [tile][half][128 rows] float
constexpr size_t kTcwSmem = kTcwX + 2048;        // (all of it dynamic, so that it begins where the block's memory does)
constexpr uint32_t kTmS = 0, kTmO = 256;         // TMEM columns of S and O, 128 a tile
// A row's weights are taken relative to the maximum of the first block that it saw something of, until half a row's
// sum of them, over all blocks so far, reaches kTopSum (2^40; fp32 and bf16 reach 2^127): then the maximum is found
// anew, or taken 2^39 higher if the sum was that already, and O and l move.  So the common block needs no maximum: its exponentials
// start with the first logits that arrive (a block that moves takes 2000 cycles more; at 2^16 every fifth block did).
// A record's sum stays below 2^41, and 304 records' below 2^50.
constexpr float kTopSum = 1099511627776.0f;
// Over packed rows the first block asks for no maximum either: weights are relative to 0 (what logits are near) until
// half a row's sum reaches kTopSum, or a row that has seen something has less than 2^-60 of weight; then its maximum
// becomes the reference, up or down (48 prompts of 1 to 2048 tokens 518 us then; 540 with a maximum found in each first block).
constexpr float kLowSum = 8.673617379884035e-19f;
constexpr int kRowFloats = kD + 2;               // of a tile's record, for each of its 128 rows: O[128], m, l

// x / d for 0 <= x < 2^31 by a multiplication: with d <= 2^l and mul = ceil(2^(31 + l) / d) the quotient is
// floor(x mul / 2^(31 + l)), since x mul / 2^(31 + l) exceeds x / d by less than x / 2^(31 + l) < 1 / d.
struct Divisor {
  uint32_t d = 1, mul = 0x80000000u, shift = 31;
  Divisor() = default;
  explicit Divisor(uint32_t n) : d(n) {
    uint32_t l = 0;
    while ((1ull << l) < n) ++l;
    shift = 31 + l;
    mul = (uint32_t)(((1ull << shift) + n - 1) / n);
  }
  __device__ __forceinline__ int divide(int x, int& rest) const {
    const int q = (int)(((unsigned long long)(uint32_t)x * mul) >> shift);
    rest = x - q * (int)d;
    return q;
  }
};

struct TcwArgs {
  WindowLaunch a;
  Divisor by_items, by_heads, by_batch, by_tiles;
  int batch;
  int g;                  // query heads of a KV head
  int items, tiles, qpt;  // items per (tile pair, KV head), tile pairs per request, queries per tile
  int total;              // items of the call
  KeyRows keys;           // keys in packed rows instead of pages
  int* tickets;           // (packed rows) items taken beside the blocks' first ones, blocks that are done
};

// D[tmem] (+)= A[smem] B[smem]^T and A[tmem] B[smem], the operands' descriptors as their low words (start address
// / 16, and above it the leading offset / 16) with one high word.  A K-major operand in the 128-byte swizzle has
// rows of 64 elements and groups of 8 rows 1024 bytes apart (the leading offset is not used); an operand with its
// N index contiguous has K as the rows, and the next 64 of N a leading offset on.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

__device__ __forceinline__ int sm_load(uint32_t at) {
  int v;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sm_store(uint32_t at, int v) { asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(at), "r"(v) : "memory"); }

__device__ __forceinline__ void tma_load_page(void* dst, const void* tmap, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float exp2_t(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 columns of this thread's lane, in flight until the wait that names the same registers.
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// 32 columns, waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[2][16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0][0]), "=r"(r[0][1]), "=r"(r[0][2]), "=r"(r[0][3]), "=r"(r[0][4]), "=r"(r[0][5]), "=r"(r[0][6]), "=r"(r[0][7]), "=r"(r[0][8]), "=r"(r[0][9]), "=r"(r[0][10]), "=r"(r[0][11]), "=r"(r[0][12]), "=r"(r[0][13]), "=r"(r[0][14]), "=r"(r[0][15]), "=r"(r[1][0]), "=r"(r[1][1]), "=r"(r[1][2]), "=r"(r[1][3]), "=r"(r[1][4]), "=r"(r[1][5]), "=r"(r[1][6]), "=r"(r[1][7]), "=r"(r[1][8]), "=r"(r[1][9]), "=r"(r[1][10]), "=r"(r[1][11]), "=r"(r[1][12]), "=r"(r[1][13]), "=r"(r[1][14]), "=r"(r[1][15])
      : "r"(taddr)
      : "memory");
}

// The n lowest of 32 bits (n may lie outside 0..32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Logits whose bit of `seen` (from bit `at`) is 0 drop out.
__device__ __forceinline__ void hide(uint32_t (&s)[16], uint32_t seen, int at) {
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (!(seen & (1u << (at + e)))) s[e] = 0xff800000u;
}

__device__ __forceinline__ float max16(const uint32_t (&s)[16]) {
  float m[2] = {__uint_as_float(s[0]), __uint_as_float(s[1])};
#pragma unroll
  for (int e = 2; e < 16; ++e) m[e & 1] = fmaxf(m[e & 1], __uint_as_float(s[e]));
  return fmaxf(m[0], m[1]);
}

// exp2(c s - mc) of 16 logits: their sum, and 8 pairs of bf16.
__device__ __forceinline__ void weights(const uint32_t (&s)[16], float c, float mc, float2& sum, uint32_t* w) {
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const float2 y = ffma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(c, c),
                           make_float2(-mc, -mc));
    const float2 p = make_float2(exp2_t(y.x), exp2_t(y.y));
    sum = fadd2(sum, p);
    w[e >> 1] = pack_bf16x2(p.x, p.y);
  }
}

// The lane, read where it is used: kept through every role of the kernel, its register makes another one spill.
__device__ __forceinline__ int lane_id() {
  uint32_t l;
  asm volatile("mov.u32 %0, %%laneid;\n" : "=r"(l));
  return (int)l;
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x != 0;
}

// Whether any thread of the two warps at named barrier `id` says so.
__device__ __forceinline__ bool pair_any(int id, bool x) {
  uint32_t y;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %2, 0;\n barrier.cta.red.or.pred p, %1, 64, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(y)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return y != 0;
}

// Request b's tokens and keys among packed rows.
__device__ __forceinline__ bool rows_span(const TokenRefs& t, const KeyRows& k, int b, int& n, int& row0, int& n_keys,
                                          int& key0, unsigned* err, bool report) {
  const int lo = t.cu[b], hi = t.cu[b + 1], klo = k.cu[b], khi = k.cu[b + 1];
  if (lo < 0 || hi < lo || hi > t.n_tokens || hi - lo > t.max_tokens || klo < 0 || khi < klo || khi > k.n_keys ||
      khi - klo > k.max_keys) {
    if (report) set_error(err, kErrTokens);
    return false;
  }
  row0 = lo;
  n = hi - lo;
  key0 = klo;
  n_keys = khi - klo;
  return true;
}

// The pages that some query of a block sees: logical pages [0, sp) and [wb, we).
struct PageList {
  int sp, wb, we;
  __device__ __forceinline__ int count() const { return sp + max(0, we - wb); }
  __device__ __forceinline__ int page(int k) const { return k < sp ? k : wb + (k - sp); }
};

// One work item, as every role sees it.
struct TcwItem {
  int b, h, row0, n, p0, i0, ntile;  // request, KV head, its tokens, the item's first query and tiles
  int last;                          // position of the item's last query
  int record;                        // its place among the items of its (tile pair, request, KV head)
  int ctx, hi, lo, sinks;            // held positions; no query sees hi or beyond; windows start at lo
  PageList pl;
  int np, j0, nb;                    // pages that some query sees; the item's key blocks [j0, j0 + nb)
  int k_clean, k_held;               // pages of the list of which some query sees every row: [k_clean, k_held)
  int k_lo, k_hi;                    // (softmax) pages of the list that every row of the tile sees whole: [k_lo, k_hi)
  int key0;                          // (packed rows) the row of position 0
};


// False: nothing to do (the request has no such queries).  SPLIT: several items share a group's keys.  ROWS: the keys
// are packed rows, a "page" 64 of them; a request's queries are the last of its positions (those before position 0
// see nothing).
template <bool SPLIT, bool ROWS>
__device__ __forceinline__ bool tcw_item(const TcwArgs& ta, int idx, TcwItem& t, bool report, int given = -1) {
  const WindowLaunch& a = ta.a;
  int item = 0, pair;
  if constexpr (!SPLIT) {  // later tiles (more keys) first
    if (given >= 0) {  // t.b and t.h are given too
      pair = given;
    } else {
      pair = ta.tiles - 1 - ta.by_batch.divide(ta.by_heads.divide(idx, t.h), t.b);
      t.record = idx;
    }
  } else {  // the tile pairs that read the same keys side by side, so that these come from memory once
    int x = ta.by_tiles.divide(idx, pair);
    x = ta.by_heads.divide(x, t.h);
    t.b = ta.by_items.divide(x, item);
    t.record = ((t.b * a.Hkv + t.h) * ta.tiles + pair) * ta.items + item;
  }
  if constexpr (ROWS) {
    if (!rows_span(a.tok, ta.keys, t.b, t.n, t.row0, t.ctx, t.key0, a.err, report)) return false;
    t.p0 = t.ctx - t.n;
  } else {
    if (!token_span(a.tok, t.b, t.p0, t.n, t.row0, a.err, report)) return false;
  }
  t.i0 = pair * 2 * ta.qpt;
  if (t.i0 >= t.n) return false;
  const int i1 = min(t.i0 + 2 * ta.qpt, t.n);
  t.ntile = t.i0 + ta.qpt < t.n ? 2 : 1;
  if constexpr (ROWS) {
    t.last = t.p0 + i1 - 1;
  } else {
    // a request whose positions are not all in 0 .. 2^31 - 2 sees nothing
    const long long last = (long long)t.p0 + i1 - 1;
    const bool out = t.p0 < 0 || last > INT32_MAX - 1;
    t.ctx = out ? 0 : max(a.ctx_len[t.b], 0);
    t.last = out ? -1 : (int)last;
    const long long limit = (long long)a.pages.max_pages * kPage;
    if (report && (out || min(t.last + 1, t.ctx) > limit)) set_error(a.err, kErrLength);
    t.ctx = (int)min((long long)t.ctx, limit);
  }
  t.hi = max(0, min(t.last + 1, t.ctx));
  // (a window of 0 holds nothing)
  t.lo = a.window < 0 ? 0 : a.window == 0 ? max(t.hi, 1) : max(0, t.p0 + t.i0 - a.window + 1);
  t.sinks = min(a.sinks, t.hi);
  t.pl.we = (t.hi + kPage - 1) / kPage;
  t.pl.sp = t.lo > 0 ? (t.sinks + kPage - 1) / kPage : 0;
  t.pl.wb = t.lo >= t.hi ? t.pl.we : max(t.lo / kPage, t.pl.sp);
  t.np = t.pl.count();
  t.k_clean = t.pl.sp + max(0, (t.lo + kPage - 1) / kPage - t.pl.wb);
  t.k_held = t.pl.sp + t.hi / kPage - t.pl.wb;
  t.j0 = 0;
  t.nb = (t.np + 1) / 2;
  if constexpr (SPLIT) {
    const int share = t.nb / ta.items, more = t.nb - share * ta.items;
    t.j0 = item * share + min(item, more);
    t.nb = share + (item < more);
  }
  return true;
}

// First position of the k-th page of an item's list; past every position if there is none, or it is outside the pool.
template <bool ROWS>
__device__ __forceinline__ int block_page(const TcwArgs& ta, const TcwItem& it, int k, bool bad) {
  const int lp = k >= it.np ? -1 : it.pl.page(k);
  return lp < 0 || (!ROWS && bad && page_of(ta.a.pages, it.b, lp, ta.a.err, false) < 0) ? INT32_MAX - 63 : lp * kPage;
}

// Whether query ql of an item (of the first of its keys' parts) sees any key: one that does and has no weight has logits of
// -infinity alone, which is not a number as a row; one that does not gets zeros.
template <bool ROWS>
__device__ __forceinline__ bool row_sees(const TcwArgs& ta, const TcwItem& it, int ql, bool bad) {
  const int p = min(it.p0 + it.i0 + ql, it.last), lim = min(p + 1, it.ctx);
  const int low = ta.a.window < 0 ? 0 : max(0, p - ta.a.window + 1);
  if (ROWS || !bad) return lim > 0 && (it.sinks > 0 || low < lim);
  for (int k = 0; k < it.np; ++k) {
    const int base = block_page<ROWS>(ta, it, k, true);
    if (base < lim && (base < it.sinks || low < min(base + kPage, lim))) return true;
  }
  return false;
}

// V rows of a block that no query of the item sees may hold anything, and 0 x NaN is not 0: they become zeros, in
// front of the products that read them.  One warp, 16 bytes a lane: four rows of 64 channels a step, by 32 rows' bits (with
// a comparison of positions a row it took longer than the weights that it runs beside, and every item's last block
// waited for it: 48 prompts of 1 to 2048 tokens 517 us, now 481).
template <bool ROWS>
__device__ __forceinline__ void clean_block(const TcwArgs& ta, const TcwItem& it, int k0, bool bad, uint8_t* v, int lane) {
  const int base[2] = {block_page<ROWS>(ta, it, k0, bad), block_page<ROWS>(ta, it, k0 + 1, bad)};
  const int hi = it.hi, lo = it.lo, sinks = it.sinks;
  v += (lane >> 3) * 128 + 16 * (lane & 7);
#pragma unroll 1
  for (int w = 0; w < (k0 + 1 < it.np ? 4 : 2); ++w) {  // 32 rows (of a page that there is)
    const int p32 = base[w >> 1] + 32 * (w & 1);
    const uint32_t unseen = ~(low_bits(hi - p32) & (low_bits(sinks - p32) | ~low_bits(lo - p32)));
    if (unseen == 0) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((unseen >> (lane >> 3) >> (4 * i)) & 1u) {
        *reinterpret_cast<uint4*>(v + 4096 * w + 512 * i) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(v + 4096 * w + 512 * i + 16384) = make_uint4(0u, 0u, 0u, 0u);
      }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Four 16-byte pieces of each lane's row to memory: a 4 x 4 exchange among four lanes first, so that they write
// 64 contiguous bytes of a row (each lane its own row took 12,000 cycles a tile; eight at once spill).  at(r): where
// row r (0..31 of the warp) has them; `live`: the warp's rows that are written.
template <typename At>
__device__ __forceinline__ void store_rows(uint4 (&x)[4], int lane, uint32_t live, At at) {
#pragma unroll
  for (int b = 1; b < 4; b <<= 1)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (!(u & b)) {
        const bool up = (lane & b) != 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t &lo = word_of(x[u], e), &hi = word_of(x[u | b], e);
          const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? lo : hi, b);
          if (up)
            lo = y;
          else
            hi = y;
        }
      }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (lane & 28) + i;
    uint4* dst = at(r);
    if ((live >> r) & 1u) dst[lane & 3] = x[i];
  }
}

// This thread's half row of O, over its sum l, into the result; or, where several items share a group's keys, into the
// group's records, which window_join_kernel joins.
template <bool SPLIT>
__device__ __forceinline__ void tcw_result(const TcwArgs& ta, const TcwItem& it, int warp, int lane,
                                        uint32_t to, int ql, bool live, bool got, float m, float l) {
  const WindowLaunch& a = ta.a;
  const int t = warp >> 3, hf = (warp >> 2) & 1, g = ta.g;
  if constexpr (!SPLIT) lane = lane_id();  // (registers: with the caller's 16 bytes spill)
  const int row = 32 * (warp & 3) + lane;
  const uint32_t rows = __ballot_sync(0xffffffffu, live);
  uint4 x[4];
  if constexpr (!SPLIT) {
    const float f = got && l != 0.f ? 1.f / l : 0.f;
    // the rows of the result [token][query head], in quarters of 64 bytes
    // (head row - (ql - t qpt) g of the KV head's; divisions by g here took 300 cycles an item)
    const uint32_t mine = (uint32_t)(it.row0 + it.i0 + ql) * a.Hq + (it.h - ql + t * ta.qpt) * g + row;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t o[16];
        if (got) {
          tmem_ld16_start(to + 32 * part + 16 * k, o);
          tmem_ld16_wait(o);
        }
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          word_of(x[2 * k + (e >> 3)], (e >> 1) & 3) =
              got ? pack_bf16x2(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f) : 0u;
      }
      store_rows(x, lane, rows, [&](int r) {
        return reinterpret_cast<uint4*>(a.out + (size_t)__shfl_sync(0xffffffffu, mine, r) * kD + 64 * hf + 32 * part);
      });
    }
  } else {
    // the records: O [row][128], then m [row], l [row]
    float* rec = reinterpret_cast<float*>(a.workspace + a.plan.off_records) + ((size_t)it.record * 256 + 128 * t) * kRowFloats;
    if (live && hf == 0) {
      rec[128 * kD + row] = got && l != 0.f ? m : -INFINITY;  // (over packed rows what saw nothing has a reference too)
      rec[129 * kD + row] = l;
    }
    if (got)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t o[16];
        tmem_ld16_start(to + 16 * k, o);
        tmem_ld16_wait(o);
#pragma unroll
        for (int e = 0; e < 16; e += 4) x[e >> 2] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        store_rows(x, lane, rows, [&](int r) {
          return reinterpret_cast<uint4*>(rec + (32 * (warp & 3) + r) * kD + 64 * hf + 16 * k);
        });
      }
  }
}

template <bool SPLIT, bool ROWS>
__global__ void __launch_bounds__(kTcwThreads, 1)
    window_tc_kernel(const __grid_constant__ TcwArgs ta, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq) {
  const WindowLaunch& a = ta.a;
  extern __shared__ __align__(1024) uint8_t sm[];
  // (by way of a shuffle, so that the compiler knows the warp's role to be uniform)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = ta.g, qpt = ta.qpt;
  const uint32_t sbase = smem_u32(sm);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kTcwBars);  // [slots] copies landed
  uint64_t* empty = full + kTcwSlots;                           // [slots] read by its products
  uint64_t* sfull = empty + kTcwSlots;                          // [2] S of tile t holds a block's logits (and O its last product)
  uint64_t* pready = sfull + 2;                                 // [2] P of tile t written, the copies for what follows landed
  uint64_t* odone = pready + 2;                                 // [2] O of tile t complete
  uint64_t* qfull = odone + 2;                                  // the item's queries landed
  uint64_t* qempty = qfull + 1;                                 // read by the item's last logits
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(qempty + 1);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_at + 2);
  // [0, 1] the relay of tile t gave up; [2] a page outside the pool was met; [3] (ROWS) the copies or the products gave up
  uint64_t* ifull = reinterpret_cast<uint64_t*>(sm + kTcwBars + 224);  // (ROWS) [2] an item is in the ring's place
  uint64_t* iempty = ifull + 2;                                        // [2] the products' and the relays' warps have it
  TcwItem* ring_items = reinterpret_cast<TcwItem*>(sm + kTcwItems) + 4;
  static_assert(6 * sizeof(TcwItem) <= kTcwX - kTcwItems, "the items' places");
  if (threadIdx.x < 4) flags[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcwSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[t], 9);  // the tile's softmax warps, and its relay for the copies
      mbar_init(&odone[t], 1);
      mbar_init(&ifull[t], 1);
      mbar_init(&iempty[t], 3);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    fence_mbar_init();
  }
  if (warp == kTcwMma) tmem_alloc(tmem_at, 512);  // all of it, so its base is column 0
  if (warp == kTcwCopy && lane == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    prefetch_tensormap(&tmq);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  bool gave_up = false;
  TcwItem it;
  // A wait for another item takes as long as the one that is under way: a minute at most, and no longer than others work.
  auto wait_ring = [&](uint64_t* bar, uint32_t phase) {
    for (int i = 0; i < 60; ++i) {
      if (__all_sync(0xffffffffu, mbar_wait_timed(bar, phase, kWaitNs))) return true;
      if (__any_sync(0xffffffffu, flags[0] | flags[1] | flags[3])) return false;
    }
    return false;
  };

  if (warp == kTcwCopy) {
    // ---- copies: an item's use 0 of the ring is K_0, 2 j + 1 is V_j, 2 j + 2 is K_(j + 1)
    const int lane = lane_id();
    uint32_t use = 0, items = 0;
    // ROWS: the first item by the block's number, the others as the blocks come to them, so that blocks with short items
    // take more; through a ring of two places.  (A ticket taken before the item ahead is copied is kept from the blocks
    // that are free: two chunks over 40,000 keys 332 us for 180.)
    uint32_t published = 0;
    auto publish = [&](bool end) {
      const uint32_t place = published & 1;
      gave_up = !wait_ring(&iempty[place], ((published >> 1) & 1) ^ 1);
      if (gave_up) return;
      if (lane == 0) {
        if (end) it.ntile = -1, it.nb = 0;
        ring_items[place] = it;
        mbar_arrive(&ifull[place]);
      }
      ++published;
      __syncwarp();
    };
    int ticket = 0;
    auto after = [&](int idx) {
      if constexpr (!ROWS) return idx + (int)gridDim.x;
      return __shfl_sync(0xffffffffu, ticket, 0);
    };
    // Whole items: request by request, its last tiles (most keys) first, so that what the blocks read at one time lies in L2
    // (48 prompts of 1 to 2048 tokens, 200 MB of K and V: their longest tiles first read 2.4 GB of memory, 560 us), and tiles
    // that a ragged batch's bound has and a request does not cost no ticket.  64 requests at a time (lane and lane + 32), from
    // `from` on, whose items are those from `before` on; idx only grows.
    constexpr bool kCounted = ROWS && !SPLIT;
    int pairs[2] = {0, 0}, upto[2] = {0, 0}, from = -64, before = 0, all = 0;
    auto locate = [&](int idx) {  // the pair of tiles; -1: there is no such item
      int q = ta.by_heads.divide(idx - before, it.h);
      while (q >= all) {
        before += all * a.Hkv;
        q -= all;
        from += 64;
        if (from >= ta.batch) return -1;
        all = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          int n, r0, nk, k0;
          const int b = from + 32 * k + lane;
          pairs[k] = b < ta.batch && rows_span(a.tok, ta.keys, b, n, r0, nk, k0, a.err, true) ? (n + 2 * qpt - 1) / (2 * qpt) : 0;
          int s = pairs[k];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
          }
          upto[k] = all + s;
          all = __shfl_sync(0xffffffffu, upto[k], 31);
        }
      }
      const uint32_t m0 = __ballot_sync(0xffffffffu, upto[0] > q), m1 = __ballot_sync(0xffffffffu, upto[1] > q);
      const int l = __ffs(m0 != 0 ? m0 : m1) - 1;
      it.b = from + (m0 != 0 ? 0 : 32) + l;
      return __shfl_sync(0xffffffffu, m0 != 0 ? upto[0] : upto[1], l) - 1 - q;
    };
    for (int idx = blockIdx.x; idx < ta.total && !gave_up; idx = after(idx)) {
      if constexpr (ROWS) {
        const int pair = kCounted ? locate(idx) : 0;
        if (pair < 0) break;
        auto next_ticket = [&]() { ticket = (int)gridDim.x + atomicAdd(ta.tickets, 1); };
        const bool some = tcw_item<SPLIT, ROWS>(ta, idx, it, lane == 0, kCounted ? pair : -1);
        if (some) publish(false);
        if (gave_up) break;
        if (!some || it.nb == 0) {
          if (lane == 0) next_ticket();
          continue;
        }
        if (lane == 0) {
          // What this loop needs of the item it reads from the ring each time (which keeps it until the item after the
          // next): the little that does not fit in registers would come from L2, 600 cycles away, since all of the SM's
          // first-level memory is shared memory (1440 cycles from a copy's start to its use then, 4000 now).
          const uint32_t my = smem_u32(&ring_items[(published - 1) & 1]);
          auto field = [&](size_t at) { return sm_load(my + (uint32_t)at); };
          auto first_row = [&](int k) {  // of the k-th page of the item, -1 if there is none
            const int kk = 2 * field(offsetof(TcwItem, j0)) + k, sp = field(offsetof(TcwItem, pl.sp));
            if (kk >= field(offsetof(TcwItem, np))) return -1;
            return field(offsetof(TcwItem, key0)) + (kk < sp ? kk : field(offsetof(TcwItem, pl.wb)) + kk - sp) * kPage;
          };
          for (int u = 0; u < 2 * field(offsetof(TcwItem, nb)) && !gave_up; ++u, ++use) {
            const uint32_t slot = use % kTcwSlots, round = use / kTcwSlots;
            if (u == max(0, 2 * field(offsetof(TcwItem, nb)) - 4)) next_ticket();  // (it arrives under the last copies)
            if (round > 0 && !mbar_wait_timed(&empty[slot], (round - 1) & 1, kWaitNs)) gave_up = true;
            if (gave_up) break;
            const int q0 = first_row(u & ~1), q1 = first_row(u | 1), h = field(offsetof(TcwItem, h));
            uint8_t* dst = sm + kTcwRing + slot * 32768;
            mbar_arrive_expect_tx(&full[slot], q1 >= 0 ? 32768u : 16384u);
            const void* tm = u & 1 ? static_cast<const void*>(&tmv) : static_cast<const void*>(&tmk);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              tma_load_page(dst + half * 16384, tm, 64 * half, q0, h, &full[slot]);
              if (q1 >= 0) tma_load_page(dst + half * 16384 + 8192, tm, 64 * half, q1, h, &full[slot]);
            }
            if (u == 0) {  // the queries, behind K_0 (whose slot is free earlier)
              if (items > 0 && !mbar_wait_timed(qempty, (items - 1) & 1, kWaitNs)) gave_up = true;
              if (gave_up) break;
              const int nt = field(offsetof(TcwItem, ntile)), row = field(offsetof(TcwItem, row0)) + field(offsetof(TcwItem, i0));
              mbar_arrive_expect_tx(qfull, (uint32_t)(nt * 2 * g * qpt * 128));
              for (int t = 0; t < nt; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  tma_load_page(sm + kTcwQ + t * 32768 + half * 16384, &tmq, 64 * half, h * g, row + t * qpt, qfull);
            }
          }
        }
        gave_up = __shfl_sync(0xffffffffu, gave_up, 0);
        use = __shfl_sync(0xffffffffu, use, 0);
        ++items;
        continue;
      }
      if (!tcw_item<SPLIT, ROWS>(ta, idx, it, lane == 0) || it.nb == 0) continue;
      int phys_l = -1, fetched = 0;
      auto phys_of = [&](int k) {  // k-th page of this item (whole warp)
        if (k >= fetched) {
          phys_l = -1;
          const int kk = 2 * it.j0 + fetched + lane;
          if (kk < min(2 * (it.j0 + it.nb), it.np)) {
            phys_l = page_of(a.pages, it.b, it.pl.page(kk), a.err, true);
            if (phys_l < 0) flags[2] = 1;
          }
          fetched += 32;
        }
        return __shfl_sync(0xffffffffu, phys_l, k & 31);
      };
      int q0 = -1, q1 = -1;
      for (int u = 0; u < 2 * it.nb && !gave_up; ++u, ++use) {
        const bool is_v = (u & 1) != 0;
        if (!is_v) {  // block u / 2: pages u, u + 1
          q0 = phys_of(u);
          q1 = phys_of(u + 1);
        }
        const uint32_t slot = use % kTcwSlots, round = use / kTcwSlots;
        __syncwarp();
        if (lane == 0) {
          if (round > 0 && !mbar_wait_timed(&empty[slot], (round - 1) & 1, kWaitNs)) gave_up = true;
          if (!gave_up) {
            uint8_t* dst = sm + kTcwRing + slot * 32768;
            mbar_arrive_expect_tx(&full[slot], (q0 >= 0 ? 16384u : 0u) + (q1 >= 0 ? 16384u : 0u));
            const void* tm = is_v ? static_cast<const void*>(&tmv) : static_cast<const void*>(&tmk);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (q0 >= 0) tma_load_page(dst + half * 16384, tm, 64 * half, it.h * kPage, q0, &full[slot]);
              if (q1 >= 0) tma_load_page(dst + half * 16384 + 8192, tm, 64 * half, it.h * kPage, q1, &full[slot]);
            }
          }
          if (u == 0 && !gave_up) {  // the queries, behind K_0 (whose slot is free earlier)
            if (items > 0 && !mbar_wait_timed(qempty, (items - 1) & 1, kWaitNs)) gave_up = true;
            if (!gave_up) {
              mbar_arrive_expect_tx(qfull, (uint32_t)(it.ntile * 2 * g * qpt * 128));
              for (int t = 0; t < it.ntile; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  tma_load_page(sm + kTcwQ + t * 32768 + half * 16384, &tmq, 64 * half, it.h * g, it.row0 + it.i0 + t * qpt, qfull);
            }
          }
        }
        gave_up = __shfl_sync(0xffffffffu, gave_up, 0);
      }
      ++items;
    }
    if constexpr (ROWS) {
      if (!gave_up) publish(true);
      if (lane == 0) {  // the last block leaves the tickets as it found them
        __threadfence();
        if (atomicAdd(ta.tickets + 1, 1) == (int)gridDim.x - 1) {
          ta.tickets[0] = 0;
          ta.tickets[1] = 0;
        }
      }
    }
    if (gave_up && lane == 0) {
      flags[3] = 1;
      set_error(a.err, kErrTimeout);
      // the copies still in flight land before the block ends
      for (int i = 0; i < kTcwSlots; ++i) {
        mbar_wait_timed(&full[i], 0, kWaitNs);
        mbar_wait_timed(&full[i], 1, kWaitNs);
      }
      mbar_wait_timed(qfull, 0, kWaitNs);
      mbar_wait_timed(qfull, 1, kWaitNs);
    }
  } else if (warp >= kTcwRelay) {
    // ---- relays: the copies that the next products read, and the next item
    const int lane = lane_id();
    const int tt = warp - kTcwRelay;
    uint32_t use = 0, blocks = 0;
    // (only of copies whose slot cannot be filled again before this warp's arrival: K_0's can)
    auto landed = [&](uint32_t u) {
      return __all_sync(0xffffffffu, mbar_wait_timed(&full[u % kTcwSlots], (u / kTcwSlots) & 1, kWaitNs)) != 0;
    };
    // The next item is worked out for the softmax warps while they are at the result of the one before; its place is
    // free since they came to that one.
    TcwItem* place = reinterpret_cast<TcwItem*>(sm + kTcwItems) + 2 * tt;
    uint32_t got = 0;  // (ROWS) items taken from the ring
    auto put = [&](int idx, int turn) {
      if constexpr (ROWS) {  // from place to place, a word a lane: what an item's 24 words hold stays out of the registers
        const uint32_t from = smem_u32(ring_items + (got & 1)), to = smem_u32(place + turn);
        auto field = [&](size_t at) { return sm_load(from + (uint32_t)at); };
        if (!gave_up) gave_up = !wait_ring(&ifull[got & 1], (got >> 1) & 1);
        if (gave_up) {
          if (lane == 0) sm_store(to + offsetof(TcwItem, ntile), -1), sm_store(to + offsetof(TcwItem, nb), 0);
        } else {
          if (lane < (int)(sizeof(TcwItem) / 4)) sm_store(to + 4 * lane, sm_load(from + 4 * lane));
          __syncwarp();
          if (lane == 0) {
            const int tf = field(offsetof(TcwItem, p0)) + field(offsetof(TcwItem, i0)) + tt * qpt;  // the tile's positions
            const int tl = min(tf + qpt - 1, field(offsetof(TcwItem, last))), shift = field(offsetof(TcwItem, pl.sp)) - field(offsetof(TcwItem, pl.wb));
            const int low = a.window < 0 ? 0 : max(0, tl - a.window + 1);
            sm_store(to + offsetof(TcwItem, k_lo), field(offsetof(TcwItem, pl.sp)) + max(0, (low + kPage - 1) / kPage - field(offsetof(TcwItem, pl.wb))));
            sm_store(to + offsetof(TcwItem, k_hi), shift + min(tf + 1, field(offsetof(TcwItem, ctx))) / kPage);
            mbar_arrive(&iempty[got & 1]);
          }
        }
        ++got;
        __syncwarp();
        return;
      }
      if (tcw_item<SPLIT, ROWS>(ta, idx, it, false)) {
        const int tf = it.p0 + it.i0 + tt * qpt, tl = min(tf + qpt - 1, it.last);  // the tile's positions
        it.k_lo = it.pl.sp + max(0, (a.window < 0 ? 0 : max(0, tl - a.window + 1) + kPage - 1) / kPage - it.pl.wb);
        it.k_hi = it.pl.sp + min(tf + 1, it.ctx) / kPage - it.pl.wb;
      } else {
        it.ntile = it.nb = 0;
      }
      if (lane == 0) place[turn] = it;
      __syncwarp();
    };
    for (int idx = blockIdx.x, turn = 0; ROWS || idx < ta.total; idx += gridDim.x, turn ^= 1) {
      put(idx, turn);
      group_sync(12 + tt, 288);
      const TcwItem& my = place[turn];
      if (ROWS && my.ntile < 0) break;
      const int nb = my.nb;
      const bool active = tt < my.ntile;
      if (active && nb > 0) {
        for (int j = 0; j < nb; ++j) {
          if (!gave_up) gave_up = !__all_sync(0xffffffffu, mbar_wait_timed(&sfull[tt], (blocks + j) & 1, kWaitNs));
          if (gave_up && lane == 0) flags[tt] = 1;
          if (!gave_up) {
            gave_up = !landed(use + 2 * j + 1) || (j + 1 < nb && !landed(use + 2 * j + 2));
            const bool bad = flags[2] != 0;
            const int k0 = 2 * (my.j0 + j);
            if (tt == 0 && !gave_up && (bad || k0 < my.k_clean || min(k0 + 1, my.np - 1) >= my.k_held))
              clean_block<ROWS>(ta, my, k0, bad, sm + kTcwRing + (use + 2 * j + 1) % kTcwSlots * 32768, lane);
            if (!gave_up && lane == 0) mbar_arrive(&pready[tt]);
          }
        }
        blocks += nb;
      }
      use += 2 * nb;
    }
    if (gave_up && lane == 0) set_error(a.err, kErrTimeout);
  } else if (warp == kTcwMma) {
    // ---- products, issued by one thread, the tiles in turn: that keeps one tile's softmax under the other's
    // products (with a thread for each tile the two fall into step: 4650 cycles a pair of blocks, 2950 in turn).
    // This thread is what the products wait for, so it does nothing else: addresses are uniform and counted up (the
    // whole warp loops, an elected thread issues), one wait a tile, for P and the copies together.
    constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, 128), idesc_s64 = umma_idesc_bf16_f32(128, 64);
    constexpr uint32_t idesc_o = umma_idesc_bf16_f32(128, 128) | (1u << 16);  // B: channels contiguous
    constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // descriptors' high words: SBO, version, swizzle
    const uint32_t q_lo = ((sbase + kTcwQ) >> 4) | (1u << 16), ring = (sbase + kTcwRing) >> 4;
    auto logits = [&](int tt, uint32_t slot, bool half) {  // half: of the block's first page alone
      const uint32_t idesc = half ? idesc_s64 : idesc_s;
      const uint32_t k_lo = (ring + slot * 2048u) | (1u << 16);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        umma_ss(kTmS + tt * 128, q_lo + tt * 2048 + (s >> 2) * 1024 + (s & 3) * 2, k_lo + (s >> 2) * 1024 + (s & 3) * 2, kHi,
                idesc, s > 0);
      umma_commit(&sfull[tt]);
    };
    uint32_t s0 = 0, round0 = 0, phase0 = 0, phase1 = 0, items = 0;  // ring slot and round of the item's K_0; P's phases
    bool ok = true;
    int idx = blockIdx.x;
    uint32_t got = 0;  // (ROWS) items taken from the ring
    auto next_item = [&]() {  // to the next item with work, from idx on
      if constexpr (ROWS) {
        for (;;) {
          const uint32_t at = got & 1;
          ok = wait_ring(&ifull[at], (got >> 1) & 1);
          if (!ok) return false;
          it.nb = ring_items[at].nb;
          it.ntile = ring_items[at].ntile;
          it.j0 = ring_items[at].j0;
          it.np = ring_items[at].np;
          __syncwarp();
          if (lane == 0) mbar_arrive(&iempty[at]);
          ++got;
          if (it.ntile < 0) return false;
          if (it.nb > 0) return true;
        }
      }
      while (idx < ta.total && (!tcw_item<SPLIT, ROWS>(ta, idx, it, false) || it.nb == 0)) idx += gridDim.x;
      return idx < ta.total;
    };
    bool have = next_item();
    while (have && ok) {
      const int nb = __shfl_sync(0xffffffffu, it.nb, 0), nt = __shfl_sync(0xffffffffu, it.ntile, 0);  // uniform
      // the last block is one page: products over 64 keys (48 prompts of 1 to 2048 tokens 464 us, 471 over 128)
      const bool odd = __shfl_sync(0xffffffffu, 2 * (it.j0 + it.nb) - it.np, 0) > 0;
      ok = __all_sync(0xffffffffu, mbar_wait_timed(&full[s0], round0 & 1, kWaitNs) && mbar_wait_timed(qfull, items & 1, kWaitNs));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        for (int tt = 0; tt < nt; ++tt) logits(tt, s0, odd && nb == 1);
        umma_commit(&empty[s0]);
        if (nb == 1) umma_commit(qempty);
      }
      __syncwarp();
      if constexpr (!ROWS) {
        idx += gridDim.x;
        have = next_item();  // (worked out while the first softmax is at it)
      }
      uint32_t sv = s0 + 1 >= kTcwSlots ? 0 : s0 + 1, sk = sv + 1 >= kTcwSlots ? 0 : sv + 1;
      for (int j = 0; j < nb && ok; ++j) {
        const bool more = j + 1 < nb;
        const uint32_t v_lo = (ring + sv * 2048u) | ((16384u >> 4) << 16);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          if (tt < nt && ok) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&pready[tt], tt ? phase1 : phase0, kWaitLimit));
            if (ok) {
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 8; ++s)  // P: keys 0-63 in S's columns 0-31, the others in 64-95
                  if (s < 4 || more || !odd)
                    umma_ts(kTmO + tt * 128, kTmS + tt * 128 + (s >> 2) * 64 + 8 * (s & 3), v_lo + 128 * s, kHi,
                            idesc_o, j > 0 || s > 0);
                if (tt == nt - 1) umma_commit(&empty[sv]);
                if (more) {
                  logits(tt, sk, odd && j + 2 == nb);
                  if (tt == nt - 1) {
                    umma_commit(&empty[sk]);
                    if (j + 2 == nb) umma_commit(qempty);
                  }
                } else {
                  umma_commit(&odone[tt]);
                }
              }
              __syncwarp();
            }
            if (tt)
              phase1 ^= 1u;
            else
              phase0 ^= 1u;
          }
        }
        sv = sv + 2 >= kTcwSlots ? sv + 2 - kTcwSlots : sv + 2;
        sk = sk + 2 >= kTcwSlots ? sk + 2 - kTcwSlots : sk + 2;
      }
      const uint32_t next = s0 + 2 * nb;
      round0 += next / kTcwSlots;
      s0 = next % kTcwSlots;
      ++items;
      if constexpr (ROWS) have = ok && next_item();  // (not before: the next item is copied behind this one)
    }
    if (!ok && lane == 0) {
      flags[3] = 1;
      set_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    // ---- softmax: this thread's half of a row.  96 registers hold 32 weights, 32 logits on their way and little
    // else: the item stays in shared memory and is read where it is needed.
    const int lane = lane_id();
    const int t = warp >> 3, hf = (warp >> 2) & 1;
    const uint32_t ts = ((uint32_t)(32 * (warp & 3)) << 16) + kTmS + t * 128 + hf * 64, to = ts - kTmS + kTmO;
    const int pair_bar = 1 + 4 * t + (warp & 3);  // named barrier of the two warps that share these rows
    const uint32_t met_bad = sbase + kTcwBars + 160;
    static_assert((kTcwX & 1023u) == 0, "the halves' places differ in one address bit");
    const float c = a.sm_scale * kLog2eT;
    // this row's query of the item's (-1: none)
    const int ql = 32 * (warp & 3) + lane < qpt * g ? t * qpt + (32 * (warp & 3) + lane) / g : -1;
    uint32_t phases = 0;  // of S and O
    TcwItem* items = reinterpret_cast<TcwItem*>(sm + kTcwItems) + 2 * t;
    static_assert(4 * sizeof(TcwItem) <= kTcwX - kTcwItems, "the items' place");
    for (int idx = blockIdx.x, turn = 0; ROWS || idx < ta.total; idx += gridDim.x, turn ^= 1) {
      group_sync(12 + t, 288);  // the item is there (from the relay)
      const TcwItem& my = items[turn];
      if (ROWS && my.ntile < 0) break;
      const int nb = my.nb;
      if (t >= my.ntile) continue;
      float m = ROWS ? 0.f : -INFINITY, l = 0.f;
      bool anchored = false;  // (ROWS) the row has weight enough, or a maximum for its reference
      const bool live = ql >= 0 && my.i0 + ql < my.n;
#pragma unroll 1
      for (int j = 0; j < nb; ++j) {
        // (after a wait that gave up, the loop goes on without tensor memory: the barriers still meet)
        bool whole;
        uint32_t seen[2];  // the row's keys of this half
        auto look = [&](bool bad) {
          const int k0 = 2 * (my.j0 + j);
          whole = k0 >= my.k_lo && k0 + 1 < my.k_hi && !bad;
          seen[0] = seen[1] = ~0u;
          if (!whole) {
            const int base = block_page<ROWS>(ta, my, k0 + hf, bad), sinks = my.sinks;
            const int p = min(my.p0 + my.i0 + max(ql, 0), my.last);
            // (over packed rows p may be below -1: lim - p32 would leave 32 bits at a page that is not there)
            const int lim = max(0, min(p + 1, my.ctx)), low = a.window < 0 ? 0 : max(0, p - a.window + 1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int p32 = base + 32 * k;
              seen[k] = low_bits(lim - p32) & (low_bits(sinks - p32) | ~low_bits(low - p32));
            }
          }
        };
        // (under the products: behind them, in the way of the weights, 48 prompts of 1 to 2048 tokens took 453 us, now 436)
        look(false);
        if (!gave_up) gave_up = !__all_sync(0xffffffffu, mbar_wait_bounded(&sfull[t], phases & 1u, kWaitLimit));
        phases ^= 1u;
        tc_fence_after();
        if (!ROWS && sm_load(met_bad) != 0) look(true);
        uint32_t w[32];
        float2 sum = make_float2(0.f, 0.f);
        float mc = m == -INFINITY ? 0.f : m * c;
        if (!gave_up && (ROWS || j > 0)) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t s[2][16];
            tmem_ld32(ts + 32 * k, s);
            if (!whole) {  // (most parts of a masked block are seen by all of the warp's rows; 442 us for 439 otherwise)
              if (__any_sync(0xffffffffu, (seen[k] & 0xffffu) != 0xffffu)) hide(s[0], seen[k], 0);
              if (__any_sync(0xffffffffu, (seen[k] >> 16) != 0xffffu)) hide(s[1], seen[k], 16);
            }
            weights(s[0], c, mc, sum, w + 16 * k);
            weights(s[1], c, mc, sum, w + 16 * k + 8);
          }
        }
        // (rows that are no query's hold leftovers: they never ask)
        const bool low = ROWS ? !anchored && l + sum.x + sum.y < kLowSum : m == -INFINITY;
        const bool move = live && (!(l + sum.x + sum.y < kTopSum) || (low && (seen[0] | seen[1]) != 0));
        if ((!ROWS && j == 0) || pair_any(pair_bar, move)) {
          // the logits are still in place: the rows' maxima anew, O and l along, and the weights again
          uint32_t s[16];
          float mb = -INFINITY;
#pragma unroll 1
          for (int k = 0; k < 4 && !gave_up; ++k) {
            tmem_ld16_start(ts + 16 * k, s);
            tmem_ld16_wait(s);
            hide(s, (k & 2 ? seen[1] : seen[0]) >> (16 * (k & 1)), 0);
            mb = fmaxf(mb, max16(s));
          }
          if (l >= 0.5f * kTopSum) mb = fmaxf(mb, m + __fdividef(39.f, c));  // (many keys, of which none stands out)
          const uint32_t mine = sbase + kTcwX + 4 * (256 * t + 128 * hf + 32 * (warp & 3) + lane_id()), theirs = mine ^ 512u;
          sm_store(mine, __float_as_int(mb));
          group_sync(pair_bar, 64);
          mb = fmaxf(mb, __int_as_float(sm_load(theirs)));
          float f = 1.f;
          // (the row that asked for it does move: its sum was 2^39, or this block's is and holds a weight of 2^33)
          if constexpr (ROWS) {  // (both halves decide alike: by the row's maximum, and by its weight so far)
            group_sync(pair_bar, 64);
            sm_store(mine, __float_as_int(l));
            group_sync(pair_bar, 64);
            const float row = l + __int_as_float(sm_load(theirs));
            const bool down = row < kLowSum && mb > -INFINITY;
            if (down || (mb - m) * c > 8.f) {
              // (what it has, 2^-126 or more, may come from higher logits than this block's)
              const float to = down && row > 0.f ? fmaxf(mb, m + __log2f(row) / c) : mb;
              f = row > 0.f ? exp2_t((m - to) * c) : 0.f;
              m = to;
              l *= f;
            }
            anchored = anchored || row >= kLowSum || mb > -INFINITY;
          } else if (mb > m && (m == -INFINITY || (mb - m) * c > 8.f)) {
            f = m == -INFINITY ? 0.f : exp2_t((m - mb) * c);
            m = mb;
            l *= f;
          }
          mc = m == -INFINITY ? 0.f : m * c;
          sum = make_float2(0.f, 0.f);
          if (!gave_up) {
            if (j > 0) {
#pragma unroll 1
              for (int k = 0; k < 4; ++k) {
                uint32_t o[16];
                tmem_ld16_start(to + 16 * k, o);
                tmem_ld16_wait(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st8u(to + 16 * k, *reinterpret_cast<uint32_t(*)[8]>(o));
                tmem_st8u(to + 16 * k + 8, *reinterpret_cast<uint32_t(*)[8]>(o + 8));
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tmem_ld16_start(ts + 16 * k, s);
              tmem_ld16_wait(s);
              hide(s, seen[k >> 1], 16 * (k & 1));
              weights(s, c, mc, sum, w + 8 * k);
            }
          }
        }
        l += sum.x + sum.y;
        if (!gave_up) {
          tmem_st32u(ts, w);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !gave_up) mbar_arrive(&pready[t]);
      }
      group_sync(pair_bar, 64);  // (the row's last exchange is read)
      if (nb > 0) {  // O is complete
        if (!gave_up) gave_up = !__all_sync(0xffffffffu, mbar_wait_timed(&odone[t], phases >> 1, kWaitNs));
        phases ^= 2u;
      }
      tc_fence_after();
      const uint32_t mine = sbase + kTcwX + 4 * (256 * t + 128 * hf + 32 * (warp & 3) + lane_id()), theirs = mine ^ 512u;
      sm_store(mine, __float_as_int(l));
      group_sync(pair_bar, 64);
      l += __int_as_float(sm_load(theirs));
      if (!SPLIT && l == 0.f && live && row_sees<ROWS>(ta, my, ql, sm_load(met_bad) != 0)) l = CUDART_NAN_F;
      tcw_result<SPLIT>(ta, items[turn], warp, lane, to, ql, live, !gave_up && nb > 0, m, l);
      // (the next item's products write O only once its first P is there, so after these loads)
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTcwMma) {
    tc_fence_after();
    tmem_dealloc(0, 512);
  }
}

// The records of each group's items into the result, in item order: a warp a row.  A kernel of its own, so that all
// SMs have a part in it: with the last item of each group joining the rest, 32 tokens at 4096 of one request took 72 us,
// now 18; 256 at 100,000 329 us, now 300.
constexpr int kJoinThreads = 256;
template <bool ROWS>
__global__ void __launch_bounds__(kJoinThreads) window_join_kernel(const __grid_constant__ TcwArgs ta) {
  const WindowLaunch& a = ta.a;
  const int g = a.Hq / a.Hkv, lane = threadIdx.x & 31, i = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int q = i / g, head = i - q * g;  // the row's query among its tile pair's, and its query head
  int pair, h, p0, n, row0;
  const int b = ta.by_heads.divide(ta.by_tiles.divide((int)blockIdx.y, pair), h);
  griddep_wait();
  griddep_launch_dependents();
  if (!(ROWS ? rows_span(a.tok, ta.keys, b, n, row0, p0, p0, a.err, false) : token_span(a.tok, b, p0, n, row0, a.err, false)) ||
      q >= 2 * ta.qpt || pair * 2 * ta.qpt + q >= n) return;
  const int tt = q >= ta.qpt, r = (q - tt * ta.qpt) * g + head;
  const float c = a.sm_scale * kLog2eT;
  constexpr size_t kStep = (size_t)256 * kRowFloats;  // from one item's record to the next's
  const float* rec = reinterpret_cast<const float*>(a.workspace + a.plan.off_records) +
                     (size_t)((b * a.Hkv + h) * ta.tiles + pair) * ta.items * kStep + (size_t)128 * tt * kRowFloats;
  float M = -INFINITY, L = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < ta.items; i0 += 32) {  // lane i: item i0 + i's maximum and sum
    const int count = min(32, ta.items - i0);
    const float* first = rec + i0 * kStep;
    float m = -INFINITY, l = 0.f;
    if (lane < count) {
      m = __ldcg(first + lane * kStep + 128 * kD + r);
      l = __ldcg(first + lane * kStep + 129 * kD + r);
    }
    // the first records' rows travel beside their maxima (64 tokens at 1000 12.2 us, now 11.4)
    constexpr int kEarly = 4;
    float4 early[kEarly];
    auto record = [&](int k) { return __ldcg(reinterpret_cast<const float4*>(first + k * kStep + r * kD) + lane); };
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (k < count) early[k] = record(k);
    const float top = fmaxf(M, warp_max(m)), down = M == -INFINITY ? 0.f : exp2_t((M - top) * c);
    const float f = m == -INFINITY ? 0.f : exp2_t((m - top) * c);
    M = top;
    L = L * down + warp_sum(l * f);
    y = make_float4(y.x * down, y.y * down, y.z * down, y.w * down);
    auto add = [&](int k, const float4& u) {  // (an item without keys wrote m and l alone)
      const float fk = __shfl_sync(0xffffffffu, f, k);
      if (fk > 0.f) y = make_float4(fmaf(u.x, fk, y.x), fmaf(u.y, fk, y.y), fmaf(u.z, fk, y.z), fmaf(u.w, fk, y.w));
    };
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (k < count) add(k, early[k]);
#pragma unroll 8
    for (int k = kEarly; k < count; ++k) add(k, record(k));
  }
  if (L == 0.f) {
    TcwItem it;
    const int idx = (b * ta.items * a.Hkv + h) * ta.tiles + pair;
    if (tcw_item<true, ROWS>(ta, idx, it, false) && row_sees<ROWS>(ta, it, q, true)) L = CUDART_NAN_F;
  }
  const float f = L == 0.f ? 0.f : 1.f / L;  // (a sum that is not a number reaches the row: its terms above were left out)
  reinterpret_cast<uint2*>(a.out + ((size_t)(row0 + pair * 2 * ta.qpt + q) * a.Hq + h * g + head) * kD)[lane] =
      make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
}

}  // namespace

// Items per (tile pair, KV head): the fewest rounds of the grid times an item's length in key blocks (plus a
// fixed part: the pipeline's fill and drain, the join), at most two items per SM.  The parts in key blocks: with 0 to 16
// for the fixed one the times are the same (256 tokens at 100,000 291 to 295 us, 302 with 32), with 0 to 3 for the join
// too (64 tokens at 1000 14.5 us, 21.1 with 8).
WindowPlan plan_window_tc(int64_t batch, int64_t max_tokens, int Hq, int Hkv, int64_t max_keys, int num_sms) {
  WindowPlan p;
  const int qpt = 128 / (Hq / Hkv);
  const int64_t groups = batch * Hkv * ((max_tokens + 2 * qpt - 1) / (2 * qpt));
  const int64_t blocks = (max_keys + 2 * qpt + 127) / 128 + 1;
  constexpr int kFixed = 8;
  const int64_t most = std::min<int64_t>(blocks / 2, kCutBlocks * (int64_t)num_sms / std::max<int64_t>(groups, 1));
  int64_t best = INT64_MAX;
  for (int64_t n = 1; n <= std::max<int64_t>(most, 1); ++n) {
    const int64_t waves = (groups * n + num_sms - 1) / std::max(num_sms, 1);
    const int64_t cost = waves * (kFixed + (blocks + n - 1) / n + (n > 1 ? 3 : 0));
    if (cost < best) {
      best = cost;
      p.items = (int)n;
    }
  }
  p.off_records = window_counter_bytes(num_sms);
  p.total = p.off_records + (size_t)kCutBlocks * num_sms * 256 * kRowFloats * sizeof(float);
  return p;
}

// rows: keys in packed rows (null: pages)
static cudaError_t launch_tc(const WindowLaunch& a, const KeyRows* rows, int batch, cudaStream_t stream) {
  static std::atomic<uint64_t> done[4];
  const bool split = a.plan.items > 1;
  const void* fn = rows == nullptr ? (split ? reinterpret_cast<const void*>(window_tc_kernel<true, false>)
                                            : reinterpret_cast<const void*>(window_tc_kernel<false, false>))
                                   : (split ? reinterpret_cast<const void*>(window_tc_kernel<true, true>)
                                            : reinterpret_cast<const void*>(window_tc_kernel<false, true>));
  const cudaError_t e = smem_attr_once(fn, kTcwSmem, done[2 * (rows != nullptr) + split]);
  if (e != cudaSuccess) return e;
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t r = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (r != cudaSuccess || q != cudaDriverEntryPointSuccess) return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  // the pools as [num_pages][Hkv 64 rows][128 channels], boxes of 64 channels x one head's page; packed rows as
  // [Hkv][n_keys][128 channels], boxes of 64 channels x 64 rows (zeros behind the last) x one head
  CUtensorMap tm[3];
  const cuuint32_t estride[3] = {1, 1, 1};
  for (int i = 0; i < 2; ++i) {
    cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)a.Hkv * kPage, (cuuint64_t)a.pages.num_pages};
    cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)a.Hkv * kPage * kD * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)kPage, 1};
    const uint16_t* base = i ? a.v_pages : a.k_pages;
    if (rows != nullptr) {
      dims[1] = (cuuint64_t)std::max(rows->n_keys, 1), dims[2] = (cuuint64_t)a.Hkv;
      strides[0] = (cuuint64_t)(i ? rows->v_stride : rows->k_stride) * 2, strides[1] = (cuuint64_t)kD * 2;
      base = rows->n_keys == 0 ? a.q : i ? rows->v : rows->k;  // (without keys nothing is read)
    }
    const CUresult r = encode(&tm[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base),
                              dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  TcwArgs ta;
  ta.a = a;
  ta.items = a.plan.items;
  ta.by_items = Divisor(ta.items);
  ta.by_heads = Divisor(a.Hkv);
  ta.batch = batch;
  ta.by_batch = Divisor(batch);
  if (rows != nullptr) ta.keys = *rows;
  ta.tickets = reinterpret_cast<int*>(a.workspace + window_counter_bytes(a.num_sms) - 256);
  ta.g = a.Hq / a.Hkv;
  ta.qpt = 128 / ta.g;
  ta.tiles = (a.tok.max_tokens + 2 * ta.qpt - 1) / (2 * ta.qpt);
  ta.by_tiles = Divisor(ta.tiles);
  long long total = (long long)ta.tiles * batch * a.Hkv * ta.items;
  // (whole items over packed rows are counted on the device, n_tokens Hkv at most: a loose bound is no error)
  if (rows != nullptr && !split) total = std::min<long long>(total, INT32_MAX - 65536);
  if (total > INT32_MAX - 65536) return cudaErrorInvalidValue;
  ta.total = (int)total;
  {  // the queries as [n_tokens][Hq][128], boxes of 64 channels x one KV head's g heads x a tile's queries
    const cuuint64_t qdims[3] = {(cuuint64_t)kD, (cuuint64_t)a.Hq, (cuuint64_t)a.tok.n_tokens};
    const cuuint64_t qstrides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t qbox[3] = {64, (cuuint32_t)(a.Hq / a.Hkv), (cuuint32_t)ta.qpt};
    const CUresult r = encode(&tm[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q), qdims, qstrides, qbox,
                              estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  void* args[] = {&ta, &tm[0], &tm[1], &tm[2]};
  const cudaError_t r = launch_pdl(fn, dim3((unsigned)std::min<long long>(total, std::max(a.num_sms, 1))),
                                   dim3(kTcwThreads), kTcwSmem, stream, args);
  if (r != cudaSuccess || !split) return r;
  const int group_rows = std::min(a.tok.max_tokens, 2 * ta.qpt) * (a.Hq / a.Hkv);
  return launch_pdl(rows == nullptr ? reinterpret_cast<const void*>(window_join_kernel<false>)
                                    : reinterpret_cast<const void*>(window_join_kernel<true>),
                    dim3((unsigned)(group_rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32), (unsigned)(total / ta.items)),
                    dim3(kJoinThreads), 0, stream, args);
}

cudaError_t launch_window_tc(const WindowLaunch& a, cudaStream_t stream) {
  return launch_tc(a, nullptr, a.pages.batch, stream);
}

cudaError_t launch_prompt(const WindowLaunch& a, const KeyRows& rows, int batch, cudaStream_t stream) {
  return launch_tc(a, &rows, batch, stream);
}

}  // namespace oscar
