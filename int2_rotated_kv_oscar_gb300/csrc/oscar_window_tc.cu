// Windowed attention of chunks and prompts over BF16 pages on the
// 5th-generation tensor cores.
//
// A block takes two tiles of 128 rows of one (request, KV head): row r of a
// tile is query r / g of the tile and query head r % g, so the g heads that
// share the keys share each of their copies.  For a block of 128 keys (two
// pages)
//   S = Q K^T   M 128 (rows), N 128 (keys), K 16 a step; both from shared memory
//   P = exp2(c S - m), rounded to bf16 (one term, at most 2^-8 of a weight, as
//       the result is; c = sm_scale log2 e, m the row's running maximum)
//   O += P V    P from tensor memory (over S's columns), V as it lies in
//       the page: keys along K, channels contiguous (an "MN-major" operand)
// with S, O and the sums in fp32.  Tensor memory: S of both tiles (2 x 128
// columns), O of both (2 x 128).
//
//   warps 0-15   softmax: tile w / 8, keys 64 (w / 4 % 2) .. + 63 of a block; a
//                thread is half a row (its TMEM lane), so that the time from S to
//                P, which the products wait for, is that of 64 exponentials
//   warp 16      copies K and V blocks (TMA, 64 channels x 64 rows, 128-byte
//                swizzle) into a ring of five 32 KB slots, in the order of
//                use: K_0, V_0, K_1, V_1, ...
//   warp 17      one thread issues the MMAs, tile by tile: S_t(j + 1) right
//                behind P_t V(j), so that one tile's softmax runs under the other
//                tile's products
//   warps 18, 19 wait for the products of tile 0, 1 and meet its softmax warps at
//                a hardware barrier: sixteen warps that poll took more issue slots
//                than their exponentials
// A block sees only the pages that some of its queries see.  With few blocks
// the keys are split over several (items) whose records (m, l, O) the last one
// to finish joins in item order.

#include "oscar_paged.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda.h>
#include <cudaTypedefs.h>

namespace oscar {
namespace {

constexpr float kLog2eT = 1.4426950408889634f;
constexpr int kTcwThreads = 20 * 32;
constexpr int kTcwCopy = 16, kTcwMma = 17, kTcwRelay = 18;  // warps
constexpr int kTcwSlots = 5;
constexpr uint32_t kTcwQ = 0;                    // queries: [tile][2 x 64 channels][128 rows][128 B]
constexpr uint32_t kTcwRing = 65536;             // slots: [2 x 64 channels][128 keys][128 B]
constexpr uint32_t kTcwBars = kTcwRing + kTcwSlots * 32768;
constexpr uint32_t kTcwX = kTcwBars + 256;        // what the two halves of a row tell each other: [tile][half][128 rows] float
constexpr size_t kTcwSmem = kTcwX + 2048;        // (all of it dynamic, so that it begins where the block's memory does)
constexpr uint32_t kTmS = 0, kTmO = 256;         // TMEM columns of S and O, 128 a tile
// A row's weights are taken relative to the maximum of the first block that it saw something of, until half a
// block's sum of them reaches kTopSum (2^40; fp32 and bf16 reach 2^127): then the maximum is found anew, and O
// and l move.  So the common block needs no maximum: its exponentials start with the first logits that arrive
// (a block that moves takes 2000 cycles more; at 2^16 every fifth block did).
constexpr float kTopSum = 1099511627776.0f;
constexpr int kRowFloats = kD + 2;               // a row's record: O[128], m, l

struct TcwArgs {
  WindowLaunch a;
  int items, tiles, qpt;  // blocks per (tile pair, KV head), tile pairs per request, queries per tile
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

// 32 columns of this thread's lane, in flight until the wait that names the same registers.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// The n lowest of 32 bits (n may lie outside 0..32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Logits whose bit in `seen` is 0 drop out.
__device__ __forceinline__ void hide(uint32_t (&s)[32], uint32_t seen) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(seen & (1u << e))) s[e] = 0xff800000u;
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float m[4] = {__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]), __uint_as_float(s[3])};
#pragma unroll
  for (int e = 4; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], __uint_as_float(s[e]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// exp2(c s - mc) of 32 logits: their sum, and 16 pairs of bf16.
__device__ __forceinline__ void weights(const uint32_t (&s)[32], float c, float mc, float2& sum, uint32_t* w) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 y = ffma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(c, c),
                           make_float2(-mc, -mc));
    const float2 p = make_float2(exp2_t(y.x), exp2_t(y.y));
    sum = fadd2(sum, p);
    w[e >> 1] = pack_bf16x2(p.x, p.y);
  }
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
  return x != 0;
}

// Whether any thread of the two warps at named barrier `id` says so in round `round` (> 0, and larger each time):
// a word of shared memory that only a thread with news writes.
__device__ __forceinline__ bool pair_any(int id, volatile int* word, int round, bool x) {
  if (x) *word = round;
  group_sync(id, 64);
  return *word == round;
}

// The pages that some query of a block sees: logical pages [0, sp) and [wb, we).
struct PageList {
  int sp, wb, we;
  __device__ __forceinline__ int count() const { return sp + max(0, we - wb); }
  __device__ __forceinline__ int page(int k) const { return k < sp ? k : wb + (k - sp); }
};

__global__ void __launch_bounds__(kTcwThreads, 1)
    window_tc_kernel(const __grid_constant__ TcwArgs ta, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv) {
  const WindowLaunch& a = ta.a;
  extern __shared__ __align__(1024) uint8_t sm[];
  // (by way of a shuffle, so that the compiler knows the warp's role to be uniform)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // block -> (tile pair, request, KV head, item); later tiles (more keys) first
  int x = blockIdx.x;
  const int item = x % ta.items;
  x /= ta.items;
  const int h = x % a.Hkv;
  x /= a.Hkv;
  const int b = x % a.pages.batch, pair = ta.tiles - 1 - x / a.pages.batch;
  const int g = a.Hq / a.Hkv, qpt = ta.qpt;
  int p0, n, row0;
  if (!token_span(a.tok, b, p0, n, row0, a.err, threadIdx.x == 0)) return;
  const int i0 = pair * 2 * qpt;  // the block's first query of the request
  if (i0 >= n) return;
  const int i1 = min(i0 + 2 * qpt, n);
  const int ntile = i0 + qpt < n ? 2 : 1;
  // positions: a negative one (or one past 2^31) sees nothing
  const long long plast = (long long)p0 + i1 - 1;
  if ((p0 + i0 < 0 || p0 < 0 || plast > INT32_MAX - 1) && threadIdx.x == 0) set_error(a.err, kErrLength);
  int ctx = max(a.ctx_len[b], 0);
  if (p0 < 0 || plast > INT32_MAX - 1) ctx = 0;
  const long long limit = (long long)a.pages.max_pages * kPage;
  if (ctx > limit) {
    if (min(plast + 1, (long long)ctx) > limit && threadIdx.x == 0) set_error(a.err, kErrLength);
    ctx = (int)limit;
  }
  const int hi = (int)min(plast + 1, (long long)ctx);  // no query of the block sees hi or beyond
  const int first = p0 + i0;
  // the windows of its queries start at lo (a window of 0 holds nothing)
  const int lo = a.window < 0 ? 0 : a.window == 0 ? max(hi, 1) : max(0, first - a.window + 1);
  const int sinks = min(a.sinks, hi);
  PageList pl;
  pl.we = (hi + kPage - 1) / kPage;
  pl.sp = lo > 0 ? (sinks + kPage - 1) / kPage : 0;
  pl.wb = lo >= hi ? pl.we : max(lo / kPage, pl.sp);
  const int np = pl.count(), nblocks = (np + 1) / 2;
  const int j0 = (int)((long long)nblocks * item / ta.items), j1 = (int)((long long)nblocks * (item + 1) / ta.items);
  const int nb = j1 - j0;
  // a page outside the pool: an error, and its positions are left out
  bool bad = false;
  for (int k = 2 * j0 + threadIdx.x; k < min(2 * j1, np); k += kTcwThreads)
    bad = bad || page_of(a.pages, b, pl.page(k), a.err, true) < 0;

  const uint32_t sbase = smem_u32(sm);
  float(*sm_x)[2][128] = reinterpret_cast<float(*)[2][128]>(sm + kTcwX);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kTcwBars);  // [slots] copies landed
  uint64_t* empty = full + kTcwSlots;                           // [slots] read by its products
  uint64_t* sfull = empty + kTcwSlots;                          // [2] S of tile t holds a block's logits (and O its last product)
  uint64_t* pready = sfull + 2;                                 // [2] P of tile t written
  uint64_t* odone = pready + 2;                                 // [2] O of tile t complete
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(odone + 2);
  volatile int* last = reinterpret_cast<volatile int*>(tmem_at + 1);
  volatile int* dead = last + 1;  // [2] a relay's wait gave up
  if (threadIdx.x < 8) reinterpret_cast<int*>(sm + kTcwBars + 192)[threadIdx.x] = 0;  // the pairs' words
  if (threadIdx.x < 2) dead[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcwSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[t], 9);  // the tile's softmax warps, and its relay for the copies
      mbar_init(&odone[t], 1);
    }
    fence_mbar_init();
  }
  if (warp == kTcwMma) tmem_alloc(tmem_at, 512);
  if (warp == kTcwCopy && lane == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  const int t = warp >> 3, hf = (warp >> 2) & 1, row = 32 * (warp & 3) + lane;  // softmax warps: tile, half and row
  const int qi = i0 + t * qpt + row / g, head = row % g;
  const bool live = warp < kTcwCopy && row < qpt * g && qi < n;
  if (warp < kTcwCopy && t < ntile) {  // the queries, into the swizzled operand layout
    const uint4* src = reinterpret_cast<const uint4*>(a.q + (size_t)(row0 + qi) * a.q_stride + (size_t)(h * g + head) * kD);
    uint8_t* dst = sm + kTcwQ + t * 32768 + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 v = live ? src[8 * hf + c] : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(dst + hf * 16384 + ((c ^ (row & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  const bool any_bad = __syncthreads_or(bad);
  tc_fence_after();
  const uint32_t tbase = 0;  // (an allocation of all 512 columns begins at column 0)
  bool gave_up = false;

  float m = -INFINITY, l = 0.f;
  if (warp == kTcwCopy) {
    // ---- copies: use 0 is K_0, 2 j + 1 is V_j, 2 j + 2 is K_(j + 1)
    int phys_l = -1, fetched = 0;
    auto phys_of = [&](int k) {  // k-th page of this item (whole warp)
      if (k >= fetched) {
        phys_l = -1;
        const int kk = 2 * j0 + fetched + lane;
        if (kk < min(2 * j1, np)) phys_l = page_of(a.pages, b, pl.page(kk), a.err, false);
        fetched += 32;
      }
      return __shfl_sync(0xffffffffu, phys_l, k & 31);
    };
    int vp0 = -1, vp1 = -1;  // V's pages of the block whose K came last
    for (int u = 0; u < 2 * nb && !gave_up; ++u) {
      const bool is_v = (u & 1) != 0;
      int q0, q1;
      if (u == 0 || !is_v) {
        q0 = phys_of(u);  // block u / 2: pages u, u + 1
        q1 = phys_of(u + 1);
      }
      // order of use: K_0, V_0, K_1, ... : V_j goes out before K_(j + 1)
      if (is_v) {
        q0 = vp0;
        q1 = vp1;
      } else {
        vp0 = q0;
        vp1 = q1;
      }
      const int slot = u % kTcwSlots;
      if (lane == 0) {
        if (u >= kTcwSlots && !mbar_wait_timed(&empty[slot], ((u / kTcwSlots) - 1) & 1, kWaitNs)) gave_up = true;
        if (!gave_up) {
          uint8_t* dst = sm + kTcwRing + slot * 32768;
          mbar_arrive_expect_tx(&full[slot], (q0 >= 0 ? 16384u : 0u) + (q1 >= 0 ? 16384u : 0u));
          const void* tm = is_v ? static_cast<const void*>(&tmv) : static_cast<const void*>(&tmk);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (q0 >= 0) tma_load_page(dst + half * 16384, tm, 64 * half, h * kPage, q0, &full[slot]);
            if (q1 >= 0) tma_load_page(dst + half * 16384 + 8192, tm, 64 * half, h * kPage, q1, &full[slot]);
          }
        }
      }
      gave_up = __shfl_sync(0xffffffffu, gave_up, 0);
    }
    if (gave_up && lane == 0) {
      set_error(a.err, kErrTimeout);
      // the copies still in flight land before the block ends
      for (int i = 0; i < kTcwSlots; ++i) {
        mbar_wait_timed(&full[i], 0, kWaitNs);
        mbar_wait_timed(&full[i], 1, kWaitNs);
      }
    }
  } else if (warp >= kTcwRelay) {
    // ---- relays: the products' logits to the softmax warps, and the copies that the next products read
    const int tt = warp - kTcwRelay;
    auto landed = [&](int u) {
      return __all_sync(0xffffffffu, mbar_wait_timed(&full[u % kTcwSlots], (u / kTcwSlots) & 1, kWaitNs)) != 0;
    };
    for (int j = 0; j <= nb && tt < ntile && nb > 0; ++j) {
      if (!gave_up) gave_up = !__all_sync(0xffffffffu, j < nb ? mbar_wait_timed(&sfull[tt], j & 1, kWaitNs)
                                                              : mbar_wait_timed(&odone[tt], 0, kWaitNs));
      if (gave_up && lane == 0) dead[tt] = 1;
      group_sync(9 + tt, 288);
      if (j < nb && !gave_up) {
        gave_up = !landed(2 * j + 1) || (j + 1 < nb && !landed(2 * j + 2));
        if (!gave_up && lane == 0) mbar_arrive(&pready[tt]);
      }
    }
    if (gave_up && lane == 0) set_error(a.err, kErrTimeout);
  } else if (warp > kTcwCopy) {
    // ---- products, issued by one thread, the tiles in turn: that keeps one tile's softmax under the other's
    // products (with a thread for each tile the two fall into step: 4650 cycles a pair of blocks).  This thread is
    // what the products wait for, so it does nothing else: addresses are uniform and counted up (the whole warp
    // loops, an elected thread issues), one wait a tile, for P and the copies together.
    const int nb = __shfl_sync(0xffffffffu, j1 - j0, 0), nt = __shfl_sync(0xffffffffu, ntile, 0);  // uniform
    if (nb > 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, 128);
      constexpr uint32_t idesc_o = umma_idesc_bf16_f32(128, 128) | (1u << 16);  // B: channels contiguous
      constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // descriptors' high words: SBO, version, swizzle
      const uint32_t q_lo = ((sbase + kTcwQ) >> 4) | (1u << 16), ring = (sbase + kTcwRing) >> 4;
      auto logits = [&](int tt, uint32_t slot) {
        const uint32_t k_lo = (ring + slot * 2048u) | (1u << 16);
#pragma unroll
        for (int s = 0; s < 8; ++s)
          umma_ss(kTmS + tt * 128, q_lo + tt * 2048 + (s >> 2) * 1024 + (s & 3) * 2, k_lo + (s >> 2) * 1024 + (s & 3) * 2, kHi,
                  idesc_s, s > 0);
        umma_commit(&sfull[tt]);
      };
      bool ok = __all_sync(0xffffffffu, mbar_wait_timed(&full[0], 0, kWaitNs));
      if (ok) {
        tc_fence_after();
        if (elect_one()) {
          for (int tt = 0; tt < nt; ++tt) logits(tt, 0);
          umma_commit(&empty[0]);
        }
        __syncwarp();
      }
      uint32_t sv = 1, sk = 2, phase = 0;
      for (int j = 0; j < nb && ok; ++j) {
        const bool more = j + 1 < nb;
        const uint32_t v_lo = (ring + sv * 2048u) | ((16384u >> 4) << 16);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          if (tt < nt && ok) {
            ok = __all_sync(0xffffffffu, mbar_wait_timed(&pready[tt], phase, kWaitNs));
            if (ok) {
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int s = 0; s < 8; ++s)  // P: keys 0-63 in S's columns 0-31, the others in 64-95
                  umma_ts(kTmO + tt * 128, kTmS + tt * 128 + (s >> 2) * 64 + 8 * (s & 3), v_lo + 128 * s, kHi, idesc_o,
                          j > 0 || s > 0);
                if (tt == nt - 1) umma_commit(&empty[sv]);
                if (more) {
                  logits(tt, sk);
                  if (tt == nt - 1) umma_commit(&empty[sk]);
                } else {
                  umma_commit(&odone[tt]);
                }
              }
              __syncwarp();
            }
          }
        }
        phase ^= 1u;
        sv = sv + 2 >= kTcwSlots ? sv + 2 - kTcwSlots : sv + 2;
        sk = sk + 2 >= kTcwSlots ? sk + 2 - kTcwSlots : sk + 2;
      }
      if (!ok && lane == 0) set_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (t < ntile) {
    // ---- softmax: this thread's half of a row
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tbase + lanes + kTmS + t * 128 + hf * 64, to = tbase + lanes + kTmO + t * 128 + hf * 64;
    const int pair_bar = 1 + 4 * t + (warp & 3);  // named barrier of the two warps that share these rows
    volatile int* pair_word = reinterpret_cast<volatile int*>(sm + kTcwBars + 192) + 4 * t + (warp & 3);
    const float c = a.sm_scale * kLog2eT;
    const int tf = first + t * qpt, tl = min(tf + qpt - 1, (int)plast);  // the tile's positions
    const int p = min(p0 + qi, (int)plast);
    const int lim = min(p + 1, ctx), low = a.window < 0 ? 0 : max(0, p - a.window + 1);
    // pages (of the block's list) of which every row of the tile sees all: [k_lo, k_hi), past the sinks
    const int k_lo = pl.sp + max(0, (a.window < 0 ? 0 : max(0, tl - a.window + 1) + kPage - 1) / kPage - pl.wb);
    const int k_hi = any_bad ? 0 : pl.sp + min(tf + 1, ctx) / kPage - pl.wb;
    for (int j = 0; j < nb; ++j) {
      const int k0 = 2 * (j0 + j);
      const bool whole = k0 >= k_lo && k0 + 1 < k_hi;
      uint32_t seen[2] = {~0u, ~0u};  // the row's keys of this half
      if (!whole) {
        // (a page outside the pool, or none: past every position)
        int base[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int lp = k0 + k < np ? pl.page(k0 + k) : -1;
          base[k] = lp < 0 || (any_bad && page_of(a.pages, b, lp, a.err, false) < 0) ? INT32_MAX - 63 : lp * kPage;
        }
        // a V row that no query of the block sees may hold anything: it becomes zeros (by both tiles, each before
        // its own product)
        const int at = (row < 64 ? base[0] : base[1]) + (row & 63);
        const bool stale = !(at < hi && (at < sinks || at >= lo));
        if (__any_sync(0xffffffffu, stale) && !gave_up) {
          const int uv = 2 * j + 1, sv = uv % kTcwSlots;
          gave_up = !__all_sync(0xffffffffu, mbar_wait_timed(&full[sv], (uv / kTcwSlots) & 1, kWaitNs));
          if (!gave_up && stale) {
            uint8_t* v = sm + kTcwRing + sv * 32768 + hf * 16384 + row * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(v + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int p32 = base[hf] + 32 * k;
          seen[k] = low_bits(lim - p32) & (low_bits(sinks - p32) | ~low_bits(low - p32));
        }
      }
      // after a wait that gave up, the loop goes on without tensor memory: the barriers still meet
      group_sync(9 + t, 288);
      gave_up = gave_up || dead[t] != 0;
      tc_fence_after();
      uint32_t w[32];
      float2 sum = make_float2(0.f, 0.f);
      float mc = m == -INFINITY ? 0.f : m * c;
      if (!gave_up) {
        uint32_t s0[32], s1[32];
        tmem_ld32_start(ts, s0);
        tmem_ld32_wait(s0);
        tmem_ld32_start(ts + 32, s1);
        if (!whole) hide(s0, seen[0]);
        weights(s0, c, mc, sum, w);
        tmem_ld32_wait(s1);
        if (!whole) hide(s1, seen[1]);
        weights(s1, c, mc, sum, w + 16);
      }
      const bool move = !(sum.x + sum.y < kTopSum) || (m == -INFINITY && (seen[0] | seen[1]) != 0);
      if (pair_any(pair_bar, pair_word, j + 1, move)) {
        // the logits are still in place: the rows' maxima anew, O and l along, and the weights again
        uint32_t s0[32];
        float mb = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < 2 && !gave_up; ++k) {
          tmem_ld32_start(ts + 32 * k, s0);
          tmem_ld32_wait(s0);
          hide(s0, k ? seen[1] : seen[0]);
          mb = fmaxf(mb, max32(s0));
        }
        sm_x[t][hf][row] = mb;
        group_sync(pair_bar, 64);
        mb = fmaxf(mb, sm_x[t][hf ^ 1][row]);
        float f = 1.f;
        // (a half's sum of kTopSum holds a weight of 2^10 at least, so the row that asked for it does move)
        if (mb > m && (m == -INFINITY || (mb - m) * c > 8.f)) {
          f = m == -INFINITY ? 0.f : exp2_t((m - mb) * c);
          m = mb;
          l *= f;
        }
        mc = m == -INFINITY ? 0.f : m * c;
        sum = make_float2(0.f, 0.f);
        if (!gave_up) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (j > 0) {
              float o[32];
              tmem_ld32(to + 32 * k, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st32(to + 32 * k, o);
            }
            tmem_ld32_start(ts + 32 * k, s0);
            tmem_ld32_wait(s0);
            hide(s0, seen[k]);
            weights(s0, c, mc, sum, w + 16 * k);
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
    if (nb > 0) group_sync(9 + t, 288);  // O is complete (and the row's last exchange is read)
    gave_up = gave_up || dead[t] != 0;
    tc_fence_after();
    sm_x[t][hf][row] = l;
    group_sync(pair_bar, 64);
    l += sm_x[t][hf ^ 1][row];
    const bool got = !gave_up && nb > 0;
    if (ta.items == 1) {
      const float f = l > 0.f ? 1.f / l : 0.f;
      uint4* dst = reinterpret_cast<uint4*>(a.out + ((size_t)(row0 + qi) * a.Hq + h * g + head) * kD + 64 * hf);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float o[32];
        if (got) tmem_ld32(to + 32 * k, o);
        if (live)
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (got)
              v = make_uint4(pack_bf16x2(o[e] * f, o[e + 1] * f), pack_bf16x2(o[e + 2] * f, o[e + 3] * f),
                             pack_bf16x2(o[e + 4] * f, o[e + 5] * f), pack_bf16x2(o[e + 6] * f, o[e + 7] * f));
            dst[4 * k + (e >> 3)] = v;
          }
      }
    } else {
      // the record, [row][O | m, l]
      float* rec = reinterpret_cast<float*>(a.workspace + a.plan.off_records) +
                   ((size_t)blockIdx.x * 256 + 128 * t + row) * kRowFloats;
      if (!got) m = -INFINITY;
      if (live && hf == 0) {
        rec[kD] = m;
        rec[kD + 1] = l;
      }
      if (got)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float o[32];
          tmem_ld32(to + 32 * k, o);
          if (live)
#pragma unroll
            for (int e = 0; e < 32; e += 2) *reinterpret_cast<float2*>(rec + 64 * hf + 32 * k + e) = make_float2(o[e], o[e + 1]);
        }
    }
  }
  tc_fence_before();
  if (ta.items > 1) __threadfence();
  __syncthreads();
  if (warp == kTcwMma) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if (ta.items == 1) return;
  // the last item's block joins the records, a warp a row
  const unsigned group = blockIdx.x / ta.items;
  if (threadIdx.x == 0) {
    unsigned* counter = reinterpret_cast<unsigned*>(a.workspace) + group;
    *last = atomicAdd(counter, 1u) == (unsigned)ta.items - 1u;
    if (*last) *counter = 0u;
  }
  __syncthreads();
  if (!*last) return;
  __threadfence();
  const float c = a.sm_scale * kLog2eT;
  const float* recs = reinterpret_cast<const float*>(a.workspace + a.plan.off_records) + (size_t)group * ta.items * 256 * kRowFloats;
  for (int rr = warp; rr < 128 * ntile; rr += kTcwThreads / 32) {
    const int tt = rr >> 7, r = rr & 127, q = i0 + tt * qpt + r / g;
    if (r >= qpt * g || q >= n) continue;
    // lane i holds item i's maximum and sum (items <= 2 SMs: the lanes go round)
    float M = -INFINITY, L = 0.f;
    for (int i = lane; i < ta.items; i += 32) M = fmaxf(M, __ldcg(recs + ((size_t)i * 256 + rr) * kRowFloats + kD));
    M = warp_max(M);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < ta.items; ++i) {
      const float* rec = recs + ((size_t)i * 256 + rr) * kRowFloats;
      const float mi = __ldcg(rec + kD), f = mi == -INFINITY ? 0.f : exp2_t((mi - M) * c);
      L = fmaf(__ldcg(rec + kD + 1), f, L);
      // (an item without keys wrote m and l = 0 alone)
      const float2 u = __ldcg(reinterpret_cast<const float2*>(rec) + 2 * lane);
      const float2 v = __ldcg(reinterpret_cast<const float2*>(rec) + 2 * lane + 1);
      if (f > 0.f) y = make_float4(fmaf(u.x, f, y.x), fmaf(u.y, f, y.y), fmaf(v.x, f, y.z), fmaf(v.y, f, y.w));
    }
    const float f = L > 0.f ? 1.f / L : 0.f;
    reinterpret_cast<uint2*>(a.out + ((size_t)(row0 + q) * a.Hq + h * g + r % g) * kD)[lane] =
        make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
  }
}

}  // namespace

// Blocks per (tile pair, KV head): the fewest waves of blocks times a block's length in key blocks (plus a
// fixed part: the queries, the pipeline's fill and drain, the join), at most two blocks per SM.
WindowPlan plan_window_tc(int64_t batch, int64_t max_tokens, int Hq, int Hkv, int64_t max_keys, int num_sms) {
  WindowPlan p;
  const int qpt = 128 / (Hq / Hkv);
  const int64_t groups = batch * Hkv * ((max_tokens + 2 * qpt - 1) / (2 * qpt));
  const int64_t blocks = (max_keys + 2 * qpt + 127) / 128 + 1;
  constexpr int kFixed = 6;
  const int64_t most = std::min<int64_t>(blocks / 2, kTcSplitBlocks * (int64_t)num_sms / std::max<int64_t>(groups, 1));
  int64_t best = INT64_MAX;
  for (int64_t n = 1; n <= std::max<int64_t>(most, 1); ++n) {
    const int64_t waves = (groups * n + num_sms - 1) / std::max(num_sms, 1);
    const int64_t cost = waves * (kFixed + (blocks + n - 1) / n + (n > 1 ? 3 : 0));
    if (cost < best) {
      best = cost;
      p.items = (int)n;
    }
  }
  p.off_records = ((size_t)kTcSplitBlocks * num_sms * sizeof(unsigned) + 255) & ~(size_t)255;
  p.total = p.off_records + (size_t)kTcSplitBlocks * num_sms * 256 * kRowFloats * sizeof(float);
  return p;
}

cudaError_t launch_window_tc(const WindowLaunch& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done;
  const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(window_tc_kernel), kTcwSmem, done);
  if (e != cudaSuccess) return e;
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t r = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (r != cudaSuccess || q != cudaDriverEntryPointSuccess) return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  // the pools as [num_pages][Hkv 64 rows][128 channels], boxes of 64 channels x one head's page
  CUtensorMap tm[2];
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)a.Hkv * kPage, (cuuint64_t)a.pages.num_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)a.Hkv * kPage * kD * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)kPage, 1}, estride[3] = {1, 1, 1};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = encode(&tm[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(i ? a.v_pages : a.k_pages),
                              dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  TcwArgs ta;
  ta.a = a;
  ta.items = a.plan.items;
  ta.qpt = 128 / (a.Hq / a.Hkv);
  ta.tiles = (a.tok.max_tokens + 2 * ta.qpt - 1) / (2 * ta.qpt);
  const long long blocks = (long long)ta.tiles * a.pages.batch * a.Hkv * ta.items;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  window_tc_kernel<<<(unsigned)blocks, kTcwThreads, kTcwSmem, stream>>>(ta, tm[0], tm[1]);
  return cudaGetLastError();
}

}  // namespace oscar
