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
//   O += P V    P from tensor memory (over half of S's columns), V as it lies in
//       the page: keys along K, channels contiguous (an "MN-major" operand)
// with S, O and the sums in fp32.  Tensor memory: S of both tiles (2 x 128
// columns), O of both (2 x 128).
//
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread is a row (its TMEM lane)
//   warp 8          copies K and V blocks (TMA, 64 channels x 64 rows, 128-byte
//                   swizzle) into a ring of five 32 KB slots, in the order of
//                   use: K_0, V_0, K_1, V_1, ...
//   warp 9          one thread issues the MMAs: S_t(j + 1) right behind
//                   P_t V(j), so that one tile's softmax runs under the other
//                   tile's products
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
constexpr int kTcwThreads = 10 * 32;
constexpr int kTcwSlots = 5;
constexpr uint32_t kTcwQ = 0;                    // queries: [tile][2 x 64 channels][128 rows][128 B]
constexpr uint32_t kTcwRing = 65536;             // slots: [2 x 64 channels][128 keys][128 B]
constexpr uint32_t kTcwBars = kTcwRing + kTcwSlots * 32768;
constexpr size_t kTcwSmem = kTcwBars + 256 + 1024;  // + 1024-byte alignment slack
constexpr uint32_t kTmS = 0, kTmO = 256;         // TMEM columns of S and O, 128 a tile
constexpr float kLazyT = 8.0f;                   // O moves when a row's maximum grew by more than 2^8
constexpr int kRowFloats = kD + 2;               // a row's record: O[128], m, l

struct TcwArgs {
  WindowLaunch a;
  int items, tiles, qpt;  // blocks per (tile pair, KV head), tile pairs per request, queries per tile
};

// Operand with its M or N index contiguous, 128-byte swizzle: rows (K) of 64 elements (128 bytes), groups of
// 8 rows `sbo` bytes apart, the next 64 elements `lbo` bytes on.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
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

// Logits of positions at, at + 1, ... that the row does not see drop out.
__device__ __forceinline__ void hide(float (&s)[32], int at, int lim, int sinks, int low) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!(at + e < lim && (at + e < sinks || at + e >= low))) s[e] = -INFINITY;
}

__device__ __forceinline__ float max32(const float (&s)[32]) {
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int e = 4; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], s[e]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// exp2(c s - mc) of 32 logits: their sum, and 16 pairs of bf16.
__device__ __forceinline__ void weights(const float (&s)[32], float c, float mc, float2& sum, uint32_t* w) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 y = ffma2(make_float2(s[e], s[e + 1]), make_float2(c, c), make_float2(-mc, -mc));
    const float2 p = make_float2(exp2_t(y.x), exp2_t(y.y));
    sum = fadd2(sum, p);
    w[e >> 1] = pack_bf16x2(p.x, p.y);
  }
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
  extern __shared__ uint8_t raw[];
  __shared__ int sm_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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

  const uint32_t raw_s = smem_u32(raw);
  uint8_t* sm = raw + (((raw_s + 1023u) & ~1023u) - raw_s);
  const uint32_t sbase = smem_u32(sm);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kTcwBars);  // [slots] copies landed
  uint64_t* empty = full + kTcwSlots;                           // [slots] read by its products
  uint64_t* sfull = empty + kTcwSlots;                          // [2] S of tile t holds a block's logits (and O its last product)
  uint64_t* pready = sfull + 2;                                 // [2] P of tile t written
  uint64_t* odone = pready + 2;                                 // [2] O of tile t complete
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(odone + 2);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcwSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[t], 4);
      mbar_init(&odone[t], 1);
    }
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(tmem_at, 512);
  if (warp == 8 && lane == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  const int t = warp >> 2, row = 32 * (warp & 3) + lane;  // softmax warps: tile and row
  const int qi = i0 + t * qpt + row / g, head = row % g;
  const bool live = warp < 8 && row < qpt * g && qi < n;
  if (warp < 8 && t < ntile) {  // the queries, into the swizzled operand layout
    const uint4* src = reinterpret_cast<const uint4*>(a.q + (size_t)(row0 + qi) * a.q_stride + (size_t)(h * g + head) * kD);
    uint8_t* dst = sm + kTcwQ + t * 32768 + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const uint4 v = live ? src[c] : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  const bool any_bad = __syncthreads_or(bad);
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(tmem_at);
  bool gave_up = false;

  float m = -INFINITY, l = 0.f;
  if (warp == 8) {
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
  } else if (warp == 9) {
    // ---- products, issued by one thread
    if (lane == 0 && nb > 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, 128);
      constexpr uint32_t idesc_o = umma_idesc_bf16_f32(128, 128) | (1u << 16);  // B: channels contiguous
      auto logits = [&](int tt, int slot) {
        const uint32_t q = sbase + kTcwQ + tt * 32768, k = sbase + kTcwRing + slot * 32768;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const uint32_t off = (s >> 2) * 16384 + (s & 3) * 32;
          umma_f16(tbase + kTmS + tt * 128, umma_desc_sw128(q + off), umma_desc_sw128(k + off), idesc_s, s > 0);
        }
        umma_commit(&sfull[tt]);
      };
      bool ok = mbar_wait_timed(&full[0], 0, kWaitNs);
      if (ok) {
        tc_fence_after();
        for (int tt = 0; tt < ntile; ++tt) logits(tt, 0);
        umma_commit(&empty[0]);
      }
      for (int j = 0; j < nb && ok; ++j) {
        const int uv = 2 * j + 1, uk = 2 * j + 2, sv = uv % kTcwSlots, sk = uk % kTcwSlots;
        ok = mbar_wait_timed(&full[sv], (uv / kTcwSlots) & 1, kWaitNs);
        for (int tt = 0; tt < ntile && ok; ++tt) {
          ok = mbar_wait_timed(&pready[tt], j & 1, kWaitNs);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v = sbase + kTcwRing + sv * 32768;
#pragma unroll
          for (int s = 0; s < 8; ++s)
            umma_f16_ts(tbase + kTmO + tt * 128, tbase + kTmS + tt * 128 + 64 + 8 * s, umma_desc_mn_sw128(v + 2048 * s, 16384, 1024),
                        idesc_o, j > 0 || s > 0);
          if (j + 1 < nb) {
            if (tt == 0) ok = mbar_wait_timed(&full[sk], (uk / kTcwSlots) & 1, kWaitNs);
            if (ok) {
              tc_fence_after();
              logits(tt, sk);
            }
          } else {
            umma_commit(&odone[tt]);
          }
        }
        if (ok) {
          umma_commit(&empty[sv]);
          if (j + 1 < nb) umma_commit(&empty[sk]);
        }
      }
      if (!ok) set_error(a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (t < ntile) {
    // ---- softmax: this thread's row
    const uint32_t ts = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + kTmS + t * 128;
    const uint32_t to = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + kTmO + t * 128;
    const float c = a.sm_scale * kLog2eT;
    const int tf = first + t * qpt, tl = min(tf + qpt - 1, (int)plast);  // the tile's positions
    const int p = min(p0 + qi, (int)plast);
    const int lim = min(p + 1, ctx), low = a.window < 0 ? 0 : max(0, p - a.window + 1);
    for (int j = 0; j < nb; ++j) {
      // the block's pages: whether every row of the tile sees all of them, and whether some row of theirs is
      // seen by no query of the block (such a V row may hold anything: it becomes zeros)
      int base[2];
      bool whole = true, clean = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int kk = 2 * (j0 + j) + k;
        const int lp = kk < np ? pl.page(kk) : -1;
        base[k] = lp < 0 || (any_bad && page_of(a.pages, b, lp, a.err, false) < 0) ? INT32_MAX - 63 : lp * kPage;
        const int end = base[k] + 63;
        whole = whole && end < min(tf + 1, ctx) && (end < sinks || a.window < 0 || base[k] > tl - a.window);
        clean = clean && end < hi && (end < sinks || base[k] >= lo);
      }
      if (t == 0 && !clean) {
        const int uv = 2 * j + 1, sv = uv % kTcwSlots;
        if (!__all_sync(0xffffffffu, mbar_wait_timed(&full[sv], (uv / kTcwSlots) & 1, kWaitNs))) {
          gave_up = true;
          break;
        }
        const int at = (row < 64 ? base[0] : base[1]) + (row & 63);
        if (!(at < hi && (at < sinks || at >= lo))) {
          uint8_t* v = sm + kTcwRing + sv * 32768 + row * 128;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            *reinterpret_cast<uint4*>(v + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(v + 16384 + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
      }
      if (!__all_sync(0xffffffffu, mbar_wait_timed(&sfull[t], j & 1, kWaitNs))) {
        gave_up = true;
        break;
      }
      tc_fence_after();
      // the first 64 keys are read twice (once for the maximum), the others stay in registers; P goes over the
      // others' columns
      float s0[32], s1[32], s2[32], s3[32];
      tmem_ld32x2(ts, ts + 32, s0, s1);
      if (!whole) {
        hide(s0, base[0], lim, sinks, low);
        hide(s1, base[0] + 32, lim, sinks, low);
      }
      const float ma = fmaxf(max32(s0), max32(s1));
      tmem_ld32x2(ts + 64, ts + 96, s2, s3);
      if (!whole) {
        hide(s2, base[1], lim, sinks, low);
        hide(s3, base[1] + 32, lim, sinks, low);
      }
      const float mb = fmaxf(ma, fmaxf(max32(s2), max32(s3)));
      // m, in units of S; O and l move when it grew by more than 2^8 in the exponent
      const bool grow = (mb - m) * c > kLazyT || (m == -INFINITY && mb > -INFINITY);
      if (__any_sync(0xffffffffu, grow)) {
        float f = 1.f;
        if (grow) {
          f = m == -INFINITY ? 0.f : exp2_t((m - mb) * c);
          m = mb;
          l *= f;
        }
        if (j > 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float o[32];
            tmem_ld32(to + 32 * k, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(to + 32 * k, o);
          }
        }
      }
      const float mc = m == -INFINITY ? 0.f : m * c;
      float2 sum = make_float2(0.f, 0.f);
      uint32_t w[32];
      weights(s2, c, mc, sum, w);
      weights(s3, c, mc, sum, w + 16);
      tmem_st32u(ts + 96, w);
      tmem_ld32x2(ts, ts + 32, s0, s1);
      if (!whole) {
        hide(s0, base[0], lim, sinks, low);
        hide(s1, base[0] + 32, lim, sinks, low);
      }
      weights(s0, c, mc, sum, w);
      weights(s1, c, mc, sum, w + 16);
      tmem_st32u(ts + 64, w);
      l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pready[t]);
    }
    if (gave_up && lane == 0) set_error(a.err, kErrTimeout);
    if (!gave_up && nb > 0) {
      if (!__all_sync(0xffffffffu, mbar_wait_timed(&odone[t], 0, kWaitNs))) {
        gave_up = true;
        if (lane == 0) set_error(a.err, kErrTimeout);
      }
      tc_fence_after();
    }
    const bool got = !gave_up && nb > 0;
    if (ta.items == 1) {
      const float f = l > 0.f ? 1.f / l : 0.f;
      uint4* dst = reinterpret_cast<uint4*>(a.out + ((size_t)(row0 + qi) * a.Hq + h * g + head) * kD);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
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
      if (live) {
        rec[kD] = m;
        rec[kD + 1] = l;
      }
      if (got)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float o[32];
          tmem_ld32(to + 32 * k, o);
          if (live)
#pragma unroll
            for (int e = 0; e < 32; e += 2) *reinterpret_cast<float2*>(rec + 32 * k + e) = make_float2(o[e], o[e + 1]);
        }
    }
  }
  tc_fence_before();
  if (ta.items > 1) __threadfence();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if (ta.items == 1) return;
  // the last item's block joins the records, a warp a row
  const unsigned group = blockIdx.x / ta.items;
  if (threadIdx.x == 0) {
    unsigned* counter = reinterpret_cast<unsigned*>(a.workspace) + group;
    sm_last = atomicAdd(counter, 1u) == (unsigned)ta.items - 1u;
    if (sm_last) *counter = 0u;
  }
  __syncthreads();
  if (!sm_last) return;
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
