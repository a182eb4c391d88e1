// Attention with a sliding window and visible first tokens, split over the
// keys: the form for single tokens (and short chunks), over BF16 pages or the
// 4-bit cache.
//
// One (query, KV head) sees a list of 16-token tiles: those of the sinks, then
// those of the window.  The list is cut into work items, one block each; the
// warps of a block take units of it (one tile of BF16 rows, two tiles of the
// 4-bit cache) in turn, each with a ring of units copied ahead by cp.async and
// an online softmax of its own (running maximum m, sum l, accumulator o, all
// fp32, base-2 exponents).  The block joins its warps' states; when there are
// several items, the last block to finish joins their records in item order,
// so the result does not depend on which one that is.
//
// Products run on m16n8k16 MMAs with the cached side as the 16 rows (tokens in
// Q K, channels in P V) and the g query heads of a KV head as the 8 columns.
// With g <= 4 (PACK) head h has columns 2 h and 2 h + 1, the value and the
// residual of its operand split into two bf16 terms (2^-17 relative), at no
// cost; with g > 4 the columns are heads.

#include "oscar_paged.cuh"

#include <algorithm>
#include <cmath>

namespace oscar {
namespace {

constexpr float kLog2eW = 1.4426950408889634f;
constexpr float kLazyW = 8.0f;  // the accumulators are rescaled when the maximum grows by more than 2^8

template <bool INT4>
struct Ring {
  static constexpr int kWarps = INT4 ? 16 : 8;
  static constexpr int kTiles = INT4 ? 2 : 1;                        // 16-token tiles of a unit
  static constexpr int kUnit = INT4 ? 2 * kTile4Bytes : 16 * kD * 4;  // bytes of a unit
  static constexpr int kStages = 3;
  static constexpr int kBytes = kWarps * kStages * kUnit;
};
constexpr int kSplitBlocks = 4;  // blocks per SM that one call may split its keys over

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

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(p)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_at(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(p)
               : "memory");
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

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What one query sees: tiles [0, s_end) and [w_begin, w_end), and inside them
// the positions j < len with j < sinks or j >= low.
struct Seen {
  int len, low, sinks, s_end, w_begin, w_end;
  __device__ __forceinline__ int tiles() const { return s_end + max(0, w_end - w_begin); }
  __device__ __forceinline__ int tile(int t) const { return t < s_end ? t : w_begin + (t - s_end); }
  __device__ __forceinline__ bool sees(int j) const { return j < len && (j < sinks || j >= low); }
};

// The request of token row i.
__device__ __forceinline__ int request_of(const TokenRefs& t, int batch, int i) {
  if (t.cu == nullptr) return i;
  int lo = 0, hi = batch;  // the last b with cu[b] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.cu[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// KU: tiles of a unit.  Sets `seen` for token row i; false when the row is no request's.
template <int KU>
__device__ __forceinline__ bool seen_by(const WindowLaunch& a, int i, int& b, Seen& s, bool report) {
  b = request_of(a.tok, a.pages.batch, i);
  int p0, n, row0;
  if (!token_span(a.tok, b, p0, n, row0, a.err, report) || i < row0 || i >= row0 + n) return false;
  const long long p = (long long)p0 + (i - row0);
  long long len = min(p + 1, (long long)max(a.ctx_len[b], 0));
  if (p0 < 0) {
    if (report) set_error(a.err, kErrLength);
    len = 0;
  }
  const long long limit = (long long)a.pages.max_pages * kPage;
  if (len > limit) {
    if (report) set_error(a.err, kErrLength);
    len = limit;
  }
  s.len = (int)len;
  s.low = a.window < 0 ? 0 : (int)min(max(p + 1 - a.window, 0ll), (long long)INT32_MAX);
  s.sinks = min(a.sinks, s.len);
  // in units of KU tiles, so that a unit never straddles two pages
  constexpr int kTok = 16 * KU;
  s.s_end = s.low > 0 ? (s.sinks + kTok - 1) / kTok * KU : 0;
  s.w_end = (s.len + kTok - 1) / kTok * KU;
  s.s_end = min(s.s_end, s.w_end);
  s.w_begin = s.low >= s.len ? s.w_end : max(s.low / kTok * KU, s.s_end);  // none of the window is held: no tiles
  return true;
}

struct WindowArgs {
  WindowLaunch a;
  int items;
};

// Copy unit `t0` (tile index in the list) of the query's keys into a stage.  BF16: rows of 256 bytes,
// 16-byte piece c of row u at c ^ (u % 8); rows that the query does not see become zeros (a V row of
// theirs may hold anything, and 0 x NaN is not 0).  4-bit: the tiles as they are.
template <bool INT4>
__device__ __forceinline__ void copy_unit(const WindowLaunch& a, const Seen& s, int T, int phys, int h, uint32_t stage,
                                          int lane) {
  if constexpr (INT4) {
    const uint8_t* src =
        a.pages4 + ((size_t)max(phys, 0) * a.Hkv + h) * kBlock4Bytes + (size_t)(T & 3) * kTile4Bytes + 16 * lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) cp_async16(stage + 16 * lane + 512 * i, src + 512 * i, phys >= 0);
    cp_async8(stage + 8 * lane + 4096, src - 8 * lane + 4096, phys >= 0);
  } else {
    const size_t off = ((size_t)max(phys, 0) * a.Hkv + h) * (kPage * kD) + (size_t)(T & 3) * 16 * kD;
    const uint4* k = reinterpret_cast<const uint4*>(a.k_pages + off);
    const uint4* v = reinterpret_cast<const uint4*>(a.v_pages + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = 2 * i + (lane >> 4), c = lane & 15;
      const uint32_t dst = stage + 256 * u + 16 * (c ^ (u & 7));
      const bool real = phys >= 0 && s.sees(16 * T + u);
      cp_async16(dst, k + 16 * u + c, real);
      cp_async16(dst + 4096, v + 16 * u + c, real);
    }
  }
}

// A warp's running state.  PACK: this lane's head is tq; else heads 2 tq and 2 tq + 1.
template <bool PACK, bool INT4>
struct State {
  static constexpr int kH = PACK ? 1 : 2;
  float m[kH], l[kH];
  float wsum[kH][2];  // 4-bit: sums of the weights of each group (what the codes' offset is multiplied by)
  float o[8][4];
};

// 4-bit words to bf16 pairs, from the bits alone.  K: 128 + c.  V: 16 + c: a smaller offset, because P V
// cancels it against the sum of the weights and the MMA's fp32 sums truncate relative to it (the logits'
// offset is cancelled inside one tile's product).  The exponent bits come in a register, so that masking
// and setting them is one LOP3 (as two constants they were two: 64 of 370 instructions a tile).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}
__device__ __forceinline__ uint32_t k_pair(uint32_t w, int i, uint32_t bits) {
  return and_or(i == 0 ? w : w >> (4 * i), 0x000F000Fu, bits);
}
__device__ __forceinline__ uint32_t v_pair(uint32_t w, int i, uint32_t bits) {
  return and_or(i == 0 ? w << 3 : w >> (4 * i - 3), 0x00780078u, bits);
}
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  uint32_t y;
  asm volatile("mov.b32 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
constexpr float kKOffset = 128.f + 7.5f, kVOffset = 16.f + 7.5f;

// value + residual of x as a bf16 pair (value in the low half)
__device__ __forceinline__ uint32_t split_bf16(float x) {
  const float v = bf16_lo(pack_bf16x2(x, 0.f));
  return pack_bf16x2(v, x - v);
}

template <bool PACK, bool INT4>
__device__ __forceinline__ void window_body(const WindowArgs& wa) {
  using R = Ring<INT4>;
  constexpr int kW = R::kWarps, kS = R::kStages, KU = R::kTiles, kH = PACK ? 1 : 2;
  const WindowLaunch& a = wa.a;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(16) float sm_q[kMaxG * kD];
  __shared__ float sm_ml[2][kW][kMaxG];
  __shared__ float sm_m[kMaxG], sm_l[kMaxG];
  __shared__ int sm_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, tq = lane & 3;
  const int items = wa.items, row = blockIdx.x / items, item = blockIdx.x % items, h = blockIdx.y;
  const int g = a.Hq / a.Hkv;
  int b;
  Seen s;
  if (!seen_by<KU>(a, row, b, s, threadIdx.x == 0 && item == 0 && h == 0)) return;
  // this item's units [u0, u1), this warp's: u0 + warp, + kW, ...
  const int units = s.tiles() / KU;
  const int u0 = (int)((long long)units * item / items), u1 = (int)((long long)units * (item + 1) / items);
  const uint32_t ring = smem_u32(sm) + warp * (kS * R::kUnit);
  int phys_l = -1, fetched = 0;  // lane i: the page of the warp's unit fetched - 32 + i
  auto issue = [&](int i) {      // the warp's i-th unit
    if (i >= fetched) {
      const int u = u0 + warp + (fetched + lane) * kW;
      phys_l = -1;
      if (u < u1) phys_l = page_of(a.pages, b, s.tile(u * KU) >> 2, a.err, true);
      fetched += 32;
    }
    const int phys = __shfl_sync(0xffffffffu, phys_l, i & 31);
    const int u = u0 + warp + i * kW;
    if (u < u1) copy_unit<INT4>(a, s, s.tile(u * KU), phys, h, ring + (i % kS) * R::kUnit, lane);
    cp_async_commit();
    return phys;
  };
  int phys_q[kS];
#pragma unroll
  for (int i = 0; i < kS - 1; ++i) phys_q[i] = issue(i);

  // the queries as MMA columns: qf[k step][2], and the offset's part of the logits
  uint32_t qf[8][2], qr[8][2];
  float q0[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // [group][column of the lane's two]
  const uint16_t* qrow = a.q + (size_t)row * a.q_stride + (size_t)h * g * kD;
  if constexpr (INT4) {
    for (int hh = warp; hh < kMaxG; hh += kW) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (hh < g) {
        const uint2 u = *reinterpret_cast<const uint2*>(qrow + hh * kD + 4 * lane);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        hadamard128(v, lane);
      }
      const float f = kInvSqrt128 * a.sm_scale * kLog2eW;
#pragma unroll
      for (int e = 0; e < 4; ++e) sm_q[hh * kD + 4 * lane + e] = v[e] * f;
    }
    __syncthreads();
    // k step 2 M + b2: k bits e, tq, kh = channel bits 0, (3, 4), 1; bits 2, 5, 6 = b2, M
    const int hh = PACK ? r >> 1 : r;
    const bool live = hh < g;
    float part[2] = {0.f, 0.f}, partr[2] = {0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        const int j = 32 * (ks >> 1) + 8 * tq + 4 * (ks & 1) + 2 * kh;
        const float x0 = live ? sm_q[hh * kD + j] : 0.f, x1 = live ? sm_q[hh * kD + j + 1] : 0.f;
        const uint32_t v = pack_bf16x2(x0, x1);
        const uint32_t res = pack_bf16x2(x0 - bf16_lo(v), x1 - bf16_hi(v));
        qf[ks][kh] = PACK && (r & 1) ? res : v;
        qr[ks][kh] = res;
        part[ks >> 2] += bf16_lo(qf[ks][kh]) + bf16_hi(qf[ks][kh]);
        partr[ks >> 2] += bf16_lo(res) + bf16_hi(res);
      }
    // sums over the column's four lanes, then to the lanes that hold columns 2 tq, 2 tq + 1 of the logits
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      float x = PACK ? part[gr] : part[gr] + partr[gr];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      q0[gr][0] = -kKOffset * __shfl_sync(0xffffffffu, x, 4 * (2 * tq));
      q0[gr][1] = -kKOffset * __shfl_sync(0xffffffffu, x, 4 * (2 * tq + 1));
    }
  } else {
    const int hh = PACK ? r >> 1 : r;
    const bool live = hh < g && !(PACK && (r & 1));  // a bf16 query has no residual
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qf[ks][0] = live ? *reinterpret_cast<const uint32_t*>(qrow + hh * kD + 16 * ks + 2 * tq) : 0u;
      qf[ks][1] = live ? *reinterpret_cast<const uint32_t*>(qrow + hh * kD + 16 * ks + 8 + 2 * tq) : 0u;
    }
  }
  const float qscale = INT4 ? 1.f : a.sm_scale * kLog2eW;

  State<PACK, INT4> st;
#pragma unroll
  for (int i = 0; i < kH; ++i) {
    st.m[i] = -INFINITY;
    st.l[i] = 0.f;
    st.wsum[i][0] = st.wsum[i][1] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) st.o[i][e] = 0.f;

  const uint32_t kbits = opaque(0x43004300u), vbits = opaque(0x41804180u);
  // units of which the query sees all: [in0, in1) of the window
  const int in0 = (s.low + 15) >> 4, in1 = s.len >> 4;
  const int mine = u1 - u0 - warp > 0 ? (u1 - u0 - warp + kW - 1) / kW : 0;
  for (int i = 0; i < mine; ++i) {
    __syncwarp();
    phys_q[kS - 1] = issue(i + kS - 1);
    cp_async_wait<kS - 1>();
    __syncwarp();
    const uint32_t stage = ring + (i % kS) * R::kUnit;
    const int T = s.tile((u0 + warp + i * kW) * KU);
    const bool bad = phys_q[0] < 0;
#pragma unroll
    for (int j = 0; j < kS - 1; ++j) phys_q[j] = phys_q[j + 1];
    // logits x[tile][row half][head], base 2
    float x[KU][2][kH];
#pragma unroll
    for (int k = 0; k < KU; ++k) {
      if constexpr (INT4) {
        const uint32_t tb = stage + k * kTile4Bytes;
        const uint4 w0 = lds128(tb + 16 * lane), w1 = lds128(tb + 512 + 16 * lane);
        float acc[2][4];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t wa0 = word_of(w0, ks >> 1), wa1 = word_of(w1, ks >> 1);
          const uint32_t a0 = k_pair(wa0, 2 * (ks & 1), kbits), a1 = k_pair(wa1, 2 * (ks & 1), kbits);
          const uint32_t a2 = k_pair(wa0, 2 * (ks & 1) + 1, kbits), a3 = k_pair(wa1, 2 * (ks & 1) + 1, kbits);
          if ((ks & 3) == 0) {  // the group's sum starts from the offset's part
            const uint32_t af[4] = {a0, a1, a2, a3};
            const float c0[4] = {q0[ks >> 2][0], q0[ks >> 2][1], q0[ks >> 2][0], q0[ks >> 2][1]};
            mma_bf16(acc[ks >> 2], af, qf[ks][0], qf[ks][1], c0);
          } else {
            mma_bf16_acc(acc[ks >> 2], a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
          }
          if constexpr (!PACK) mma_bf16_acc(acc[ks >> 2], a0, a1, a2, a3, qr[ks][0], qr[ks][1]);
        }
#pragma unroll
        for (int rh = 0; rh < 2; ++rh) {
          const uint32_t u = lds32(tb + kTile4Scales + 4 * (r + 8 * rh));
          const float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&u));
          if constexpr (PACK) {
            x[k][rh][0] = (acc[0][2 * rh] + acc[0][2 * rh + 1]) * sc.x + (acc[1][2 * rh] + acc[1][2 * rh + 1]) * sc.y;
          } else {
            x[k][rh][0] = acc[0][2 * rh] * sc.x + acc[1][2 * rh] * sc.y;
            x[k][rh][kH - 1] = acc[0][2 * rh + 1] * sc.x + acc[1][2 * rh + 1] * sc.y;
          }
        }
      } else {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        const int mr = (lane & 7) + 8 * ((lane >> 3) & 1);  // ldmatrix: lane's row, and the 16-byte piece below
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t a0, a1, a2, a3;
          ldmatrix_x4_at(a0, a1, a2, a3, stage + 256 * mr + 16 * ((2 * ks + (lane >> 4)) ^ (mr & 7)));
          mma_bf16_acc(acc, a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
        }
#pragma unroll
        for (int rh = 0; rh < 2; ++rh) {
          x[k][rh][0] = acc[2 * rh] * qscale;
          if constexpr (!PACK) x[k][rh][kH - 1] = acc[2 * rh + 1] * qscale;
        }
      }
    }
    // positions that the query does not see (or whose page is bad) drop out by selection
    uint32_t hid = 0;  // bit 2 k + rh: token r + 8 rh of tile k
    if (bad || !((T >= in0 || 16 * (T + KU) <= s.sinks) && T + KU <= in1)) {
#pragma unroll
      for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int rh = 0; rh < 2; ++rh)
          if (bad || !s.sees(16 * (T + k) + r + 8 * rh)) hid |= 1u << (2 * k + rh);
#pragma unroll
      for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int rh = 0; rh < 2; ++rh)
#pragma unroll
          for (int e = 0; e < kH; ++e)
            if ((hid >> (2 * k + rh)) & 1u) x[k][rh][e] = -INFINITY;
    }
    // running maximum; the accumulators move only when it grew a lot
    float sub[kH];
#pragma unroll
    for (int e = 0; e < kH; ++e) {
      float m = x[0][0][e];
#pragma unroll
      for (int k = 0; k < KU; ++k)
#pragma unroll
        for (int rh = 0; rh < 2; ++rh) m = fmaxf(m, x[k][rh][e]);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      sub[e] = m;
    }
    bool grow = false;
#pragma unroll
    for (int e = 0; e < kH; ++e) grow = grow || sub[e] > st.m[e] + kLazyW || (st.m[e] == -INFINITY && sub[e] > -INFINITY);
    if (__any_sync(0xffffffffu, grow)) {
      float f[kH];
#pragma unroll
      for (int e = 0; e < kH; ++e) {
        const float m = fmaxf(st.m[e], sub[e]);
        f[e] = st.m[e] == -INFINITY ? 0.f : exp2_fast(st.m[e] - m);
        st.m[e] = m;
        st.l[e] *= f[e];
        st.wsum[e][0] *= f[e];
        st.wsum[e][1] *= f[e];
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[mt][e] *= PACK ? f[0] : f[(e & 1) * (kH - 1)];
    }
#pragma unroll
    for (int e = 0; e < kH; ++e) sub[e] = st.m[e] == -INFINITY ? 0.f : st.m[e];
#pragma unroll
    for (int k = 0; k < KU; ++k) {
      // weights, as the MMA's columns: transposed 8 x 8 blocks (tokens 0-7 and 8-15)
      uint32_t bv[INT4 ? 2 : 1][2];
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        float p[kH];
#pragma unroll
        for (int e = 0; e < kH; ++e) {
          p[e] = exp2_fast(x[k][rh][e] - sub[e]);
          st.l[e] += p[e];
        }
        if constexpr (INT4) {
          const uint32_t u = lds32(stage + k * kTile4Bytes + kTile4Scales + 64 + 4 * (r + 8 * rh));
          float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&u));
          if ((hid >> (2 * k + rh)) & 1u) sc = make_float2(0.f, 0.f);  // a row nobody wrote may hold any scale
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            const float sg = gr ? sc.y : sc.x;
            if constexpr (PACK) {
              const float w = p[0] * sg;
              st.wsum[0][gr] += w;
              bv[gr][rh] = movmatrix_trans(split_bf16(w));
            } else {
              // one bf16 term per weight (2^-9): the offset is taken off with the rounded weights
              const uint32_t w = pack_bf16x2(p[0] * sg, p[kH - 1] * sg);
              st.wsum[0][gr] += bf16_lo(w);
              st.wsum[kH - 1][gr] += bf16_hi(w);
              bv[gr][rh] = movmatrix_trans(w);
            }
          }
        } else {
          bv[0][rh] = movmatrix_trans(PACK ? split_bf16(p[0]) : pack_bf16x2(p[0], p[kH - 1]));
        }
      }
      if constexpr (INT4) {
        const uint32_t vb = stage + k * kTile4Bytes + kTile4V + 16 * lane;
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          const uint4 w = lds128(vb + 512 * gr);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t wq = word_of(w, q);
            mma_bf16_acc(st.o[4 * gr + q], v_pair(wq, 0, vbits), v_pair(wq, 1, vbits), v_pair(wq, 2, vbits),
                         v_pair(wq, 3, vbits), bv[gr][0], bv[gr][1]);
          }
        }
      } else {
        const int mr = (lane & 7) + 8 * (lane >> 4);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          uint32_t a0, a1, a2, a3;
          ldmatrix_x4_trans(a0, a1, a2, a3, stage + 4096 + 256 * mr + 16 * ((2 * mt + ((lane >> 3) & 1)) ^ (mr & 7)));
          mma_bf16_acc(st.o[mt], a0, a1, a2, a3, bv[0][0], bv[0][1]);
        }
      }
    }
  }
  cp_async_wait<0>();
  // sums over the lanes of a column
#pragma unroll
  for (int e = 0; e < kH; ++e)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], o);
      if constexpr (INT4) {
        st.wsum[e][0] += __shfl_xor_sync(0xffffffffu, st.wsum[e][0], o);
        st.wsum[e][1] += __shfl_xor_sync(0xffffffffu, st.wsum[e][1], o);
      }
    }
  __syncthreads();  // every warp is done with the ring: it becomes the warps' accumulators [warp][head][128]
  float* so = reinterpret_cast<float*>(sm);
  if (r == 0)
#pragma unroll
    for (int e = 0; e < kH; ++e) {
      const int hh = PACK ? tq : 2 * tq + e;
      sm_ml[0][warp][hh] = st.m[e];
      sm_ml[1][warp][hh] = st.l[e];
    }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      // 4-bit: the MMA row (c, half) of word m is channel bits (0, 1, 3) = c, 4 = half, (2, 5, 6) = m
      const int ch = INT4 ? (r & 3) | ((mt & 1) << 2) | ((r >> 2) << 3) | (hf << 4) | ((mt >> 1) << 5)
                          : 16 * mt + 8 * hf + r;
      if constexpr (PACK) {
        float y = st.o[mt][2 * hf] + st.o[mt][2 * hf + 1];
        if constexpr (INT4) y = fmaf(-kVOffset, st.wsum[0][mt >> 2], y);
        if (tq < g) so[(warp * g + tq) * kD + ch] = y;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = st.o[mt][2 * hf + e];
          if constexpr (INT4) y = fmaf(-kVOffset, st.wsum[e * (kH - 1)][mt >> 2], y);
          if (2 * tq + e < g) so[(warp * g + 2 * tq + e) * kD + ch] = y;
        }
      }
    }
  __syncthreads();
  // join the warps
  if (warp == 0 && lane < g) {
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) M = fmaxf(M, sm_ml[0][w][lane]);
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const float m = sm_ml[0][w][lane], f = m == -INFINITY ? 0.f : exp2_fast(m - M);
      L = fmaf(sm_ml[1][w][lane], f, L);
      sm_ml[0][w][lane] = f;
    }
    sm_m[lane] = M;
    sm_l[lane] = L;
  }
  __syncthreads();
  const int rec = g * (kD + 2);  // floats of a record: o[g][128], m[g], l[g]
  unsigned* counter = reinterpret_cast<unsigned*>(a.workspace) + (size_t)row * a.Hkv + h;
  float* records = reinterpret_cast<float*>(a.workspace + a.plan.off_records) + ((size_t)row * a.Hkv + h) * items * rec;
  for (int i = threadIdx.x; i < g * kD; i += 32 * kW) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) y = fmaf(so[w * g * kD + i], sm_ml[0][w][i >> 7], y);
    if (items > 1)
      records[(size_t)item * rec + i] = y;
    else
      sm_q[i] = y;
  }
  if (items > 1) {
    if (threadIdx.x < g) {
      records[(size_t)item * rec + g * kD + threadIdx.x] = sm_m[threadIdx.x];
      records[(size_t)item * rec + g * kD + g + threadIdx.x] = sm_l[threadIdx.x];
    }
    // the last block of the (query, KV head) joins the items' records, in item order
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      const unsigned t = atomicAdd(counter, 1u);
      sm_last = t == (unsigned)items - 1u;
      if (sm_last) *counter = 0u;
    }
    __syncthreads();
    if (!sm_last) return;
    __threadfence();
    // a warp a head: maximum, sum and the items' factors (over the ring: every record is in the workspace)
    float* fac = so;  // [head][items]
    for (int hh = warp; hh < g; hh += kW) {
      float M = -INFINITY, L = 0.f;
      for (int i = lane; i < items; i += 32) M = fmaxf(M, __ldcg(records + (size_t)i * rec + g * kD + hh));
      M = warp_max(M);
      for (int i = lane; i < items; i += 32) {
        const float m = __ldcg(records + (size_t)i * rec + g * kD + hh), f = m == -INFINITY ? 0.f : exp2_fast(m - M);
        L = fmaf(__ldcg(records + (size_t)i * rec + g * kD + g + hh), f, L);
        fac[hh * items + i] = f;
      }
      L = warp_sum(L);
      if (lane == 0) sm_l[hh] = L;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g * kD; i += 32 * kW) {
      const float* f = fac + (i >> 7) * items;
      float y = 0.f;
#pragma unroll 8
      for (int k = 0; k < items; ++k) y = fmaf(__ldcg(records + (size_t)k * rec + i), f[k], y);
      sm_q[i] = y;
    }
  }
  __syncthreads();
  // normalise, turn back, round once
  for (int hh = warp; hh < g; hh += kW) {
    const float f = sm_l[hh] > 0.f ? 1.f / sm_l[hh] : 0.f;
    const float4 y = reinterpret_cast<const float4*>(sm_q + hh * kD)[lane];
    float v[4] = {y.x * f, y.y * f, y.z * f, y.w * f};
    if constexpr (INT4) {
      hadamard128(v, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= kInvSqrt128;
    }
    reinterpret_cast<uint2*>(a.out + ((size_t)row * a.Hq + h * g + hh) * kD)[lane] =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

template <bool PACK, bool INT4>
__global__ void __launch_bounds__(32 * Ring<INT4>::kWarps, 1) window_split_kernel(const __grid_constant__ WindowArgs wa) {
  window_body<PACK, INT4>(wa);
}

template <bool PACK, bool INT4>
cudaError_t launch_one(const WindowLaunch& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done;
  const void* fn = reinterpret_cast<const void*>(window_split_kernel<PACK, INT4>);
  constexpr size_t smem = Ring<INT4>::kBytes;
  static_assert(Ring<INT4>::kWarps * kMaxG * kD * 4 <= Ring<INT4>::kBytes, "the warps' accumulators in the ring");
  const cudaError_t e = smem_attr_once(fn, smem, done);
  if (e != cudaSuccess) return e;
  WindowArgs wa;
  wa.a = a;
  wa.items = a.plan.items;
  window_split_kernel<PACK, INT4>
      <<<dim3((unsigned)(a.tok.n_tokens * (long long)wa.items), a.Hkv), 32 * Ring<INT4>::kWarps, smem, stream>>>(wa);
  return cudaGetLastError();
}

}  // namespace

// Items per (query, KV head): the fewest waves of blocks (one per SM) times a block's length, which is a
// fixed part (the queries, the first copies, the join: about kFixed units of a warp's time) and the units
// per warp.  At most four blocks per SM are split off, so the workspace has one size for every call.
WindowPlan plan_window(bool int4, int64_t rows, int Hq, int Hkv, int64_t max_keys, int num_sms) {
  WindowPlan p;
  const int warps = int4 ? Ring<true>::kWarps : Ring<false>::kWarps;
  const int tok = 16 * (int4 ? Ring<true>::kTiles : Ring<false>::kTiles);
  const int64_t units = (max_keys + 2 * tok - 2) / tok + 1, pairs = std::max<int64_t>(rows * Hkv, 1);
  constexpr int kFixed = 10;
  const int64_t most = std::min<int64_t>((units + warps - 1) / warps, kSplitBlocks * (int64_t)num_sms / pairs);
  int64_t best = INT64_MAX;
  for (int64_t n = 1; n <= std::max<int64_t>(most, 1); ++n) {
    const int64_t waves = (pairs * n + num_sms - 1) / std::max(num_sms, 1);
    const int64_t cost = waves * (kFixed + (units + n * warps - 1) / (n * warps) + (n > 1 ? 2 : 0));
    if (cost < best) {
      best = cost;
      p.items = (int)n;
    }
  }
  p.off_records = ((size_t)kSplitBlocks * num_sms * sizeof(unsigned) + 255) & ~(size_t)255;
  p.total = p.off_records + (size_t)kSplitBlocks * num_sms * (Hq / Hkv) * (kD + 2) * sizeof(float);
  return p;
}

cudaError_t launch_window_split(const WindowLaunch& a, cudaStream_t stream) {
  const bool pack = a.Hq / a.Hkv <= 4;
  if (a.pages4 != nullptr) return pack ? launch_one<true, true>(a, stream) : launch_one<false, true>(a, stream);
  return pack ? launch_one<true, false>(a, stream) : launch_one<false, false>(a, stream);
}

}  // namespace oscar
