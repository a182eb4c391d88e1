// Attention with a sliding window and visible first tokens, split over the
// keys: single tokens over BF16 pages, and all calls over the 4-bit cache.
//
// One (query, KV head) sees a list of 16-token tiles: those of the sinks, then
// those of the window, in units of one tile (BF16) or two (4 bits).  The units
// of all (query, KV head) pairs, one pair after another, are cut into one equal
// range for each block (every block adds up the rows' lengths for itself), so
// that ragged lengths leave no SM idle; a range holds one or more segments of
// pairs.  The warps of a block take a segment's units in turn, each with a ring
// of units copied ahead by cp.async and an online softmax of its own (running
// maximum m, sum l, accumulator o, all fp32, base-2 exponents).  The block
// joins its warps' states; a pair that is cut leaves a record of each segment,
// and the last block to finish joins them in block order, so the result does
// not depend on which one that is.
//
// Products run on m16n8k16 MMAs with the cached side as the 16 rows (tokens in
// Q K, channels in P V) and the g query heads of a KV head as the 8 columns.
// With g <= 4 (PACK) head h has columns 2 h and 2 h + 1, the value and the
// residual of its operand split into two bf16 terms (2^-17 relative), at no
// cost; with g > 4 the columns are heads.
//
// What bounds it: BF16 the copies (64 requests x 4100 visible keys of 8 heads,
// 1.07 GB: 166 us, 95% of the copy bandwidth); 4 bits in part the instructions
// that make operands of the codes, about 240 for 16 tokens (8 ragged requests of
// 8K to 128K tokens, 657 MB: 118 us, 82%), and for short calls the way in
// (positions, page table, first copies: 6 us) and out (the join: 5 us): batch 1 x
// 100K, 109 MB, 27.4 us, of which the loop takes 15.

#include "oscar_paged.cuh"

#include <algorithm>
#include <cmath>

#include <math_constants.h>

namespace oscar {
namespace {

constexpr float kLog2eW = 1.4426950408889634f;
constexpr float kLazyW = 8.0f;  // the accumulators are rescaled when the maximum grows by more than 2^8

// WIDE: 16 warps and one block per SM (4 bits), for few pairs, whose cuts each cost a join (8 pairs x 100K keys:
// 27.4 us, 29.8 us with two blocks of 8; x 32K 16.4, 18.8; but x 4K 13.6, 11.7); else two blocks of 8, one of which
// copies and computes while the other begins or joins a segment (9 pairs x 100K 36.3 us, 38.6 wide; 16 pairs 44.2, 52.4;
// 24 pairs 63.5, 66.9; 64 pairs of ragged lengths 118, 123; 224 pairs x 4160 visible keys 35.0, 41.3).  From 9 pairs on
// only calls of about 1000 keys are faster wide, by up to 2 us.  BF16 has one block of 8 (its units are larger).
template <bool INT4, bool WIDE>
struct Ring {
  static constexpr int kWarps = INT4 && WIDE ? 16 : 8;
  static constexpr int kBlocks = INT4 && !WIDE ? 2 : 1;              // blocks per SM
  static constexpr int kTiles = INT4 ? 2 : 1;                        // 16-token tiles of a unit
  static constexpr int kUnit = INT4 ? 2 * kTile4Bytes : 16 * kD * 4;  // bytes of a unit
  static constexpr int kStages = 3;
  static constexpr int kBytes = kWarps * kStages * kUnit;
};
constexpr int kWidePairs = 9;  // (query, KV head) pairs from which on the blocks are the smaller ones
// Units at a pair's ends that go to the neighbouring range (8 pairs x 100K keys: 27.4 us with 4 to 16, 35.4 us with
// none; 104 pairs x 1000 18.6 us with 4 or none, 14.2 with 8, 12.5 with 16; 224 pairs x 4160 35.0, 35.2 with 16)
constexpr int kSlack = 8;
constexpr int kMaxRows = 1024;  // query rows whose lengths a block adds up; with more, a block takes one whole pair

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
  // (not beyond the length: nothing there is held, and roundings of a low near 2^31 would overflow)
  s.low = a.window < 0 ? 0 : (int)min(max(p + 1 - a.window, 0ll), len);
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
  bool cut;  // the pairs' units are cut into equal ranges (else a block a pair)
  int most;  // cut: units of a row, at most, so that all of them stay below 2^30 whatever the lengths on the device
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
  // 4-bit: sums of the weights of each group since the levels' offset last came off.  Two heads a lane: as the
  // products of rows of ones, two MMAs a tile for sixteen instructions (8 ragged requests 126 -> 121 us); one head: in
  // [g][0] this lane's part, whose two additions a row are cheaper than the registers (batch 1 x 100K 28.1 us with them)
  float wsum[2][PACK ? 1 : 4];
  float o[8][4];
};

// 4-bit words to operands: the low byte of a 16-bit float without any exponent bits is a whole number of its smallest
// subnormals (fp16: 2^-24; bf16: 2^-133, whose first binade goes on where they end), so bytes and nibbles in place are
// operands, a low nibble as c and a byte as c + 16 c': four instructions for eight codes (8 ragged requests 115 us then; low
// and high nibbles masked each: five, 121 us; nibbles shifted under exponent bits, with offsets of 16 to 256 to cancel:
// six to eight, 139 us).  K: q c + q' c' = (q - q'/16) c + (q'/16) (c + 16 c'), so the queries go in as those, fp16 with a power
// of two that makes up for 2^-24.  V: the row of bytes less the row of low nibbles, at the end; the weights are bf16, for
// their range, and 2^64 times larger.  What is left is the levels' own 7.5: inside a tile's product for the logits, for P V
// against the sum of the weights, every kCentre units: the MMA truncates what it has summed by up to 2^-23 a step, and
// that is of the size of the offset's part, not of the result (taken off at the end alone, the result was off by 1% for
// 28 requests of 100,000 keys, 2% for 64, and lost at 1,000,000).
// nibbles (2 h, 2 h + 4) and bytes (h, h + 2) of a word
__device__ __forceinline__ void code_bytes(uint32_t w, int h, uint32_t& low, uint32_t& both) {
  both = h ? __byte_perm(w, 0u, 0x4341) : w & 0x00FF00FFu;
  low = (h ? both : w) & 0x000F000Fu;
}
// D = A B + C, m16n8k16, fp16 operands, fp32 sums
__device__ __forceinline__ void mma_f16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
constexpr float kOffset4 = 7.5f;
constexpr int kCentre = 16;  // (relative error at 1,000,000 keys 0.0017 with 8, 0.0018 with 16, 0.0023 with 32; the same time)
constexpr float kKUnit = 5.9604644775390625e-8f;  // 2^-24
constexpr float kVUp = 18446744073709551616.f, kVDown = 590295810358705651712.f;  // 2^64; 2^69 = 2^133 / 2^64
constexpr float kVUnit = 9.183549615799121e-41f;  // 2^-133

// value + residual of x as a bf16 pair (value in the low half)
__device__ __forceinline__ uint32_t split_bf16(float x) {
  const float v = bf16_lo(pack_bf16x2(x, 0.f));
  return pack_bf16x2(v, x - v);
}

template <bool PACK, bool INT4, bool WIDE>
__device__ __forceinline__ void window_body(const WindowArgs& wa) {
  using R = Ring<INT4, WIDE>;
  constexpr int kW = R::kWarps, kS = R::kStages, KU = R::kTiles, kH = PACK ? 1 : 2;
  const WindowLaunch& a = wa.a;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ __align__(16) float sm_q[kMaxG * kD];
  __shared__ float sm_ml[2][kW][kMaxG];
  __shared__ float sm_m[kMaxG], sm_l[kMaxG];
  __shared__ int sm_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, tq = lane & 3;
  __shared__ int pre[kMaxRows + 1], scan[kW];
  griddep_wait();
  griddep_launch_dependents();  // (behind the wait: what is before this kernel is complete once the next one starts)
  const int g = a.Hq / a.Hkv, rows = a.tok.n_tokens, G = gridDim.x, block = blockIdx.x;
  const bool few = rows <= 32;  // each warp adds the rows up for itself, lane i row i
  int at = 0, end = 1, total = 0;  // this block's range of all units
  int pre_l = 0, units_l = 0;                // few: units before row `lane` (of one KV head), and its own
  if (wa.cut) {
    int b;
    Seen s;
    auto units_of = [&](int i, bool report) {  // (far more than the host's bound allows: nothing, and an error)
      const int n = seen_by<KU>(a, i, b, s, report) ? s.tiles() / KU : 0;
      if (n > wa.most && report) set_error(a.err, kErrLength);
      return n > wa.most ? 0 : n;
    };
    if (few) {
      if (lane < rows) units_l = units_of(lane, block == 0 && warp == 0);
      pre_l = units_l;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, pre_l, o);
        if (lane >= o) pre_l += y;
      }
      total = __shfl_sync(0xffffffffu, pre_l, 31);
      pre_l -= units_l;
    } else {
      // pre[i]: units of the rows before row i
      constexpr int kPer = kMaxRows / (32 * kW);
      const int per = (rows + 32 * kW - 1) / (32 * kW), first = threadIdx.x * per;
      int n[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        n[i] = 0;
        if (i < per && first + i < rows) n[i] = units_of(first + i, block == 0);
        sum += n[i];
      }
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      int before = inc - sum;
      for (int w = 0; w < warp; ++w) before += scan[w];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < per && first + i < rows) {
          pre[first + i] = before;
          before += n[i];
          if (first + i == rows - 1) pre[rows] = before;
        }
      __syncthreads();
      total = pre[rows];
    }
    total *= a.Hkv;
    // queries that see nothing get zeros
    for (int i = block; i < rows; i += G) {
      const int n = few ? __shfl_sync(0xffffffffu, units_l, i) : pre[i + 1] - pre[i];
      if (n == 0 && seen_by<KU>(a, i, b, s, false))
        for (int c = threadIdx.x; c < a.Hq * (kD / 8); c += 32 * kW)
          reinterpret_cast<uint4*>(a.out + (size_t)i * a.Hq * kD)[c] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // the pair that unit x belongs to: its row, KV head, first unit and units
  auto pair_of = [&](int x, int& row, int& h, int& units) {
    int before;
    if (few) {
      row = __ffs(__ballot_sync(0xffffffffu, pre_l * a.Hkv <= x && x < (pre_l + units_l) * a.Hkv)) - 1;
      before = __shfl_sync(0xffffffffu, pre_l, row);
      units = __shfl_sync(0xffffffffu, units_l, row);
    } else {
      int hi_r = rows;
      row = 0;  // the last row whose units start at or before x (rows without units share their successor's start)
      while (hi_r - row > 1) {
        const int mid = (row + hi_r) >> 1;
        if (pre[mid] * a.Hkv <= x)
          row = mid;
        else
          hi_r = mid;
      }
      before = pre[row];
      units = pre[row + 1] - before;
    }
    const int in = x - before * a.Hkv;
    h = (int)__fdividef((float)in, (float)units);  // within one of the quotient, as long as it is below 2^20
    h += (h + 1) * units <= in ? 1 : h * units > in ? -1 : 0;
    return before * a.Hkv + h * units;
  };
  // where block k's range begins: near the k-th of G equal parts (a product of floats: the same everywhere and
  // monotonic in k, which is all that matters), or at the pair's edge when that is at most kSlack units away (a
  // segment costs as much as several units of every warp).  G is the grid, which the host sized from its bound of the
  // lengths; but when there are fewer units than blocks, as many blocks as have a unit for each warp, since a range
  // without units inside a pair would be one whose block adds nothing to the pair's counter and yet lies between the
  // pair's first and last (the rest begin at `total`: a little more than total / G takes the product past it)
  const float step = total >= G ? (float)total / (float)G
                                : (float)total / (float)max(1, (total + kW - 1) / kW) * (1.f + 1.f / (1 << 20));
  auto begin_of = [&](int k) {
    const int x = k >= G ? total : min(total, (int)(step * (float)k));
    if (x == 0 || x >= total) return x;
    int row, h, units;
    const int p = pair_of(x, row, h, units);
    return x - p <= kSlack && x - p < units ? p : p + units - x <= kSlack ? p + units : x;
  };
  auto block_of = [&](int x) {  // the block whose range holds unit x
    int k = min(G - 1, (int)__fdividef((float)x, step));
    while (begin_of(k) > x) --k;
    while (begin_of(k + 1) <= x) ++k;
    return k;
  };
  if (wa.cut) {
    at = begin_of(block);
    end = begin_of(block + 1);
  }
  for (bool again = false; at < end; again = true) {
  if (again) __syncthreads();  // the segment before is done with shared memory
  int row, h, u0 = 0, u1, units, b;
  Seen s;
  if (wa.cut) {
    u0 = at - pair_of(at, row, h, units);
    u1 = min(units, u0 + (end - at));
    seen_by<KU>(a, row, b, s, false);
  } else {
    row = block / a.Hkv;
    h = block % a.Hkv;
    if (!seen_by<KU>(a, row, b, s, h == 0 && threadIdx.x == 0)) return;
    u1 = units = s.tiles() / KU;
  }
  // this segment's units [u0, u1), this warp's: u0 + warp, + kW, ...
  const int pair0 = at - u0;  // the pair's first unit among all
  at += wa.cut ? u1 - u0 : 1;
  const uint32_t ring = smem_u32(sm) + warp * (kS * R::kUnit);
  int phys_l = -1, fetched = 0;  // lane i: the page of the warp's unit fetched - 32 + i
  uint32_t put = ring;  // the next unit copied goes there
  auto issue = [&](int i) {      // the warp's i-th unit
    if (i >= fetched) {
      const int u = u0 + warp + (fetched + lane) * kW;
      phys_l = -1;
      if (u < u1) phys_l = page_of(a.pages, b, s.tile(u * KU) >> 2, a.err, true);
      fetched += 32;
    }
    const int phys = __shfl_sync(0xffffffffu, phys_l, i & 31);
    const int u = u0 + warp + i * kW;
    if (u < u1) copy_unit<INT4>(a, s, s.tile(u * KU), phys, h, put, lane);
    put = put == ring + (kS - 1) * R::kUnit ? ring : put + R::kUnit;
    cp_async_commit();
    return phys;
  };
  const uint16_t* qrow = a.q + (size_t)row * a.q_stride + (size_t)h * g * kD;
  uint4 qx[4];  // 4 bits: pieces tq + 4 M of the column's query (loaded before the copies wait for their pages)
  if constexpr (INT4) {
    const int hh = PACK ? r >> 1 : r;
#pragma unroll
    for (int M = 0; M < 4; ++M)
      qx[M] = hh < g ? reinterpret_cast<const uint4*>(qrow + hh * kD)[tq + 4 * M] : make_uint4(0u, 0u, 0u, 0u);
  }
  int phys_q[kS];
#pragma unroll
  for (int i = 0; i < kS - 1; ++i) phys_q[i] = issue(i);

  // the queries as MMA columns: qf[k step][2], and the offset's part of the logits
  uint32_t qf[8][2];
  float q0[2][4];  // 4 bits: [group] the offset's part of a tile's logits, as the MMA's C
  float qscale[kH];  // logits to base-2 exponents, by the lane's heads
  if constexpr (INT4) {
    // q H / sqrt(128) as the append turns K: column r's head is row r of the MMAs, so that the lane ends up
    // with the channels of its column's fragments (k step 2 M + b2: k bits e, tq, kh = channel bits 0, (3, 4), 1)
    const uint32_t s1 = signs_bf16(odd_bits(2 * tq & r), odd_bits((2 * tq + 1) & r));
    float2 d[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        mma_bf16_acc(acc, word_of(qx[i >> 1], 2 * (i & 1)), 0u, word_of(qx[i >> 1], 2 * (i & 1) + 1), 0u, s1,
                     nt ? s1 ^ 0x80008000u : s1);
        d[i][nt] = make_float2(acc[0], acc[1]);
      }
    butterfly(d, 1);
    butterfly(d, 2);
    butterfly(d, 4);
    // fp16 with a power of two taken out (the largest channel becomes 2^14..2^15); PACK: value and residual (2^-22),
    // else the value alone (2^-11 of a channel's part of the logit)
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) top = fmaxf(top, fmaxf(fabsf(d[i][nt].x), fabsf(d[i][nt].y)));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^(14 - floor(log2 top)) and its inverse times 2^24, from the exponent bits (kept where both are normal)
    const int ex = min(max((int)(__float_as_uint(top) >> 23), 15), 244);
    const float up = __uint_as_float((uint32_t)(127 + 14 - (ex - 127)) << 23), down = __uint_as_float((uint32_t)(ex + 10) << 23);
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        const float x0 = kh ? d[ks][1].x * (up / 16.f) : fmaf(d[ks][1].x, -1.f / 16.f, d[ks][0].x) * up;
        const float x1 = kh ? d[ks][1].y * (up / 16.f) : fmaf(d[ks][1].y, -1.f / 16.f, d[ks][0].y) * up;
        __half2 v = __floats2half2_rn(x0, x1);
        if (PACK && (r & 1)) v = __floats2half2_rn(x0 - __low2float(v), x1 - __high2float(v));
        qf[ks][kh] = h2_as_u32(v);
        part[ks >> 2] = fmaf(kh ? -17.f * kOffset4 * kKUnit : -kOffset4 * kKUnit, __low2float(v) + __high2float(v), part[ks >> 2]);
      }
    // sums over the column's four lanes, then to the lanes that hold columns 2 tq, 2 tq + 1 of the logits
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      float x = part[gr];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      q0[gr][0] = q0[gr][2] = __shfl_sync(0xffffffffu, x, 4 * (2 * tq));
      q0[gr][1] = q0[gr][3] = __shfl_sync(0xffffffffu, x, 4 * (2 * tq + 1));
    }
    const float f = down * (kInvSqrt128 * a.sm_scale * kLog2eW);
    qscale[0] = __shfl_sync(0xffffffffu, f, 4 * (2 * tq));
    qscale[kH - 1] = PACK ? qscale[0] : __shfl_sync(0xffffffffu, f, 4 * (2 * tq + 1));
  } else {
    const int hh = PACK ? r >> 1 : r;
    const bool live = hh < g && !(PACK && (r & 1));  // a bf16 query has no residual
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qf[ks][0] = live ? *reinterpret_cast<const uint32_t*>(qrow + hh * kD + 16 * ks + 2 * tq) : 0u;
      qf[ks][1] = live ? *reinterpret_cast<const uint32_t*>(qrow + hh * kD + 16 * ks + 8 + 2 * tq) : 0u;
    }
    qscale[0] = qscale[kH - 1] = a.sm_scale * kLog2eW;
  }
  const bool split = u0 > 0 || u1 < units;
  const int kf = split ? block_of(pair0) : block;  // the blocks that hold the pair's units
  const int pieces = split ? block_of(pair0 + units - 1) - kf + 1 : 1;

  State<PACK, INT4> st;
#pragma unroll
  for (int i = 0; i < kH; ++i) {
    st.m[i] = -INFINITY;
    st.l[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) st.o[i][e] = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < (PACK ? 1 : 4); ++e) st.wsum[i][e] = 0.f;

  // units of which the query sees all: [in0, in1) of the window
  const int in0 = (s.low + 15) >> 4, in1 = s.len >> 4;
  const int mine = u1 - u0 - warp > 0 ? (u1 - u0 - warp + kW - 1) / kW : 0;
  for (int i = 0; i < mine; ++i) {
    __syncwarp();
    phys_q[kS - 1] = issue(i + kS - 1);
    cp_async_wait<kS - 1>();
    __syncwarp();
    const uint32_t stage = put;  // (kS - 1 units ahead of the one used now: the copy after next goes where that is)
    const int T = s.tile((u0 + warp + i * kW) * KU);
    const bool bad = phys_q[0] < 0;
#pragma unroll
    for (int j = 0; j < kS - 1; ++j) phys_q[j] = phys_q[j + 1];
    // logits x[tile][row half][head]; x qscale is the base-2 exponent
    float x[KU][2][kH];
#pragma unroll
    for (int k = 0; k < KU; ++k) {
      if constexpr (INT4) {
        const uint32_t tb = stage + k * kTile4Bytes;
        const uint4 w0 = lds128(tb + 16 * lane), w1 = lds128(tb + 512 + 16 * lane);
        float acc[2][4];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t a0, a1, a2, a3;
          code_bytes(word_of(w0, ks >> 1), ks & 1, a0, a2);
          code_bytes(word_of(w1, ks >> 1), ks & 1, a1, a3);
          if ((ks & 3) == 0)  // the group's sum starts from the offset's part
            mma_f16_from(acc[ks >> 2], a0, a1, a2, a3, qf[ks][0], qf[ks][1], q0[ks >> 2]);
          else
            mma_f16(acc[ks >> 2], a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
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
          x[k][rh][0] = acc[2 * rh];
          if constexpr (!PACK) x[k][rh][kH - 1] = acc[2 * rh + 1];
        }
      }
    }
    // positions that the query does not see (or whose page is bad) drop out by selection
    if (bad || !((T >= in0 || 16 * (T + KU) <= s.sinks) && T + KU <= in1)) {
      uint32_t hid = 0;  // bit 2 k + rh: token r + 8 rh of tile k
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
      if constexpr (INT4) {  // a V row nobody wrote may hold any scale: 0 in the stage
#pragma unroll
        for (int i = 0; i < 2 * KU; ++i)
          if (tq == 0 && ((hid >> i) & 1u))
            asm volatile("st.shared.b32 [%0], 0;\n" ::"r"(stage + (i >> 1) * kTile4Bytes + kTile4Scales + 64 + 4 * (r + 8 * (i & 1))) : "memory");
        __syncwarp();
      }
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
    for (int e = 0; e < kH; ++e) grow = grow || (sub[e] - st.m[e]) * qscale[e] > kLazyW || (st.m[e] == -INFINITY && sub[e] > -INFINITY);
    if (__any_sync(0xffffffffu, grow)) {
      float f[kH];
#pragma unroll
      for (int e = 0; e < kH; ++e) {
        const float m = fmaxf(st.m[e], sub[e]);
        f[e] = st.m[e] == -INFINITY ? 0.f : exp2_fast((st.m[e] - m) * qscale[e]);
        st.m[e] = m;
        st.l[e] *= f[e];
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[mt][e] *= PACK ? f[0] : f[(e & 1) * (kH - 1)];
      if constexpr (INT4)
#pragma unroll
        for (int gr = 0; gr < 2; ++gr)
#pragma unroll
          for (int e = 0; e < (PACK ? 1 : 4); ++e) st.wsum[gr][e] *= PACK ? f[0] : f[(e & 1) * (kH - 1)];
    }
#pragma unroll
    for (int e = 0; e < kH; ++e) sub[e] = st.m[e] == -INFINITY ? 0.f : -st.m[e] * qscale[e];
#pragma unroll
    for (int k = 0; k < KU; ++k) {
      // weights, as the MMA's columns: transposed 8 x 8 blocks (tokens 0-7 and 8-15)
      uint32_t bv[INT4 ? 2 : 1][2];
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        float p[kH];
#pragma unroll
        for (int e = 0; e < kH; ++e) {
          p[e] = exp2_fast(fmaf(x[k][rh][e], qscale[e], sub[e]));
          st.l[e] += p[e];
        }
        if constexpr (INT4) {
          const uint32_t u = lds32(stage + k * kTile4Bytes + kTile4Scales + 64 + 4 * (r + 8 * rh));
          const float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&u));
#pragma unroll
          for (int e = 0; e < kH; ++e) p[e] *= kVUp;
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            const float sg = gr ? sc.y : sc.x;
            if constexpr (PACK) {
              const float w = p[0] * sg;
              st.wsum[gr][0] += w;
              bv[gr][rh] = movmatrix_trans(split_bf16(w));
            } else {
              // one bf16 term per weight (2^-9): the offset is taken off with the rounded weights
              bv[gr][rh] = movmatrix_trans(pack_bf16x2(p[0] * sg, p[kH - 1] * sg));
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
          if constexpr (!PACK) {
            constexpr uint32_t kOnes = 0x3F803F80u;
            mma_bf16_acc(st.wsum[gr], kOnes, kOnes, kOnes, kOnes, bv[gr][0], bv[gr][1]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t wq = word_of(w, q);
            uint32_t a0, a1, a2, a3;
            code_bytes(wq, 0, a0, a1);
            code_bytes(wq, 1, a2, a3);
            mma_bf16_acc(st.o[4 * gr + q], a0, a1, a2, a3, bv[gr][0], bv[gr][1]);
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
    if (INT4 && ((i & (kCentre - 1)) == kCentre - 1 || i + 1 == mine)) {
      // the levels' offset off the sums: rows of low nibbles c, and of bytes c + 16 c'
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        if constexpr (PACK)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) st.wsum[gr][0] += __shfl_xor_sync(0xffffffffu, st.wsum[gr][0], o);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < kH; ++e) {  // (PACK: the weights are the sum of two columns, the offset comes off the first)
            float(&o)[4] = st.o[4 * gr + q];
            o[e] = fmaf(-kOffset4 * kVUnit, st.wsum[gr][e], o[e]);
            o[2 + e] = fmaf(-17.f * kOffset4 * kVUnit, st.wsum[gr][e], o[2 + e]);
          }
#pragma unroll
        for (int e = 0; e < (PACK ? 1 : 4); ++e) st.wsum[gr][e] = 0.f;
      }
    }
  }
  cp_async_wait<0>();
  // sums over the lanes of a column
#pragma unroll
  for (int e = 0; e < kH; ++e)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], o);
  __syncthreads();  // every warp is done with the ring: it becomes the warps' accumulators [warp][head][128]
  float* so = reinterpret_cast<float*>(sm);
  if (r == 0)
#pragma unroll
    for (int e = 0; e < kH; ++e) {
      const int hh = PACK ? tq : 2 * tq + e;
      sm_ml[0][warp][hh] = st.m[e] * qscale[e];  // (a base-2 exponent from here on)
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
        if constexpr (INT4) {
          if (hf) y -= st.o[mt][0] + st.o[mt][1];
          y *= hf ? kVDown / 16.f : kVDown;
        }
        if (tq < g) so[(warp * g + tq) * kD + ch] = y;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = st.o[mt][2 * hf + e];
          if constexpr (INT4) {
            if (hf) y -= st.o[mt][e];
            y *= hf ? kVDown / 16.f : kVDown;
          }
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
  const int rec = (g * (kD + 2) + 3) & ~3;  // floats of a record: o[g][128], m[g], l[g]
  // block k's records: 2 k (a pair that began in an earlier block), 2 k + 1 (a pair that goes on in the next)
  float* records = reinterpret_cast<float*>(a.workspace + a.plan.off_records);
  float* mine_rec = records + (size_t)(2 * block + (block == kf)) * rec;
  for (int i = threadIdx.x; i < g * kD; i += 32 * kW) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) y = fmaf(so[w * g * kD + i], sm_ml[0][w][i >> 7], y);
    if (split)
      mine_rec[i] = y;
    else
      sm_q[i] = y;
  }
  if (split) {
    if (threadIdx.x < g) {
      mine_rec[g * kD + threadIdx.x] = sm_m[threadIdx.x];
      mine_rec[g * kD + g + threadIdx.x] = sm_l[threadIdx.x];
    }
    // the last block of the pair joins the pieces' records, in block order
    __syncthreads();
    if (threadIdx.x == 0) {
      // releases the block's records (the barrier put them before it) and acquires the other blocks'
      unsigned* counter = reinterpret_cast<unsigned*>(a.workspace) + kf;  // one pair at most goes on from block kf
      unsigned t;
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(t) : "l"(counter) : "memory");
      sm_last = t == (unsigned)pieces - 1u;
      if (sm_last) *counter = 0u;
    }
    __syncthreads();
    if (!sm_last) continue;
    auto piece = [&](int i) { return records + (size_t)(2 * (kf + i) + (i == 0)) * rec; };
    // thread -> (four channels of a head, every kParts-th piece): its loads go out before the factors are known
    constexpr int kCells = (PACK ? 4 : 8) * (kD / 4), kParts = 32 * kW / kCells, kAhead = 8;
    const int cell = threadIdx.x % kCells, part = threadIdx.x / kCells, ch = cell / (kD / 4);
    float4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = part + i * kParts;
      v[i] = k < pieces && ch < g ? __ldcg(reinterpret_cast<const float4*>(piece(k)) + cell) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // a warp a head: maximum, sum and the pieces' factors (over the ring: every record is in the workspace)
    float* fac = so;  // [head][pieces], then the parts' sums [part][cell]
    float4* sums = reinterpret_cast<float4*>(so + kMaxG * G);
    for (int hh = warp; hh < g; hh += kW) {
      float M = -INFINITY, L = 0.f, m0 = -INFINITY, l0 = 0.f;
      if (lane < pieces) {
        m0 = __ldcg(piece(lane) + g * kD + hh);
        l0 = __ldcg(piece(lane) + g * kD + g + hh);
      }
      M = m0;
      for (int i = lane + 32; i < pieces; i += 32) M = fmaxf(M, __ldcg(piece(i) + g * kD + hh));
      M = warp_max(M);
      for (int i = lane; i < pieces; i += 32) {
        const float m = i < 32 ? m0 : __ldcg(piece(i) + g * kD + hh), f = m == -INFINITY ? 0.f : exp2_fast(m - M);
        L = fmaf(i < 32 ? l0 : __ldcg(piece(i) + g * kD + g + hh), f, L);
        fac[hh * pieces + i] = f;
      }
      L = warp_sum(L);
      if (lane == 0) sm_l[hh] = L;
    }
    __syncthreads();
    if (ch < g) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = part + i * kParts;
        const float f = k < pieces ? fac[ch * pieces + k] : 0.f;
        y = make_float4(fmaf(v[i].x, f, y.x), fmaf(v[i].y, f, y.y), fmaf(v[i].z, f, y.z), fmaf(v[i].w, f, y.w));
      }
#pragma unroll 4
      for (int k = part + kAhead * kParts; k < pieces; k += kParts) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(piece(k)) + cell);
        const float f = fac[ch * pieces + k];
        y = make_float4(fmaf(u.x, f, y.x), fmaf(u.y, f, y.y), fmaf(u.z, f, y.z), fmaf(u.w, f, y.w));
      }
      sums[part * kCells + cell] = y;
    }
    __syncthreads();
    if (part == 0 && ch < g) {
      float4 y = sums[cell];
#pragma unroll
      for (int i = 1; i < kParts; ++i) {
        const float4 u = sums[i * kCells + cell];
        y = make_float4(y.x + u.x, y.y + u.y, y.z + u.z, y.w + u.w);
      }
      reinterpret_cast<float4*>(sm_q)[cell] = y;
    }
  }
  __syncthreads();
  // normalise, turn back, round once
  for (int hh = warp; hh < g; hh += kW) {
    float sum = sm_l[hh];
    if (sum == 0.f) {  // it sees nothing (zeros), or its logits are all -infinity (NaN)
      bool any = false;
      for (int u = lane; u - lane < units && !any; u += 32) {
        const int j = u < units ? 16 * s.tile(u * KU) : s.len, end = min(j + 16 * KU, s.len);
        any = __any_sync(0xffffffffu, j < s.len && (j < s.sinks || s.low < end) && page_of(a.pages, b, j / kPage, a.err, false) >= 0);
      }
      if (any) sum = CUDART_NAN_F;
    }
    const float f = sum != 0.f ? 1.f / sum : 0.f;
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
}

template <bool PACK, bool INT4, bool WIDE>
__global__ void __launch_bounds__(32 * Ring<INT4, WIDE>::kWarps, Ring<INT4, WIDE>::kBlocks)
    window_split_kernel(const __grid_constant__ WindowArgs wa) {
  window_body<PACK, INT4, WIDE>(wa);
}

template <bool PACK, bool INT4, bool WIDE>
cudaError_t launch_one(const WindowLaunch& a, cudaStream_t stream) {
  using R = Ring<INT4, WIDE>;
  static std::atomic<uint64_t> done;
  const void* fn = reinterpret_cast<const void*>(window_split_kernel<PACK, INT4, WIDE>);
  static_assert(R::kWarps * kMaxG * kD * 4 <= R::kBytes, "the warps' accumulators in the ring");
  const cudaError_t e = smem_attr_once(fn, R::kBytes, done);
  if (e != cudaSuccess) return e;
  WindowArgs wa;
  wa.a = a;
  wa.cut = a.plan.items > 0;
  wa.most = wa.cut ? (1 << 30) / (a.tok.n_tokens * a.Hkv) : 0;
  const long long blocks = wa.cut ? a.plan.items : (long long)a.tok.n_tokens * a.Hkv;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  void* args[] = {&wa};
  return launch_pdl(fn, dim3((unsigned)blocks), dim3(32 * R::kWarps), R::kBytes, stream, args);
}

bool wide(int64_t rows, int Hkv) { return rows * Hkv < kWidePairs; }

template <bool INT4, bool WIDE>
int blocks_of(int64_t units, int num_sms) {
  using R = Ring<INT4, WIDE>;
  return (int)std::min<int64_t>((int64_t)R::kBlocks * num_sms, std::max<int64_t>(1, units / (2 * R::kWarps)));
}

}  // namespace

// Blocks of a call: what the GPU holds at once, but no more than give a warp two units.  Many rows are not cut
// (items 0): a block takes a whole pair.
WindowPlan plan_window(bool int4, int64_t rows, int Hq, int Hkv, int64_t max_keys, int num_sms) {
  WindowPlan p;
  const int tok = 16 * (int4 ? Ring<true, true>::kTiles : Ring<false, true>::kTiles);
  const int64_t units = rows * Hkv * ((max_keys + tok - 1) / tok + 1);
  p.items = rows > kMaxRows || units >= (INT64_C(1) << 30) ? 0
            : !int4               ? blocks_of<false, true>(units, num_sms)
            : wide(rows, Hkv)     ? blocks_of<true, true>(units, num_sms)
                                  : blocks_of<true, false>(units, num_sms);
  static_assert(Ring<true, false>::kBlocks == kCutBlocks && Ring<true, true>::kBlocks <= kCutBlocks && Ring<false, true>::kBlocks <= kCutBlocks);
  const int64_t most = (int64_t)kCutBlocks * num_sms;  // blocks of any call
  p.off_records = window_counter_bytes(num_sms);
  p.total = p.off_records + (size_t)most * 2 * ((Hq / Hkv) * (kD + 2) + 3) * sizeof(float);
  return p;
}

cudaError_t launch_window_split(const WindowLaunch& a, cudaStream_t stream) {
  const bool pack = a.Hq / a.Hkv <= 4;
  if (a.pages4 == nullptr) return pack ? launch_one<true, false, true>(a, stream) : launch_one<false, false, true>(a, stream);
  if (wide(a.tok.n_tokens, a.Hkv))
    return pack ? launch_one<true, true, true>(a, stream) : launch_one<false, true, true>(a, stream);
  return pack ? launch_one<true, true, false>(a, stream) : launch_one<false, true, false>(a, stream);
}

}  // namespace oscar
