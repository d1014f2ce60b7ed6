// chunk_tc.cuh -- attention of chunks of new tokens over a 16-bit compressed
// cache on the tensor cores.
//
//   out[j] = sum_t p_t V_t / sum_t p_t,  p_t = 2^(scale log2(e) q_j . K_t - m),
// one pass over the row's tokens with a running maximum m and sum. A unit is up to
// 128 or 256 query rows of one kv head; a persistent CTA per SM takes an equal run
// of 96-token tiles (chunk.cuh).
//
// chunk_tc, one launch: warps with fixed roles.
//   0-3, 4-7   two softmax groups: thread = query row of a 128-row tile. They
//              read scores from tensor memory, keep the running maximum and sum
//              and write the weights back as binary16 (the A operand of P V).
//   8-10       rebuild key tiles, 11-13 value tiles: codes and outliers straight
//              from the pages into binary16 operands in shared memory (32 tokens
//              per warp, 32 channels of four tokens per lane).
//   14         issues the products: S = Q K^T (both operands in shared memory)
//              and O += P V (P in tensor memory, V read token-major).
// Units of more than 128 query rows (par = 1) pair two row tiles on every K and
// V tile; smaller ones (par = 2) give the two groups alternate tiles of the same
// rows, each with an accumulator of its own; up to 32 rows (SMALL) the softmax
// groups need one warp each, and the other six rebuild every other tile.
//
// chunk_rebuild, then chunk_attend: where many row blocks read the same tiles they
// are rebuilt once, as they will lie in shared memory, and fetched by bulk copies.
// The softmax groups then have the SM's issue slots and instruction caches to
// themselves, and two warps share 32 rows, half of a tile's columns each (one warp
// per 32 rows: 2 chunks of 4096 tokens 540 us, two 500 us when that was built, 484 us now).
//
// The low-rank part of prompt tokens is not rebuilt per element: with K = D + L Rf^T,
// q K^T = q D^T + (q Rf) L^T takes 16 more columns of the inner dimension, and
// P V = P D + (P L) Rf^T 16 more output columns, joined with Rf when a segment
// ends. An outlier's slot holds its value minus the token's low-rank part there.
// Flushed blocks (20 tokens with an Rf of their own, say) are rebuilt in full.
// Tensor memory: two score tiles of 96 columns, the weights over their first 48, two
// accumulators of 128 + 16; with tiles of 128 the extra 16 would not fit its 512.
//
// The softmax reference of a row moves only when a tile's maximum passes it by
// 2^8, so that the accumulator in tensor memory is rarely rescaled. Weights are
// 2^7 times the formula's (their sum too): with 2^8 above the reference they stay
// below 2^15, and down to 2^-21 of it they keep binary16's 11 bits. Rounding to
// binary16 happens to K and V (to the scale, the middle value and the sum of a code: twice
// the error of one rounding; to an outlier less its low-rank part; for flushed blocks
// after every four ranks), to q Rf and L, and to the weights (their sum takes them
// unrounded): the tensor cores take no wider operands at this rate, and an output's error
// (0.7e-3 to 1.1e-3 of its norm, where rounding a binary32 result alone gives 0.2e-3) stays
// well below what quantizing K and V to 4 bits does. Sums, statistics and accumulators are
// binary32. A bf16 cache's values can lie outside
// binary16's range: every 32 tokens of K and V, and every query row, carry a power of
// two that scales them into it (2^0 in ordinary ranges). An fp16 cache's are halved.
//
// What bounds it (one B200, 1965 MHz). 16 rows x 4 tokens x 32 heads over 8192 4-bit
// tokens (826 MB): 0.57 ms, 1.46 TB/s, bound by the producers, which issue about 1250
// instructions per 32 tokens and tensor at 0.5 per cycle and scheduler; their code
// is kept small because with straight-line copies for keys and values a tile took five
// times as long in instruction fetches. 2048 tokens x 32 heads over 8192 (311 GFLOP):
// 0.45 ms, 690 TFLOP/s: about 3500 cycles a tile of 2 x 128 rows, of which the products take
// 2060 and the exponentials 1540 (16 lanes per cycle and SM), at the 1.7 GHz the power limit leaves.
#pragma once

#include "chunk.cuh"
#include "common.cuh"

namespace gear {

constexpr int kTcThreads = 512;   // (warp 15 idles: it completes a group of four for the register split)
// Registers per thread: 128 at launch; the softmax groups hand 32 to the others. (The
// assembler takes the split in whole-program compilation and without calls only: these
// files are compiled without relocatable device code, and everything is inlined.)
constexpr int kSoftRegs = 96, kProdRegs = 160;
static_assert(kSoftRegs + kProdRegs == 2 * 65536 / kTcThreads, "the split uses what the launch has");
constexpr int kTile = kChunkTile;
constexpr uint32_t kTcHalf = kTile * 128;                   // 64 channels of a K or V tile
constexpr uint32_t kTcQ = 0;                                // two row tiles of 32 KB
constexpr uint32_t kTcK = 65536;                            // two stages of two halves
constexpr uint32_t kTcV = kTcK + 2 * 2 * kTcHalf;           // two stages of two halves and the L columns
constexpr uint32_t kTcQx = kTcV + 2 * 3 * kTcHalf;          // q Rf: 128 rows x 16, two row tiles
constexpr uint32_t kTcKx = kTcQx + 2 * 4096;                // L of a key tile, two stages
constexpr uint32_t kTcRf = kTcKx + 2 * kTile * 32;          // Rf of block 0: K, V
constexpr uint32_t kTcRfBytes = 128 * 16 * 4;
constexpr uint32_t kTcPair = kTcRf + kTcRfBytes;            // chunk_attend, which stages no Rf of values: exchanges of row halves
constexpr uint32_t kTcBars = kTcRf + 2 * kTcRfBytes;
constexpr uint32_t kTcSmem = kTcBars + 1024 + 1024;
static_assert(kTcSmem <= 232448, "shared memory of one CTA");
// A rebuilt tile in memory: K (two halves, L columns), V (two halves, L columns), exponents.
constexpr uint32_t kImgV = 2 * kTcHalf + kTile * 32, kImgE = kImgV + 3 * kTcHalf;
static_assert(kImgE + 32 <= kImgBytes && kImgBytes % 128 == 0, "layout of a rebuilt tile");
constexpr uint32_t kImgSmem = kImgE + 2 * kTcRfBytes + 256 + 1024;
constexpr uint32_t kTmO = 2 * kTile, kTmOCols = 144;        // accumulators in tensor memory
constexpr float kWeightShift = 7.0f;                        // log2 of what weights are multiplied by

struct __align__(16) TcBars {
  int32_t ek[4][4], ev[2][4];   // exponents of the 32-token groups of a K / V tile; ev[][3]: of the V unit's Rf
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], qfull[2], sfull[2], pfull[2], ofull[2];
  // The K unit's Rf has been staged; no softmax warp reads it any more. One phase each per staging, and
  // every warp on both sides takes part in each: a wait is never more than one phase from what it is for,
  // which is all that a parity tells apart.
  uint64_t rfull, rfree;
  int32_t er;                   // exponent of the K unit's Rf
  int32_t pu[12][8];            // what a producer warp needs of its unit now and then
  uint32_t tmem;
  int32_t* status;              // the device error word
  int32_t dead;                 // a bounded wait ran out: nothing waits any more
};

// Bounded wait; a probe sleeps until the phase completes, for a microsecond at most.
__device__ __forceinline__ void tc_wait_slow(TcBars* b, uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 255) == 0) {
      if (*reinterpret_cast<volatile int32_t*>(&b->dead)) return;
      if (global_timer_ns() - t0 > kSpinNanos) break;
    }
  }
  *reinterpret_cast<volatile int32_t*>(&b->dead) = 1;
  atomicCAS(b->status, 0, (int32_t)GEAR_ERR_TIMEOUT);
}
__device__ __forceinline__ void tc_wait(TcBars* b, uint64_t* bar, uint32_t parity) {
  if (!mbar_try_wait(bar, parity)) tc_wait_slow(b, bar, parity);
}

// D[tmem] (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x4(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^e, e clamped to binary32's normal range
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }

__device__ __forceinline__ int exp_of(float m) { return (int)((__float_as_uint(m) >> 23) & 255) - 127; }

// Exponent of the power of two that what is at most `m` is divided by: none in [2^-6, 2^(top + 1)),
// else one that puts m at 2^top. Queries and Rf meet in a product of 128 terms that is rounded to
// binary16: 2^7 2^5 2^3 = 2^15 at most.
constexpr int kQueryTop = 4, kRfTop = 2;
__device__ __forceinline__ int range_exp(float m, int top) {
  const int e = exp_of(m);
  return e >= -6 && e <= top ? 0 : max(e - top, -120);
}

// An fp16 cache's keys and values are all taken half as large: rounded codes and outliers less their
// low-rank part stay in range up to 65504. (Below 2^-13 that costs a bit of the little that binary16 has there.)
constexpr int kF16Exp = 1;

// bf16: the same for 32 tokens of keys or values: none in [2^-6, 2^14), else one that brings m to the near end of
// that range. Groups of like size then have like exponents on either side of an end: where a group's
// exponent is below its neighbours', its softmax weights take the difference (weigh), and lose bits to it
// once it is a good deal more than the 2^7 that they have in hand.
__device__ __forceinline__ int group_exp(float m) {
  const int e = exp_of(m);
  return max(e < -6 ? e + 6 : e >= 14 ? e - 13 : 0, -120);
}

// the n lowest bits (none for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Which of the 32 tokens from t on a row sees: those below its limit, but for padding [plen, b0).
__device__ __forceinline__ uint32_t seen_bits(int t, int limit, int plen, int b0) {
  return low_bits(limit - t) & (low_bits(plen - t) | ~low_bits(b0 - t));
}

// |x| 2^e, kept away from 0 and infinity so that a masked score, an infinity, stays one.
__device__ __forceinline__ float score_scale(float x, int e) {
  return fminf(fmaxf(fabsf(x) * pow2i(e >> 1) * pow2i(e - (e >> 1)), 1e-36f), 1e36f);
}

// Byte offset of 16-byte chunk c (channels 8c ..) of row r in an operand tile of
// ROWS rows: 64 channels at a time, 128-byte rows with the 128-byte swizzle.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (uint32_t)((c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Byte offset of 16-byte chunk c (0 or 1) of row r in a K-major operand of 16
// columns without swizzle: 8 rows x 16 bytes are contiguous.
__device__ __forceinline__ uint32_t ext_off(int r, int c) { return (uint32_t)((r >> 3) * 256 + c * 128 + (r & 7) * 16); }
__device__ __forceinline__ uint64_t smem_desc_ext(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(256 >> 4) << 32 | (uint64_t)1 << 46;
}

template <typename T>
__device__ __forceinline__ float to_f(uint16_t bits) {
  if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(bits));
  else return __uint_as_float((uint32_t)bits << 16);
}

// Two packed cache values, times f, as binary16.
template <typename T>
__device__ __forceinline__ uint32_t to_half2(uint32_t w, float f) {
  if constexpr (std::is_same<T, __half>::value) {
    if (f == 1.0f) return w;
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pack_half2(v.x * f, v.y * f);
  } else return pack_half2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}
// max(m, |both values|); NaN is passed over
template <typename T>
__device__ __forceinline__ float max_abs2(uint32_t w, float m) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
  }
  return fmaxf(m, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
}

// The larger magnitudes of two bf16 pairs.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
  const uint32_t v = w & 0x7fff7fffu;
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&v));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float warp_max(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));   // m >= 0
}

// ------------------------------------------------------------------ producers
// Bytes of a warp's 32 compressed tokens: codes and (scale, zero) of lane =
// (token tsub + 8 j, channels 32 qd ..) with qd = lane % 4 and tsub = lane / 4, its bit 1
// flipped for qd >= 2 (the eight lanes of a store phase then write eight different 16-byte
// columns, although they hold two halves of the channels); outlier entries lane + 32 i
// of the group's consecutive list; the first four L entries of token lane.
template <int BITS>
struct RawTile {
  uint32_t code[4][BITS];
  uint2 meta[4];              // two binary32, or .x two binary16
  uint32_t oi[4], ov[4];      // channel, value bits
  uint2 l;
};

// Loads of what is read once: they leave the L1 lines to others.
__device__ __forceinline__ uint4 ldg_stream(const uint4* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg_stream(const uint2* p) {
  uint2 v;
  asm("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ldg_stream(const uint32_t* p) {
  uint32_t v;
  asm("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
// (into a 32-bit register: a conversion would wait for the load at once)
__device__ __forceinline__ uint32_t ldg_stream(const uint16_t* p) {
  uint32_t v;
  asm("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ldg_stream(const uint8_t* p) {
  uint32_t v;
  asm("ld.global.nc.L1::no_allocate.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// Untiled bulk copy of this GPU's memory (16-byte aligned, whole 16-byte pieces).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
template <int N>
__device__ __forceinline__ float max_of(const uint32_t (&s)[N]) {
  float m = __uint_as_float(s[0]), n = __uint_as_float(s[1]);
#pragma unroll
  for (int c = 2; c + 4 <= N; c += 4) {
    m = max3(m, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    n = max3(n, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
  }
  return max3(m, n, fmaxf(__uint_as_float(s[N - 2]), __uint_as_float(s[N - 1])));
}
// Scores that a row does not see become -infinity.
template <int N>
__device__ __forceinline__ void hide(uint32_t (&s)[N], uint32_t seen) {
#pragma unroll
  for (int c = 0; c < N; ++c)
    if (!(seen >> c & 1)) s[c] = 0xff800000u;
}

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Codes to values, two channels per instruction. A code is masked where it lies in its byte, in
// the mantissa of a binary16 number whose bit there is worth 1: 1024 for bits 0 on, 256 for 2, 64 for
// 4 and 16 for 6. Less that number and the middle code m (2^(b-1)) it is exact, and
//   value = (code - m) scale + (zero + m scale)
// rounds scale, the middle value and the sum once each to 11 bits: relative to the group's
// half range and its middle, not to `zero` (a code taken from 0 would lose a bit or two).
template <int BITS>
struct HalfCodes {
  static constexpr uint32_t kMid = 1u << (BITS - 1);
  uint32_t s, z;
  __device__ __forceinline__ HalfCodes(float scale, float zero) {
    const float m = fmaf((float)kMid, scale, zero);
    z = pack_half2(m, m);
    s = pack_half2(scale, scale);
  }
  // binary16 whose mantissa bit `bit` is worth 1, and that number plus kMid, negative
  static constexpr uint32_t one_at(int bit) { return (uint32_t)(25 - bit) << 10; }
  static constexpr uint32_t less_mid(int bit) { return 0x8000u | one_at(bit) | kMid << bit; }
  // eight channels: chunk i of the lane's four
  __device__ __forceinline__ uint4 eight(const uint32_t (&code)[BITS], int i) const {
    uint32_t o[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t c, off;
      if constexpr (BITS == 8) {
        c = __byte_perm(code[2 * i + (p >> 1)], 0x64646464u, p & 1 ? 0x4342 : 0x4140);
        off = less_mid(0) | less_mid(0) << 16;
      } else if constexpr (BITS == 4) {   // bytes p, 0, p, 0: code 2p in bits 0 on, code 2p + 1 in bits 4 on
        c = (__byte_perm(code[i], 0, 0x4040 | p | p << 8) & 0x00F0000Fu) | one_at(0) | one_at(4) << 16;
        off = less_mid(0) | less_mid(4) << 16;
      } else {
        const int byte = 2 * (i & 1) + (p >> 1), at = p & 1 ? 4 : 0;
        c = (__byte_perm(code[i >> 1], 0, 0x4040 | byte | byte << 8) & (3u << at | 3u << (18 + at))) | one_at(at) | one_at(at + 2) << 16;
        off = less_mid(at) | less_mid(at + 2) << 16;
      }
      o[p] = hfma2(hadd2(c, off), s, z);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

// Entries past the rank, which may never have been written, as zeros.
__device__ __forceinline__ float4 clip4(float4 v, int left) {
  return make_float4(v.x, left > 1 ? v.y : 0.0f, left > 2 ? v.z : 0.0f, left > 3 ? v.w : 0.0f);
}

__device__ __forceinline__ float4 scale4(float4 v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }

// Four L entries q .. of a token (row of r_max binary16) as two half2, those past the rank zero.
__device__ __forceinline__ uint2 l_clip(uint2 v, int left) {
  if (left < 4) {
    v.y = left == 3 ? v.y & 0xffffu : 0u;
    if (left < 2) v.x &= left == 1 ? 0xffffu : 0u;
  }
  return v;
}
__device__ __forceinline__ uint2 l_quad(const __half* row, int r_max, int q, int rank) {
  uint2 v = make_uint2(0, 0);
  if ((r_max & 3) == 0) {   // rows of whole 8-byte pieces
    v = __ldg(reinterpret_cast<const uint2*>(row + q));
  } else {
    const uint16_t* u = reinterpret_cast<const uint16_t*>(row + q);
    v.x = __ldg(u);
    if (q + 1 < rank) v.x |= (uint32_t)__ldg(u + 1) << 16;
    if (q + 2 < rank) v.y = __ldg(u + 2);
    if (q + 3 < rank) v.y |= (uint32_t)__ldg(u + 3) << 16;
  }
  return l_clip(v, rank - q);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// The low-rank part of flushed blocks' tokens of a group, added to their rows
// (lane = four channels). Tokens [lead, end) of the group; g: Rf of block 1 at the
// lane's channels, `past` = the group's first token counted from block 1's start;
// lrow: L row of token lane, row0: first operand row.
__device__ __forceinline__ void add_blocks(uint32_t tile, int row0, int lead, int end, int past, int n_b, const float* g,
                                               int64_t blk_floats, int rp, int rank, const __half* lrow, int r_max,
                                               float f) {
  const int lane = lane_id();
#pragma unroll 1
  for (int q = 0; q < rank; q += 4) {
    const uint2 lq = l_quad(lrow, r_max, q, rank);
    float4 v[4];
    int cur = -1;
#pragma unroll 1
    for (int tk = lead; tk < end; ++tk) {
      const int blk = (past + tk) / n_b;
      if (blk != cur) {   // an Rf of its own
        cur = blk;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = clip4(__ldg(reinterpret_cast<const float4*>(g + blk * blk_floats + e * rp + q)), rank - q);
      }
      const uint32_t lx = __shfl_sync(0xffffffffu, lq.x, tk), ly = __shfl_sync(0xffffffffu, lq.y, tk);
      const float2 la = __half22float2(*reinterpret_cast<const __half2*>(&lx));
      const float2 lb = __half22float2(*reinterpret_cast<const __half2*>(&ly));
      const uint32_t p = tile + tile_off<kTile>(row0 + tk, lane >> 1) + (lane & 1) * 8;
      const uint2 o = lds64(p);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&o.x));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&o.y));
      const float z[4] = {x.x, x.y, y.x, y.y};
      float s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[e] = fmaf(f, fmaf(la.x, v[e].x, fmaf(la.y, v[e].y, fmaf(lb.x, v[e].z, lb.y * v[e].w))), z[e]);
      sts64(p, make_uint2(pack_half2(s[0], s[1]), pack_half2(s[2], s[3])));
    }
  }
  __syncwarp();
}

// Rf of a block (128 rows of rp) into shared memory by one warp (`write`), entries past the
// rank as zeros; the exponent that its entries are to be divided by.
__device__ __forceinline__ int rf_to_smem(const float* g, int rp, int rank, uint32_t rf, bool write) {
  float m = 0.0f;
#pragma unroll 4
  for (int i = lane_id(); i < 32 * rp; i += 32) {   // four entries; every warp sees all of them
    float4 v = __ldg(reinterpret_cast<const float4*>(g) + i);
    const int left = rank - (i * 4) % rp;
    v = clip4(v, left);
    if (left < 1) v.x = 0.0f;
    m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    if (write)
      sts128(rf + i * 16, make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)));
  }
  return range_exp(warp_max(m), kRfTop);
}

// One code path for keys and values: the producers, the softmax groups and the
// product issuer run different code at the same time, and together have to fit
// the instruction caches (with both unrolled, a tile took five times as long).
// SETS = 2: two sets of three key and three value warps take every other tile each.
template <typename T, int BITS, bool KC, int SETS = 1>
struct Producer {
  static constexpr bool SC = !std::is_same<T, __half>::value;   // values carry exponents
  const ChunkArgs& a;
  const bool isk;
  TcBars* bars;
  // operand tiles and low-rank columns in shared memory: stage 0, bytes per stage
  uint32_t tile0, tile_step, l0, l_step;
  uint32_t rf;          // Rf of block 0 there, entries past the rank zero
  int w, lane, tsub, qd, set;
  // of the current unit
  int nc, b0, plen, unit;
  volatile int32_t* pu; // the rest, in shared memory: registers are short
  // lanes 0 .. 4: the per-token array that the lane asks for ahead, and its bytes per token
  const uint8_t* ahead;
  int ahead_row;

  __device__ __forceinline__ int mrow() const { return a.G * (a.meta_f16 ? 4 : 8); }
  __device__ __forceinline__ void init() {
    ahead = reinterpret_cast<const uint8_t*>(codes());
    ahead_row = lane == 0 ? 16 * BITS : 0;
    if (lane == 1 && !(KC && isk)) ahead = reinterpret_cast<const uint8_t*>(meta()), ahead_row = mrow();
    if (lane == 2) ahead = oidx(), ahead_row = a.k;
    if (lane == 3) ahead = reinterpret_cast<const uint8_t*>(oval()), ahead_row = 2 * a.k;
    if (lane == 4) ahead = reinterpret_cast<const uint8_t*>(lfac()), ahead_row = 2 * a.r_max;
  }

  // arrays of the tensor (selected where they are used: held, they would cost 14 registers)
  __device__ __forceinline__ const uint32_t* codes() const { return isk ? a.K.codes : a.V.codes; }
  __device__ __forceinline__ const float* meta() const { return isk ? a.K.meta : a.V.meta; }
  __device__ __forceinline__ const uint8_t* oidx() const { return isk ? a.K.oidx : a.V.oidx; }
  __device__ __forceinline__ const uint16_t* oval() const { return reinterpret_cast<const uint16_t*>(isk ? a.K.oval : a.V.oval); }
  __device__ __forceinline__ const __half* lfac() const { return reinterpret_cast<const __half*>(isk ? a.K.lfac : a.V.lfac); }
  __device__ __forceinline__ const float* rfac() const { return isk ? a.K.rfac : a.V.rfac; }
  __device__ __forceinline__ const T* buf() const { return reinterpret_cast<const T*>(isk ? a.K.buf : a.V.buf); }

  __device__ __forceinline__ int b() const { return pu[0]; }
  __device__ __forceinline__ int h() const { return pu[1]; }
  __device__ __forceinline__ int nb() const { return pu[2]; }
  __device__ __forceinline__ int keys() const { return pu[3]; }
  __device__ __forceinline__ int er() const { return pu[4]; }
  __device__ __forceinline__ int tok0() const { return pu[5]; }

  // Rows of the per-token arrays (fewer than 2^31).
  __device__ __forceinline__ int first_row(int t, int pg) const {
    if (!a.table) return unit * a.n_max + t;
    const int off = a.plog >= 0 ? t & (a.page_tokens - 1) : t % a.page_tokens;
    return (min(max(pg, 0), a.num_pages - 1) * a.H + h()) * a.page_tokens + off;
  }
  // (looked at in first_row only, a tile later)
  __device__ __forceinline__ int page_of(int t) const {
    if (!a.table || t >= nc) return 0;
    int pg;   // (volatile: the load is issued here, not where its result is used)
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(pg) : "l"(a.table + (int64_t)b() * a.ppr + (a.plog >= 0 ? t >> a.plog : t / a.page_tokens)));
    return pg;
  }
  __device__ __forceinline__ bool padded(int t) const { return t >= plen && t < b0; }
  // token of outlier entry e (k <= 16, e < 512)
  __device__ __forceinline__ int entry_token(int e) const { return (e * a.krecip) >> 16; }
  __device__ __forceinline__ bool quads() const { return (a.r_max & 3) == 0; }   // L rows of whole 8-byte pieces
  __device__ __forceinline__ const __half* l_row(int row) const { return lfac() + (int64_t)row * a.r_max; }

  // The group's bytes; every load is issued before any result is looked at. Pages and
  // contiguous units hold whole groups: tokens past the last one are read too (nothing
  // comes of them).
  __device__ __forceinline__ void load(RawTile<BITS>& r, int row0) const {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(codes()) + (int64_t)(row0 + tsub) * (16 * BITS) + qd * (4 * BITS);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BITS == 2) {
        const uint2 v = ldg_stream(reinterpret_cast<const uint2*>(p + j * (128 * BITS)));
        r.code[j][0] = v.x, r.code[j][1] = v.y;
      } else {
#pragma unroll
        for (int c = 0; c < BITS / 4; ++c) {
          const uint4 v = ldg_stream(reinterpret_cast<const uint4*>(p + j * (128 * BITS)) + c);
          r.code[j][4 * c] = v.x, r.code[j][4 * c + 1] = v.y, r.code[j][4 * c + 2] = v.z, r.code[j][4 * c + 3] = v.w;
        }
      }
    }
    if (!(KC && isk)) {
      const int g = (qd * 32) >> a.glog;
      const uint8_t* m = reinterpret_cast<const uint8_t*>(meta()) + (int64_t)(row0 + tsub) * mrow();
      const int m8 = 8 * mrow();
      if (a.meta_f16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.meta[j].x = ldg_stream(reinterpret_cast<const uint32_t*>(m + j * m8) + g);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.meta[j] = ldg_stream(reinterpret_cast<const uint2*>(m + j * m8) + g);
      }
    }
    const uint8_t* oi = oidx() + (int64_t)row0 * a.k + lane;
    const uint16_t* ov = oval() + (int64_t)row0 * a.k + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < a.k) {
        r.oi[i] = ldg_stream(oi + 32 * i);
        r.ov[i] = ldg_stream(ov + 32 * i);
      }
    if (quads()) r.l = ldg_stream(reinterpret_cast<const uint2*>(l_row(row0 + lane)));
  }
  __device__ __forceinline__ float2 scale_zero(const RawTile<BITS>& r, int j) const {
    return a.meta_f16 ? __half22float2(*reinterpret_cast<const __half2*>(&r.meta[j].x))
                      : make_float2(__uint_as_float(r.meta[j].x), __uint_as_float(r.meta[j].y));
  }

  // Asks for a later group's bytes (consecutive in each array, whole 16-byte pieces): the
  // loads of a tile then find them in L2.
  __device__ __forceinline__ void prefetch(int row0) const {
    if (ahead_row > 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ahead + (int64_t)row0 * ahead_row), "r"(32 * ahead_row));
  }

  __device__ __forceinline__ int slot_of(int t) const {
    return t < b0 ? t >> a.glog : ((b0 + a.g - 1) >> a.glog) + ((t - b0) >> a.glog);
  }

  // Byte address of the low-rank columns q .. q + 3 of the lane's token.
  __device__ __forceinline__ uint32_t l_addr(int st, int q) const {
    const int r = w * 32 + lane;
    return l0 + st * l_step + (isk ? ext_off(r, q >> 3) : tile_off<kTile>(r, 16 + (q >> 3))) + (q & 4) * 2;
  }
  // L of the group's prompt tokens (lane = token) into the extra columns, zeros for
  // all others; f undoes the scale of the values, and of Rf (which carries the size of the
  // unit's values: without it L 2^-ex leaves binary16 where they are far from 1). Columns
  // past the rank were cleared when the kernel began.
  __device__ __forceinline__ void put_l(int t0, int row0, uint2 lq, int st, float f) const {
    const int t = t0 + lane;
    const bool has = t < b0 && !padded(t);
#pragma unroll 1
    for (int q = 0; q < a.blk0_rank; q += 4) {
      uint2 v = make_uint2(0, 0);
      if (has) {
        v = q == 0 && quads() ? l_clip(lq, a.blk0_rank) : l_quad(l_row(row0 + lane), a.r_max, q, a.blk0_rank);
        v.x = to_half2<__half>(v.x, f);
        v.y = to_half2<__half>(v.y, f);
      }
      sts64(l_addr(st, q), v);
    }
  }

  // Largest magnitude that the group's compressed tokens are scaled for.
  __device__ __forceinline__ float compressed_max(const RawTile<BITS>& r, int t0, int row0, int ne) const {
    constexpr float top = (float)((1 << BITS) - 1);
    float m = 0.0f;
    if (KC && isk) {
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const int t = min(t0 + tsub + 8 * j, nc - 1);
        if (padded(t)) continue;
        const float2* s = reinterpret_cast<const float2*>(meta()) + ((int64_t)unit * a.ch_slots + slot_of(t)) * 128 + qd * 32;
#pragma unroll 4
        for (int c = 0; c < 32; ++c) m = fmaxf(m, fmaxf(fabsf(s[c].y), fabsf(fmaf(top, s[c].x, s[c].y))));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 z = scale_zero(r, j);
        const int t = t0 + tsub + 8 * j;
        if (t < nc && !padded(t)) m = fmaxf(m, fmaxf(fabsf(z.y), fabsf(fmaf(top, z.x, z.y))));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 32 * i;
      if (e < ne && !padded(t0 + entry_token(e))) m = fmaxf(m, fabsf(to_f<T>((uint16_t)r.ov[i])));
    }
#pragma unroll 1
    for (int e = lane + 128; e < ne; e += 32)
      if (!padded(t0 + entry_token(e))) m = fmaxf(m, fabsf(to_f<T>(__ldg(oval() + (int64_t)row0 * a.k + e))));
    return warp_max(m);
  }

  // Whether a scale of the group (of any of its 32 tokens' places), times f, lies below binary16's normal
  // range, 2^-14 (0 does not): it would keep fewer than 11 bits.
  static constexpr uint32_t kFineScale = 0x38800000u;
  __device__ __forceinline__ bool fine_scales(const RawTile<BITS>& r, float f) const {
    uint32_t least = ~0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) least = min(least, __float_as_uint(scale_zero(r, j).x * f) - 1u);
    return __any_sync(0xffffffffu, least < kFineScale - 1u);
  }

  // D of the group's compressed tokens, times f. Padding, whatever it decodes to, becomes zeros.
  __device__ __forceinline__ void dequant(const RawTile<BITS>& r, int t0, uint32_t tile, float f) const {
    // rows tsub + 8 j have the same row & 7: the swizzle is the lane's own
    const uint32_t at = tile + (qd >> 1) * kTcHalf + (w * 32 + tsub) * 128, c0 = (((qd & 1) * 4) ^ (tsub & 7)) << 4;
    const bool fine = !(KC && isk) && fine_scales(r, f);
    uint32_t lifted = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + tsub + 8 * j;
      const bool in = t < nc, live = !padded(t);
      if (KC && isk) {
        const float4* sz = reinterpret_cast<const float4*>(reinterpret_cast<const float2*>(meta()) +
                                                           ((int64_t)unit * a.ch_slots + slot_of(min(t, nc - 1))) * 128);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {   // every channel has a scale of its own: binary32
          float x[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 v = __ldg(sz + (qd * 4 + i) * 4 + e);
            x[2 * e] = fmaf(code_of(r.code[j], i * 8 + 2 * e), v.x, v.y) * f;
            x[2 * e + 1] = fmaf(code_of(r.code[j], i * 8 + 2 * e + 1), v.z, v.w) * f;
          }
          uint4 o = make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
          if (!live) o = make_uint4(0, 0, 0, 0);
          if (in) sts128(at + j * 1024 + (c0 ^ (i << 4)), o);
        }
      } else {
        const float2 m = scale_zero(r, j);
        float scale = live ? m.x * f : 0.0f, zero = live ? m.y * f : 0.0f;
        if (fine) {
          // 2^12 times the values for now; next to a middle of 8 and more the scale's lost bits are below a rounding
          if (scale < __uint_as_float(kFineScale) && fabsf(zero) < 8.0f) scale *= 4096.0f, zero *= 4096.0f, lifted |= 1u << j;
        }
        const HalfCodes<BITS> h2(scale, zero);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 o = h2.eight(r.code[j], i);
          if (in) sts128(at + j * 1024 + (c0 ^ (i << 4)), o);
        }
      }
    }
    if (fine) {   // rare, and so in a few instructions
#pragma unroll 1
      for (int n = 0; n < 16; ++n)
        if ((lifted >> (n >> 2) & 1) && t0 + tsub + 8 * (n >> 2) < nc) {
          const uint32_t p = at + (n >> 2) * 1024 + (c0 ^ ((n & 3) << 4)), down = 0x0C000C00u;   // 2^-12
          const uint4 o = lds128(p);
          sts128(p, make_uint4(hmul2(o.x, down), hmul2(o.y, down), hmul2(o.z, down), hmul2(o.w, down)));
        }
    }
  }
  // Code of the lane's channel c (register index by selection: c is not constant).
  __device__ __forceinline__ static float code_of(const uint32_t (&code)[BITS], int c) {
    uint32_t w = code[0];
#pragma unroll
    for (int i = 1; i < BITS; ++i)
      if (c * BITS / 32 == i) w = code[i];
    return (float)((w >> (c * BITS % 32)) & ((1u << BITS) - 1u));
  }

  // The group's outliers over their slots, less the low-rank part that the extra columns
  // add for prompt tokens. With up to four entries per lane and a rank up to four the
  // entries go together, token factors by shuffle; the rest one by one.
  __device__ __forceinline__ void put_outliers(const RawTile<BITS>& r, int t0, int row0, uint32_t tile, int ne, float f) const {
    const int rp = rpad_of(a.r_max);
    const bool together = quads() && a.blk0_rank <= 4;
    const bool pad = plen < b0, flat = t0 + 32 <= b0;   // (the same for all lanes)
    if (together) {
      const uint2 lc = l_clip(r.l, a.blk0_rank);
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= a.k) break;
        const int tk = entry_token(lane + 32 * i);   // (i < k: below 32)
        uint2 l;
        l.x = __shfl_sync(0xffffffffu, lc.x, tk);
        l.y = __shfl_sync(0xffffffffu, lc.y, tk);
        v[i] = to_f<T>((uint16_t)r.ov[i]);
        if (a.blk0_rank > 0) v[i] = less(v[i], l, lds_f4(rf + (r.oi[i] & 127) * rp * 4), flat || t0 + tk < b0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < a.k) place(t0, lane + 32 * i, ne, r.oi[i], v[i], tile, f, pad);
    }
#pragma unroll 1
    for (int e = lane + (together ? 128 : 0); e < ne; e += 32) {
      const int tk = entry_token(e), c = __ldg(oidx() + (int64_t)row0 * a.k + e);
      float v = to_f<T>(__ldg(oval() + (int64_t)row0 * a.k + e));
#pragma unroll 1
      for (int q = 0; q < a.blk0_rank; q += 4)
        v = less(v, l_quad(l_row(row0 + tk), a.r_max, q, a.blk0_rank), lds_f4(rf + ((c & 127) * rp + q) * 4), t0 + tk < b0);
      place(t0, e, ne, c, v, tile, f, pad);
    }
  }
  __device__ __forceinline__ void place(int t0, int e, int ne, uint32_t c, float v, uint32_t tile, float f, bool pad) const {
    const uint32_t tk = entry_token(e);
    // channel c of row 32 w + tk: half c / 64, 16-byte column (c / 8) ^ tk within it
    const uint32_t at = tile + w * 4096 + tk * 128 + ((c & 64) ? kTcHalf : 0u) + (((c << 1) ^ (tk << 4)) & 0x70) + ((c << 1) & 0xe);
    if (e < ne && !(pad && padded(t0 + tk))) sts16(at, __half_as_ushort(__float2half_rn(v * f)));
  }
  __device__ __forceinline__ static float less(float v, uint2 l, float4 g, bool on) {
    const float2 la = __half22float2(*reinterpret_cast<const __half2*>(&l.x));
    const float2 lb = __half22float2(*reinterpret_cast<const __half2*>(&l.y));
    const float u = fmaf(-la.x, g.x, fmaf(-la.y, g.y, fmaf(-lb.x, g.z, fmaf(-lb.y, g.w, v))));
    return on ? u : v;
  }

  // Where token t >= nc lies (buffered, the chunk's own), null behind the last key.
  __device__ __forceinline__ const uint4* raw_row(int t) const {
    if (t < nc || t >= keys()) return nullptr;
    const int o = t - nc, n = nb();
    const T* p = o < n ? buf() + ((int64_t)unit * a.n_b + o) * 128
                        : reinterpret_cast<const T*>(isk ? a.kn : a.vn) + (int64_t)(tok0() + o - n) * (isk ? a.ks : a.vs) +
                              h() * 128;
    return reinterpret_cast<const uint4*>(p) + qd * 4;
  }

  // Two of the lane's uncompressed tokens (tsub + 16 jj, + 8), zeros behind the last key.
  __device__ __forceinline__ void load_raw(uint4 (&v)[2][4], int t0, int jj) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4* p = raw_row(t0 + tsub + 16 * jj + 8 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[j][i] = make_uint4(0, 0, 0, 0);
        if (p) v[j][i] = __ldg(p + i);
      }
    }
  }

  // Exponent that the group's uncompressed tokens need.
  __device__ __forceinline__ int raw_exp(int t0) const {
    uint32_t m2 = 0;   // two magnitudes at a time
#pragma unroll 1
    for (int jj = 0; jj < 2; ++jj) {
      uint4 v[2][4];
      load_raw(v, t0, jj);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m2 = abs_max2(m2, v[j][i].x);
          m2 = abs_max2(m2, v[j][i].y);
          m2 = abs_max2(m2, v[j][i].z);
          m2 = abs_max2(m2, v[j][i].w);
        }
    }
    return group_exp(warp_max(max_abs2<T>(m2, 0.0f)));
  }

  static constexpr uint32_t kHalf2 = 0x38003800u;   // 2^-kF16Exp twice
  // Buffered tokens and the chunk's own (t >= nc), times f.
  __device__ __forceinline__ void copy_raw(int t0, uint32_t tile, float f) const {
#pragma unroll 1
    for (int jj = 0; jj < 2; ++jj) {
      uint4 v[2][4];
      load_raw(v, t0, jj);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int tk = tsub + 16 * jj + 8 * j;
        if (t0 + tk >= nc) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 x = v[j][i];
            const uint4 o = SC ? make_uint4(to_half2<T>(x.x, f), to_half2<T>(x.y, f), to_half2<T>(x.z, f), to_half2<T>(x.w, f))
                               : make_uint4(hmul2(x.x, kHalf2), hmul2(x.y, kHalf2), hmul2(x.z, kHalf2), hmul2(x.w, kHalf2));
            sts128(tile + tile_off<kTile>(w * 32 + tk, qd * 4 + i), o);
          }
        }
      }
    }
  }

  // Rf of the unit's prompt block into shared memory (96 threads), and the exponent that its
  // entries are divided by in q Rf, or (bf16 values) when P L is multiplied by it.
  __device__ __forceinline__ void stage_rf() {
    const int rp = rpad_of(a.r_max), bar = isk ? 1 : 2;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(96 * SETS) : "memory");   // no warp still reads the last unit's
    const int er = rf_to_smem(rfac() + (int64_t)unit * a.nblk_max * 128 * rp, rp, a.blk0_rank, rf, w == 0 && set == 0);
    if (lane == 0) pu[4] = er;
    if (bars && isk && w == 0 && set == 0 && lane == 0) *reinterpret_cast<volatile int32_t*>(&bars->er) = er;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(96 * SETS) : "memory");
    if (bars && isk && lane == 0) mbar_arrive(&bars->rfull);
  }

  // The low-rank columns past the rank stay zero.
  __device__ __forceinline__ void clear_l(int stages) const {
    for (int st = 0; st < stages; ++st)
      for (int q = 0; q < 16; q += 4) sts64(l_addr(st, q), make_uint2(0, 0));
  }

  // Takes up unit h of sequence i, with the keys of row block t.
  __device__ __forceinline__ bool take(int i, int hh, int t) {
    const int b = a.row[i], now = b * a.H + hh;
    nc = a.ncomp[i];
    b0 = a.b0[i];
    plen = a.plen ? min(max(__ldg(a.plen + b), 0), b0) : b0;
    const bool fresh = now != unit;
    unit = now;
    __syncwarp();
    if (lane == 0) {
      pu[0] = b;
      pu[1] = hh;
      pu[2] = a.nbuf[i];
      pu[3] = chunk_unit_keys(a, i, t);
      pu[5] = a.tok0[i];
    }
    __syncwarp();
    return fresh && nc > 0 && a.blk0_rank > 0;   // an Rf to stage
  }

  // The warp's group of a tile into stage st; its exponent. cur: the group's bytes.
  __device__ __forceinline__ int produce(RawTile<BITS>& cur, int t0, int row0, int st) const {
    const uint32_t tile = tile0 + st * tile_step;
    const bool mixed = t0 < nc && t0 + 32 > nc;   // a group that ends in uncompressed tokens: one exponent for both
    const int ne = t0 < nc ? min(32, nc - t0) * a.k : 0;
    int ex = -120;
    float f = 0.5f;   // 2^-kF16Exp
    if constexpr (SC) {
      if (t0 >= nc || mixed) ex = raw_exp(t0);
      if (t0 < nc) ex = max(ex, group_exp(compressed_max(cur, t0, row0, ne)));
    }
    if constexpr (SC) f = pow2i(-ex);
    if (t0 < nc) {
      dequant(cur, t0, tile, f);
      put_l(t0, row0, cur.l, st, SC || isk ? pow2i(er() - (SC ? ex : kF16Exp)) : f);   // (fp16 values: without Rf's)
      __syncwarp();
      if (t0 + 32 > b0 && nc > b0 && a.buffer_rank > 0) {
        const int rp = rpad_of(a.r_max);
        add_blocks(tile, w * 32, max(0, b0 - t0), min(32, nc - t0), t0 - b0, a.n_b,
                   rfac() + ((int64_t)unit * a.nblk_max + 1) * 128 * rp + lane * 4 * rp, 128 * rp, rp, a.buffer_rank,
                   l_row(row0 + min(lane, nc - 1 - t0)), a.r_max, f);
      }
      put_outliers(cur, t0, row0, tile, ne, f);
    } else {
      put_l(max(t0, b0), row0, make_uint2(0, 0), st, 1.0f);   // no L columns here
    }
    if (t0 >= nc || mixed) copy_raw(t0, tile, f);
    return ex;
  }

  // Tiles of the fused attention kernel.
  __device__ __forceinline__ void run() {
    const int total = a.tile0[a.nseq], end = min(total, (int)(blockIdx.x + 1) * a.seg);
    uint64_t* full = isk ? bars->kfull : bars->vfull;
    uint64_t* empty = isk ? bars->kempty : bars->vempty;
    init();
    clear_l(2);   // (two sets: both clear both stages, before anything is written there)
    asm volatile("bar.sync %0, %1;" ::"r"(isk ? 1 : 2), "n"(96 * SETS) : "memory");
    int it = 0;
    unit = -1;
    if (lane == 0) pu[4] = 0, pu[6] = 0;   // [6]: Rf's staged
    __syncwarp();
    const int begin = blockIdx.x * a.seg;
    ChunkUnit u;
    for (int x = begin; x < end;) {
      u = x == begin ? chunk_find(a, x) : chunk_next(a, u);
      x = max(x, u.tile);
      if (x >= end) break;
      const int x1 = min(end, u.tile + u.tiles);
      if (take(u.i, u.h, u.t)) {
        const int staged = pu[6];
        __syncwarp();
        if (lane == 0) pu[6] = staged + 1;
        if (isk && staged > 0) tc_wait(bars, &bars->rfree, (staged - 1) & 1);   // the softmax groups have read the last one
        stage_rf();
      }
      // the set's tiles: number x + skip on, every SETS-th
      const int n = x1 - x, skip = SETS == 2 ? (it ^ set) & 1 : 0;
      constexpr int kStep = SETS * kTile;
      int t0 = (x + skip - u.tile) * kTile + w * 32;
      // pages are looked up three tiles ahead, lines asked for two ahead
      int row[3];
      int pg[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) pg[i] = page_of(t0 + i * kStep);
#pragma unroll
      for (int i = 0; i < 3; ++i) row[i] = first_row(t0 + i * kStep, pg[i]);
      RawTile<BITS> cur;
      if (t0 < nc) load(cur, row[0]);
#pragma unroll 1
      for (int j = skip; j < n; j += SETS, t0 += kStep) {
        if (j + 2 * SETS < n && t0 + 2 * kStep < nc) prefetch(row[2]);
        const int pg3 = page_of(t0 + 3 * kStep);
        const int tile = it + j, st = tile & 1;
        tc_wait(bars, &empty[st], ((tile >> 1) & 1) ^ 1);
        const int ex = produce(cur, t0, row[0], st);
        if (SC && lane == 0) {
          if (isk) bars->ek[tile & 3][w] = ex;
          else bars->ev[st][w] = ex;
          if (!isk && w == 0) bars->ev[st][3] = er();
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        // the next tile's bytes, asked for two tiles ago: they arrive while the product of this
        // one is awaited
        row[0] = row[1];
        row[1] = row[2];
        if (j + SETS < n && t0 + kStep < nc) load(cur, row[0]);
        row[2] = first_row(t0 + 3 * kStep, pg3);
      }
      it += n;
      x = x1;
    }
  }

  // Tiles [x, end) of chunk_rebuild (numbered by a.img0), one after the other through one
  // stage: rebuilt, then stored as they lie in shared memory.
  __device__ __forceinline__ void run_images(int x, int end) {
    init();
    clear_l(1);
    unit = -1;
    if (lane == 0) pu[4] = 0;
    __syncwarp();
    const int bar = isk ? 3 : 4;
    while (x < end) {
      int i = 0, hi = a.nseq;
      while (hi - i > 1) {
        const int m = (i + hi) >> 1;
        if (a.img0[m] <= x) i = m;
        else hi = m;
      }
      const int per = (a.img0[i + 1] - a.img0[i]) / a.H, hh = (x - a.img0[i]) / per;
      const int first = a.img0[i] + hh * per, x1 = min(end, first + per);
      if (take(i, hh, chunk_blocks(a, i) - 1)) stage_rf();
      int t0 = (x - first) * kTile + w * 32;
      int row = first_row(t0, page_of(t0)), pg = page_of(t0 + kTile);
      RawTile<BITS> cur;
      if (t0 < nc) load(cur, row);
#pragma unroll 1
      for (; x < x1; ++x, t0 += kTile) {
        const int next = first_row(t0 + kTile, pg);
        if (x + 1 < x1 && t0 + kTile < nc) prefetch(next);
        pg = page_of(t0 + 2 * kTile);
        const int ex = produce(cur, t0, row, 0);
        uint8_t* dst = a.img + (int64_t)x * kImgBytes;
        if (SC && lane == 0) {
          reinterpret_cast<int32_t*>(dst + kImgE)[(isk ? 0 : 4) + w] = ex;
          if (!isk && w == 0) reinterpret_cast<int32_t*>(dst + kImgE)[7] = er();
        }
        row = next;
        if (x + 1 < x1 && t0 + kTile < nc) load(cur, row);
        fence_proxy_async_smem();
        asm volatile("bar.sync %0, 96;" ::"r"(bar) : "memory");
        if (w == 0 && lane == 0) {
          const uint32_t bytes = 2 * kTcHalf + (isk ? kTile * 32 : kTcHalf);
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(isk ? dst : dst + kImgV), "r"(tile0),
                       "r"(bytes)
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        asm volatile("bar.sync %0, 96;" ::"r"(bar) : "memory");
      }
    }
    if (w == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
};

// ------------------------------------------------------------------ softmax
// The warp's 32 rows of the result, channels 64 hv .. + 63, 32 at a time: accumulator plus (P L) Rf^T,
// times the lane's `mul`, to row `at` (elements) of the output or of the partial rows. Rf and then the
// rows go through the warp's 4 KB of the query tile, which no product reads any more, so that eight
// lanes write a row's 128 bytes. Lanes that each wrote their own row and read Rf from memory took 15000
// cycles a segment: 12 ragged rows of 2-bit codes 265 us, this way 248 us (long units alike to 1 %).
template <typename T>
__device__ __forceinline__ void store_rows(const ChunkArgs& a, uint32_t own, uint32_t to, const float* gv, float rscale, int rp,
                                           int rank, int hv, float mul, bool real, int64_t at, bool whole) {
  const int lane = lane_id();
  const uint32_t reals = __ballot_sync(0xffffffffu, real);
#pragma unroll 1
  for (int c0 = 64 * hv; c0 < 64 * hv + 64; c0 += 32) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(to + c0, o);
    for (int q = 0; q < rank; q += 4) {
      float4 f = clip4(__ldg(reinterpret_cast<const float4*>(gv + (c0 + lane) * rp + q)), rank - q);
      if constexpr (!std::is_same<T, __half>::value) f = scale4(f, rscale);
      sts128(own + (lane * 16 + q) * 4, make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w)));
    }
    __syncwarp();
    tmem_ld_wait();
#pragma unroll 1
    for (int q = 0; q < rank; q += 4) {
      uint32_t wl[4];
      tmem_ld_32x32b_x4(to + 128 + q, wl);
      tmem_ld_wait();
#pragma unroll
      for (int e = 1; e < 4; ++e)
        if (q + e >= rank) wl[e] = 0;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float4 f = lds_f4(own + (c * 16 + q) * 4);
        float v = fmaf(__uint_as_float(wl[0]), f.x, __uint_as_float(o[c]));
        v = fmaf(__uint_as_float(wl[1]), f.y, v);
        v = fmaf(__uint_as_float(wl[2]), f.z, v);
        o[c] = __float_as_uint(fmaf(__uint_as_float(wl[3]), f.w, v));
      }
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * mul);
    if (!whole || a.out_dtype == GEAR_F32) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        sts128(own + lane * 128 + ((c ^ (lane & 7)) << 4), make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
      __syncwarp();
      float* p = whole ? reinterpret_cast<float*>(a.out) : a.part;
#pragma unroll 4
      for (int k = 0; k < 8; ++k) {
        const int row = 4 * k + (lane >> 3), c = lane & 7;
        const int64_t to_row = __shfl_sync(0xffffffffu, at, row);
        const uint4 v = lds128(own + row * 128 + ((c ^ (row & 7)) << 4));
        if (reals >> row & 1) *reinterpret_cast<uint4*>(p + to_row + c0 + 4 * c) = v;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __uint_as_float(o[8 * c + 2 * e]), y = __uint_as_float(o[8 * c + 2 * e + 1]);
          if constexpr (std::is_same<T, __half>::value) {
            w[e] = pack_half2(x, y);
          } else {
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(x, y);
            w[e] = *reinterpret_cast<const uint32_t*>(&b2);
          }
        }
        sts128(own + lane * 128 + ((c ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 8 * k + (lane >> 2), c = lane & 3;
        const int64_t to_row = __shfl_sync(0xffffffffu, at, row);
        const uint4 v = lds128(own + row * 128 + ((c ^ (row & 7)) << 4));
        if (reals >> row & 1) *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + to_row + c0 + 8 * c) = v;
      }
    }
    __syncwarp();
  }
}

// SPLIT (chunk_attend): two warps share 32 rows, half `hv` of them has 48 of a tile's columns,
// read once and held, with loops unrolled, and half of the row's other work. They exchange
// maxima and sums through shared memory. Otherwise one warp, 32 columns at a time, twice.
// PAR: a.par where the kernel knows it, else 0.
template <typename T, bool SPLIT, int PAR>
__device__ __forceinline__ void softmax_role(const ChunkArgs& a, TcBars* bars, uint8_t* smem, int grp, int hv) {
  const int par = PAR ? PAR : a.par;
  constexpr bool SC = !std::is_same<T, __half>::value;   // values carry exponents
  const int tid = threadIdx.x & 127, lane = tid & 31, wq = tid >> 5;
  const int total = a.tile0[a.nseq], end = min(total, (int)(blockIdx.x + 1) * a.seg);
  const uint32_t lanes = (uint32_t)(wq * 32) << 16;
  const uint32_t ts = bars->tmem + grp * kTile + lanes, to = bars->tmem + kTmO + grp * kTmOCols + lanes;
  const int rp = rpad_of(a.r_max);
  const uint32_t sb = smem_u32(smem);
  // the other warp's value of slot 0, 1 (maxima of even and odd tiles), 2 (queries) or 3 (sums); a slot's
  // next use is behind another exchange
  const uint32_t mine = sb + kTcPair + ((grp * 2 + hv) * 128 + tid) * 4, other = mine + (hv ? -512 : 512);
  [[maybe_unused]] auto meet = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + grp * 4 + wq) : "memory"); };
  [[maybe_unused]] auto exchange = [&](int slot, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + slot * 2048), "f"(v) : "memory");
    meet();
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(other + slot * 2048) : "memory");
    return r;
  };
  int64_t rf_unit = -1;
  int it = 0, nq = 0, ns = 0, nrf = 0;   // tiles of the CTA; segments and tiles of this group; K units' Rf
  const int begin = blockIdx.x * a.seg;
  ChunkUnit u;
  for (int x = begin; x < end;) {
    u = x == begin ? chunk_find(a, x) : chunk_next(a, u);
    x = max(x, u.tile);
    if (x >= end) break;
    const int i = u.i, x1 = min(end, u.tile + u.tiles), n = x1 - x;
    const int rows = a.n[i] * a.hq;
    const int r = u.t * a.R + (par == 1 ? grp * 128 : 0) + tid;
    const bool real = r < min(rows, (u.t + 1) * a.R);
    const bool any = __any_sync(0xffffffffu, real);
    const int b0 = a.b0[i], base = a.ncomp[i] + a.nbuf[i];
    const int rank = a.ncomp[i] > 0 ? a.blk0_rank : 0;
    const int64_t unit = (int64_t)a.row[i] * a.H + u.h;
    const int tok = r / a.hq, j = r - tok * a.hq;
    const int limit = real ? base + (a.kn ? tok + 1 : 0) : 0;
    const int plen = a.plen ? min(max(__ldg(a.plen + a.row[i]), 0), b0) : b0;
    const int first = par == 1 ? 0 : grp, step = par;   // tiles of this group
    int eq = 0;
    // the row, and its products with Rf, into the operand tiles
    const uint32_t qt = sb + kTcQ + grp * 32768, qx = sb + kTcQx + grp * 4096;
    if (first < n) {
      if (any) {
        const int64_t at = (int64_t)(a.tok0[i] + (real ? tok : 0)) * a.qs + (u.h * a.hq + (real ? j : 0)) * 128;
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + at);
        if constexpr (SPLIT) {   // eight lanes to a row's 128 bytes (a lane each its own row: 32 lines per load, here 4)
          uint4 v[8];
          const uint32_t reals = __ballot_sync(0xffffffffu, real);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int row = 4 * k + (lane >> 3);
            const uint4* pr = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + __shfl_sync(0xffffffffu, at, row));
            v[k] = reals >> row & 1 ? __ldg(pr + 8 * hv + (lane & 7)) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) sts128(qt + tile_off<128>(wq * 32 + 4 * k + (lane >> 3), 8 * hv + (lane & 7)), v[k]);
          __syncwarp();
        } else {
        // (compact rather than quick: what runs once per launch is paid in instruction fetches)
#pragma unroll 1
          for (int c0 = 0; c0 < 16; c0 += 8) {
            uint4 v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = real ? __ldg(p + c0 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 8; ++c) sts128(qt + tile_off<128>(tid, c0 + c), v[c]);
          }
        }
        float m = 0.0f;
#pragma unroll 2
        for (int c = SPLIT ? 8 * hv : 0; c < (SPLIT ? 8 * hv + 8 : 16); ++c) {
          const uint4 v = lds128(qt + tile_off<128>(tid, c));
          m = max_abs2<T>(v.x, max_abs2<T>(v.y, max_abs2<T>(v.z, max_abs2<T>(v.w, m))));
        }
        if constexpr (SPLIT) m = fmaxf(m, exchange(2, m));
        eq = m > 0.0f ? range_exp(m, kQueryTop) : 0;
        const float f = copysignf(pow2i(-eq), a.scale_log2);   // a negative scale turns the query's sign instead
        if (SC || f != 1.0f) {
#pragma unroll 2
          for (int c = SPLIT ? 8 * hv : 0; c < (SPLIT ? 8 * hv + 8 : 16); ++c) {
            const uint32_t at = qt + tile_off<128>(tid, c);
            const uint4 v = lds128(at);
            sts128(at, make_uint4(to_half2<T>(v.x, f), to_half2<T>(v.y, f), to_half2<T>(v.z, f), to_half2<T>(v.w, f)));
          }
        }
      }
    }
    if (rank > 0 && unit != rf_unit) {   // the key producers stage every unit's Rf once; a group without tiles here waits too
      tc_wait(bars, &bars->rfull, nrf & 1);
      ++nrf;
      rf_unit = unit;
    }
    if (first < n) {
      if (any && a.blk0_rank > 0) {
        if constexpr (SPLIT) meet();   // the whole query
        const float fr = pow2i(-*reinterpret_cast<volatile int32_t*>(&bars->er));
#pragma unroll 1
        for (int q = SPLIT ? 8 * hv : 0; q < (SPLIT ? 8 * hv + 8 : 16); q += 4) {
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (q < rank) {
#pragma unroll(SPLIT ? 4 : 1)
            for (int c = 0; c < 16; ++c) {
              const uint2 v0 = lds64(qt + tile_off<128>(tid, c)), v1 = lds64(qt + tile_off<128>(tid, c) + 8);
              const uint32_t w[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 q2 = __half22float2(*reinterpret_cast<const __half2*>(&w[e >> 1]));
                const float qv = e & 1 ? q2.y : q2.x;
                const float4 rv = lds_f4(sb + kTcRf + ((c * 8 + e) * rp + q) * 4);
                s[0] = fmaf(qv, rv.x, s[0]);
                s[1] = fmaf(qv, rv.y, s[1]);
                s[2] = fmaf(qv, rv.z, s[2]);
                s[3] = fmaf(qv, rv.w, s[3]);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = q + e < rank ? s[e] * fr : 0.0f;   // (no compressed tokens: all zero)
          sts64(qx + ext_off(tid, q >> 3) + (q & 4) * 2, make_uint2(pack_half2(s[0], s[1]), pack_half2(s[2], s[3])));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->qfull[grp]);
    }
    if (rank > 0 && u.t + 1 == chunk_blocks(a, i)) {   // the last segment that reads this Rf
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->rfree);
    }
    float mref = -INFINITY, l = 0.0f;
    int E = -120;
    [[maybe_unused]] int erv = 0;   // exponent that L of the values was multiplied by, for Rf to lose
    for (int jt = first; jt < n; jt += step) {
      const int tile = it + jt, t0 = (x - u.tile + jt) * kTile;
      tc_wait(bars, &bars->sfull[grp], ns & 1);
      ++ns;
      if (any) {
        tc_fence_after();
        const bool open =
            __all_sync(0xffffffffu, t0 + kTile <= limit && (plen >= b0 || t0 >= b0 || t0 + kTile <= plen));
        // exponents of the tile's groups (one by one below: the loops stay rolled)
        volatile int* ek = bars->ek[tile & 3];
        volatile int* ev = bars->ev[tile & 1];
        int E1 = E;
        if constexpr (SC) {
          tc_wait(bars, &bars->vfull[tile & 1], (tile >> 1) & 1);
          E1 = max(max(E, ev[0]), max(ev[1], ev[2]));
          erv = ev[3];
        }
        float m = -INFINITY;
        uint32_t held[32], mid[16];   // SPLIT: group 2 hv, and half of group 1
        if constexpr (SPLIT) {
          tmem_ld_32x32b_x32(ts + 64 * hv, held);
          tmem_ld_32x32b_x16(ts + 32 + 16 * hv, mid);
          const float sc = score_scale(a.scale_log2, eq + (SC ? ek[2 * hv] : kF16Exp));
          const float sc1 = score_scale(a.scale_log2, eq + (SC ? ek[1] : kF16Exp));
          tmem_ld_wait();
          if (!open) {
            hide(held, seen_bits(t0 + 64 * hv, limit, plen, b0));
            hide(mid, seen_bits(t0 + 32, limit, plen, b0) >> (16 * hv));
          }
          m = fmaxf(max_of(held) * sc, max_of(mid) * sc1);
          tc_fence_before();   // (the weights of one half go over scores of the other)
          m = fmaxf(m, exchange(ns & 1, m));
          tc_fence_after();
        } else {
#pragma unroll 1
          for (int g = 0; g < 3; ++g) {
            tmem_ld_32x32b_x32(ts + 32 * g, held);
            const float sc = score_scale(a.scale_log2, eq + (SC ? ek[g] : kF16Exp));
            tmem_ld_wait();
            if (!open) hide(held, seen_bits(t0 + 32 * g, limit, plen, b0));
            m = fmaxf(m, max_of(held) * sc);
          }
        }
        float fs = 1.0f;
        if (m > mref + 8.0f || (mref == -INFINITY && m > -INFINITY)) {
          fs = mref == -INFINITY ? 0.0f : ex2(mref - m);
          mref = m;
        }
        float fac = fs;
        if constexpr (SC) {
          fac *= pow2i(E - E1);
          E = E1;
        }
        l *= fs;
        const float ref = (mref == -INFINITY ? 0.0f : mref) - kWeightShift;
        float2 sum = make_float2(0.0f, 0.0f);
        auto weigh = [&](auto& s, int g, uint32_t at) {
          constexpr int N = sizeof(s) / 4;
          const float sc = score_scale(a.scale_log2, eq + (SC ? ek[g] : kF16Exp));
          // a group of smaller values than the accumulator's: its weights take the power of two before they are
          // rounded, and their sum gives it back (beyond 2^-60 nothing is left of the values either way)
          const int down = SC ? max(ev[g] - E1, -60) : 0;
          const float rg = SC ? ref - (float)down : ref;
          float2 part = make_float2(0.0f, 0.0f);
          uint32_t p[N / 2];
#pragma unroll
          for (int c = 0; c < N; c += 2) {
            float2 x = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), make_float2(sc, sc), make_float2(-rg, -rg));
            x = make_float2(ex2(x.x), ex2(x.y));
            if constexpr (SC) part = add2(part, x);
            else sum = add2(sum, x);
            p[c / 2] = pack_half2(x.x, x.y);
          }
          if constexpr (SC) {
            const float back = pow2i(-down);
            sum = fma2(part, make_float2(back, back), sum);
          }
          tmem_st(at, p);
        };
        if constexpr (SPLIT) {
          weigh(held, 2 * hv, ts + 32 * hv);
          weigh(mid, 1, ts + 16 + 8 * hv);
        } else {
#pragma unroll 1
          for (int g = 0; g < 3; ++g) {
            tmem_ld_32x32b_x32(ts + 32 * g, held);
            tmem_ld_wait();
            if (!open) hide(held, seen_bits(t0 + 32 * g, limit, plen, b0));
            weigh(held, g, ts + 16 * g);
          }
        }
        l += sum.x + sum.y;
        if (jt != first && __any_sync(0xffffffffu, fac != 1.0f)) {   // O of the tiles before (complete: S came after it)
#pragma unroll 1
          for (int g = SPLIT ? hv : 0; g < 9; g += SPLIT ? 2 : 1) {
            if (g == 8 && a.blk0_rank == 0) break;
            uint32_t o[16];
            tmem_ld_32x32b_x16(to + 16 * g, o);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * fac);
            tmem_st(to + 16 * g, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->pfull[grp]);
    }
    // the segment's rows
    if (first < n) {
      tc_wait(bars, &bars->ofull[grp], nq & 1);
      ++nq;
      tc_fence_after();
    }
    if (any) {
      const bool whole = par == 1 && n == u.tiles;   // no other CTA has a part of this unit
      const int64_t orow = ((int64_t)a.tok0[i] + tok) * a.Hq + u.h * a.hq + j;
      const int64_t prow = par == 1 ? ((int)blockIdx.x * 2 + (u.tile >= begin)) * kRowsUnit + grp * 128 + tid
                                      : (orow - (int64_t)a.tok0[0] * a.Hq) * a.slots + ((int)blockIdx.x - u.tile / a.seg) * 2 + grp;
      float* part = a.part + prow * kPartRow;
      if constexpr (SPLIT) l += exchange(3, l);
      const float up = pow2i(SC ? E : kF16Exp);
      const float mul = whole ? (l > 0.0f ? up * __fdividef(1.0f, l) : (l == 0.0f ? 0.0f : l)) : up;
      if (real && !whole && hv == 0) *reinterpret_cast<float2*>(part) = make_float2(first < n ? mref : -INFINITY, l);
      if (first < n) {
        const float* gv = a.V.rfac + unit * a.nblk_max * 128 * rp;
        const float rscale = SC ? pow2i(-erv) : 1.0f;
        if constexpr (SPLIT) {
          store_rows<T>(a, sb + kTcQ + grp * 32768 + hv * 16384 + wq * 4096, to, gv, rscale, rp, rank, hv, mul, real,
                        whole ? orow * 128 : prow * kPartRow + 4, whole);
        } else {
          if (rank > 0)   // its lines come together, not one after the other
            for (int e = lane; e < 4 * rp; e += 32) asm volatile("prefetch.global.L1 [%0];" ::"l"(gv + e * 32));
#pragma unroll 1
          for (int g = 0; g < 16; ++g) {
            uint32_t o[8];
            tmem_ld_32x32b_x8(to + 8 * g, o);
            tmem_ld_wait();
            float v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = __uint_as_float(o[c]);
#pragma unroll 1
            for (int q = 0; q < rank; q += 4) {   // + (P L) Rf^T
              uint32_t wl[4];
              tmem_ld_32x32b_x4(to + 128 + q, wl);
              float4 rv[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) rv[c] = __ldg(reinterpret_cast<const float4*>(gv + (8 * g + c) * rp + q));
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                if (q + 4 > rank) rv[c] = clip4(rv[c], rank - q);
                if constexpr (SC) rv[c] = scale4(rv[c], rscale);
                v[c] = fmaf(__uint_as_float(wl[0]), rv[c].x, v[c]);
                v[c] = fmaf(q + 1 < rank ? __uint_as_float(wl[1]) : 0.0f, rv[c].y, v[c]);
                v[c] = fmaf(q + 2 < rank ? __uint_as_float(wl[2]) : 0.0f, rv[c].z, v[c]);
                v[c] = fmaf(q + 3 < rank ? __uint_as_float(wl[3]) : 0.0f, rv[c].w, v[c]);
              }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] *= mul;
            if (real) {
              if (!whole || a.out_dtype == GEAR_F32) {
                float4* p = reinterpret_cast<float4*>(whole ? reinterpret_cast<float*>(a.out) + orow * 128 : part + 4) + 2 * g;
                p[0] = make_float4(v[0], v[1], v[2], v[3]);
                p[1] = make_float4(v[4], v[5], v[6], v[7]);
              } else {
                uint32_t w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  if constexpr (SC) {
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * c], v[2 * c + 1]);
                    w[c] = *reinterpret_cast<const uint32_t*>(&b2);
                  } else {
                    w[c] = pack_half2(v[2 * c], v[2 * c + 1]);
                  }
                }
                reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + orow * 128)[g] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    it += n;
    x = x1;
  }
  if (threadIdx.x == 0) {   // for chunk_join
    const bool shared = u.tile >= begin && u.tile < end && u.tile + u.tiles > end;
    int4* p = reinterpret_cast<int4*>(a.join + blockIdx.x * 8);
    p[0] = make_int4(u.i, u.h, u.t, u.tile);
    p[1] = make_int4(shared ? u.tiles : 0, 0, 0, 0);
  }
}

// ------------------------------------------------------------------ products
// One lane of the warp (the same one in every call of a converged warp).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Run by a whole warp, so that descriptors are uniform values; one lane issues.
// Items of a segment: (row tile i % 2, key tile i / 2) with paired row tiles, key tile i
// (accumulator i % 2) otherwise. Scores run two items ahead of the values, so that the
// tensor pipe has work while a softmax group makes its weights; the products of one
// thread run in the order of issue, so that scores may overwrite weights just read.
template <int PAR>
__device__ __forceinline__ void mma_role(const ChunkArgs& a, TcBars* bars, uint8_t* smem) {
  constexpr uint32_t kIdS = idesc_f16(128, kTile, false, false, false);
  const bool ext = a.blk0_rank > 0;   // the low-rank columns
  const uint32_t kIdO = ext ? idesc_f16(128, 144, false, false, true) : idesc_f16(128, 128, false, false, true);
  const int total = a.tile0[a.nseq], end = min(total, (int)(blockIdx.x + 1) * a.seg);
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0), sb = smem_u32(smem);
  const bool pair = (PAR ? PAR : a.par) == 1;
  int it = 0, nseg0 = 0, nseg1 = 0, np0 = 0, np1 = 0;
  const int begin = blockIdx.x * a.seg;
  ChunkUnit u;
  for (int x = begin; x < end;) {
    u = x == begin ? chunk_find(a, x) : chunk_next(a, u);
    x = max(x, u.tile);
    if (x >= end) break;
    const int n = min(end, u.tile + u.tiles) - x, items = pair ? 2 * n : n;
#pragma unroll 1
    for (int i = -2; i < items; ++i) {
      if (i >= 0) {   // O += P V
        const int s = i & 1, tile = it + (pair ? i >> 1 : i);
        if (!pair || s == 0) tc_wait(bars, &bars->vfull[tile & 1], (tile >> 1) & 1);
        const int np = s ? np1 : np0;
        tc_wait(bars, &bars->pfull[s], np & 1);
        if (s) ++np1;
        else ++np0;
        tc_fence_after();
        const uint64_t vd = smem_desc_sw128(sb + kTcV + (tile & 1) * 3 * kTcHalf, kTcHalf, 1024);
        const uint32_t d = tmem + kTmO + s * kTmOCols, p = tmem + s * kTile;
        const uint32_t keep = i >= 2;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc_mma_f16_ts(d, p + kk * 8, vd + kk * (2048 >> 4), kIdO, kk > 0 ? 1 : keep);
          if (i + 2 >= items) tc_commit(&bars->ofull[s]);
          if (!pair || s == 1) tc_commit(&bars->vempty[tile & 1]);
        }
        __syncwarp();
      }
      if (i + 2 < items) {   // S = Q K^T
        const int s = i & 1, tile = it + (pair ? (i + 2) >> 1 : i + 2);
        if (i < 0) {
          const int ns = s ? nseg1 : nseg0;
          tc_wait(bars, &bars->qfull[s], ns & 1);
          if (s) ++nseg1;
          else ++nseg0;
        }
        if (!pair || s == 0) tc_wait(bars, &bars->kfull[tile & 1], (tile >> 1) & 1);
        tc_fence_after();
        const uint64_t qd = smem_desc_sw128(sb + kTcQ + s * 32768, 16, 1024);
        const uint64_t kd = smem_desc_sw128(sb + kTcK + (tile & 1) * 2 * kTcHalf, 16, 1024);
        const uint64_t qe = smem_desc_ext(sb + kTcQx + s * 4096), ke = smem_desc_ext(sb + kTcKx + (tile & 1) * (kTile * 32));
        const uint32_t d = tmem + s * kTile;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_f16(d, qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), kd + (((kk >> 2) * kTcHalf + (kk & 3) * 32) >> 4),
                       kIdS, kk > 0);
          if (ext) tc_mma_f16(d, qe, ke, kIdS, 1);
          tc_commit(&bars->sfull[s]);
          if (!pair || s == 1) tc_commit(&bars->kempty[tile & 1]);
        }
        __syncwarp();
      }
    }
    it += n;
    x += n;
  }
}

// Barriers and tensor memory; `producers` warps complete a K tile, as many a V tile,
// `stagers` a unit's Rf, rows32 a softmax group's row tile.
__device__ __forceinline__ void tc_begin(const ChunkArgs& a, TcBars* bars, int producers, int stagers, int rows32, bool alloc_warp) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->kfull[s], producers);
      mbar_init(&bars->vfull[s], producers);
      mbar_init(&bars->kempty[s], 1);
      mbar_init(&bars->vempty[s], 1);
      mbar_init(&bars->qfull[s], rows32);
      mbar_init(&bars->sfull[s], 1);
      mbar_init(&bars->pfull[s], rows32);
      mbar_init(&bars->ofull[s], 1);
    }
    mbar_init(&bars->rfull, stagers);
    mbar_init(&bars->rfree, 2 * rows32);
    bars->dead = 0;
    bars->status = a.status;
    fence_mbarrier_init();
  }
  if (alloc_warp) tmem_alloc(&bars->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}
__device__ __forceinline__ void tc_end(TcBars* bars, bool alloc_warp) {
  __syncwarp();
  tc_fence_before();
  __syncthreads();   // the softmax groups have waited for every product
  tc_fence_after();
  if (alloc_warp) tmem_dealloc(bars->tmem, 512);
}

// SMALL (units of at most 32 query rows): one warp of each softmax group has rows, and the
// other three rebuild tiles too: twelve producers in two sets.
template <typename T, int BITS, bool KC, bool SMALL>
__global__ void __launch_bounds__(kTcThreads, 1) chunk_tc(const __grid_constant__ ChunkArgs a) {
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = align_smem_1024(raw_smem);
  TcBars* bars = reinterpret_cast<TcBars*>(smem + kTcBars);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (broadcast: uniform)
  constexpr int kSets = SMALL ? 2 : 1;
  tc_begin(a, bars, 3, 3 * kSets, SMALL ? 1 : 4, warp == 14);
  const bool rows = SMALL ? warp == 0 || warp == 4 : warp < 8;
  if constexpr (!SMALL) {
    if (warp < 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kProdRegs));
  }
  if (rows) {
    softmax_role<T, false, SMALL ? 2 : 0>(a, bars, smem, warp >> 2, 0);
  } else if (warp < 14) {
    // producer p of (set, tensor, group)
    const int p = SMALL ? (warp < 4 ? warp - 1 : warp - 2) : warp - 8;
    const bool isk = p / 3 % 2 == 0;
    const uint32_t sb = smem_u32(smem);
    Producer<T, BITS, KC, kSets> w{a, isk, bars,
                                   sb + (isk ? kTcK : kTcV), (isk ? 2 : 3) * kTcHalf,
                                   sb + (isk ? kTcKx : kTcV), isk ? kTile * 32 : 3 * kTcHalf,
                                   sb + kTcRf + (isk ? 0 : kTcRfBytes), p % 3, lane, (lane >> 2) ^ (lane & 2), lane & 3, p / 6};
    w.pu = bars->pu[p];
    w.run();
  } else if (warp == 14) {
    mma_role<SMALL ? 2 : 0>(a, bars, smem);
  }
  tc_end(bars, warp == 14);
}

// Attention over tiles that chunk_rebuild has made: the same softmax groups and products,
// fed by bulk copies (warps 0-7 and 8-15: halves of the rows of both groups; warp 16: keys,
// and Rf for the queries; warp 17: values; warp 18 issues the products).
constexpr int kAttendThreads = 608;

template <typename T>
__device__ __forceinline__ void fetch_role(const ChunkArgs& a, TcBars* bars, uint8_t* smem, bool isk) {
  constexpr bool SC = !std::is_same<T, __half>::value;
  const int lane = lane_id(), rp = rpad_of(a.r_max);
  const int total = a.tile0[a.nseq], end = min(total, (int)(blockIdx.x + 1) * a.seg);
  const uint32_t sb = smem_u32(smem), rf = sb + kTcRf;
  uint64_t* full = isk ? bars->kfull : bars->vfull;
  uint64_t* empty = isk ? bars->kempty : bars->vempty;
  int it = 0, staged = 0;
  int64_t unit = -1;
  const int begin = blockIdx.x * a.seg;
  ChunkUnit u;
  for (int x = begin; x < end;) {
    u = x == begin ? chunk_find(a, x) : chunk_next(a, u);
    x = max(x, u.tile);
    if (x >= end) break;
    const int x1 = min(end, u.tile + u.tiles);
    const int64_t now = (int64_t)a.row[u.i] * a.H + u.h;
    if (isk && now != unit && a.ncomp[u.i] > 0 && a.blk0_rank > 0) {
      if (staged > 0) tc_wait(bars, &bars->rfree, (staged - 1) & 1);   // the softmax groups have read the last one
      ++staged;
      const int er = rf_to_smem(a.K.rfac + now * a.nblk_max * 128 * rp, rp, a.blk0_rank, rf, true);
      if (lane == 0) *reinterpret_cast<volatile int32_t*>(&bars->er) = er;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->rfull);
    }
    unit = now;
    if (lane == 0) {
      const uint8_t* src = a.img + (int64_t)(a.img0[u.i] + u.h * ((a.img0[u.i + 1] - a.img0[u.i]) / a.H) + x - u.tile) * kImgBytes;
      const uint32_t l_bytes = a.blk0_rank > 0 ? (isk ? kTile * 32 : kTcHalf) : 0;
#pragma unroll 1
      for (int k = 0; k < x1 - x; ++k, src += kImgBytes) {
        const int tile = it + k, st = tile & 1;
        tc_wait(bars, &empty[st], ((tile >> 1) & 1) ^ 1);
        mbar_arrive_expect_tx(&full[st], 2 * kTcHalf + l_bytes + (SC ? 16 : 0));
        if (isk) {
          bulk_load(sb + kTcK + st * 2 * kTcHalf, src, 2 * kTcHalf, &full[st]);
          if (l_bytes) bulk_load(sb + kTcKx + st * (kTile * 32), src + 2 * kTcHalf, l_bytes, &full[st]);
        } else {
          bulk_load(sb + kTcV + st * 3 * kTcHalf, src + kImgV, 2 * kTcHalf + l_bytes, &full[st]);
        }
        if (SC) bulk_load(smem_u32(isk ? bars->ek[tile & 3] : bars->ev[st]), src + kImgE + (isk ? 0 : 16), 16, &full[st]);
      }
    }
    __syncwarp();
    it += x1 - x;
    x = x1;
  }
}

template <typename T>
__global__ void __launch_bounds__(kAttendThreads, 1) chunk_attend(const __grid_constant__ ChunkArgs a) {
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = align_smem_1024(raw_smem);
  TcBars* bars = reinterpret_cast<TcBars*>(smem + kTcBars);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (broadcast: uniform)
  tc_begin(a, bars, 1, 1, 8, warp == 18);
  if (warp < 16) softmax_role<T, true, 1>(a, bars, smem, (warp >> 2) & 1, warp >> 3);
  else if (warp < 18) fetch_role<T>(a, bars, smem, warp == 16);
  else mma_role<1>(a, bars, smem);
  tc_end(bars, warp == 18);
}

// Rebuilds every key and value tile of the launch's units once, for units whose tiles many
// row blocks read (192 threads: three warps of keys, three of values).
template <typename T, int BITS, bool KC>
__global__ void __launch_bounds__(192, 2) chunk_rebuild(const __grid_constant__ ChunkArgs a) {
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = align_smem_1024(raw_smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (broadcast: uniform)
  const bool isk = warp < 3;
  const uint32_t sb = smem_u32(smem);
  int32_t(*pu)[8] = reinterpret_cast<int32_t(*)[8]>(smem + kImgE + 2 * kTcRfBytes);
  Producer<T, BITS, KC> p{a, isk, nullptr,
                          sb + (isk ? 0 : kImgV), 0,
                          sb + (isk ? 2 * kTcHalf : kImgV), 0,
                          sb + kImgE + (isk ? 0 : kTcRfBytes), warp - (isk ? 0 : 3), lane, (lane >> 2) ^ (lane & 2), lane & 3, 0};
  p.pu = pu[warp];
  const int total = a.img0[a.nseq], per = (total + gridDim.x - 1) / gridDim.x, x = blockIdx.x * per;
  p.run_images(x, min(total, x + per));
}

template <typename T, int BITS, bool KC, bool SMALL>
static cudaError_t chunk_tc_go(const ChunkArgs& a, cudaStream_t st) {
  static std::atomic<int> slots[kMaxDevices];
  cudaError_t e = ensure_smem_limit(chunk_tc<T, BITS, KC, SMALL>, kTcSmem, slots);
  if (e != cudaSuccess) return e;
  chunk_tc<T, BITS, KC, SMALL><<<a.ctas, kTcThreads, kTcSmem, st>>>(a);
  return cudaGetLastError();
}

// Rebuilds first, then attends.
template <typename T, int BITS, bool KC>
static cudaError_t chunk_two_go(const ChunkArgs& a, cudaStream_t st) {
  static std::atomic<int> slots[kMaxDevices], slots2[kMaxDevices];
  cudaError_t e = ensure_smem_limit(chunk_rebuild<T, BITS, KC>, kImgSmem, slots);
  if (e == cudaSuccess) e = ensure_smem_limit(chunk_attend<T>, kTcSmem, slots2);
  if (e != cudaSuccess) return e;
  const int tiles = a.img0[a.nseq], most = 2 * a.sms;
  chunk_rebuild<T, BITS, KC><<<tiles < most ? tiles : most, 192, kImgSmem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  chunk_attend<T><<<a.ctas, kAttendThreads, kTcSmem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int BITS, bool KC>
static cudaError_t chunk_tc_bits(const ChunkArgs& a, cudaStream_t st) {
  if (a.img) return chunk_two_go<T, BITS, KC>(a, st);
  return a.small ? chunk_tc_go<T, BITS, KC, true>(a, st) : chunk_tc_go<T, BITS, KC, false>(a, st);
}

template <typename T, bool KC>
static cudaError_t chunk_tc_dispatch(const ChunkArgs& a, cudaStream_t st) {
  if (a.bits == 2) return chunk_tc_bits<T, 2, KC>(a, st);
  if (a.bits == 4) return chunk_tc_bits<T, 4, KC>(a, st);
  return chunk_tc_bits<T, 8, KC>(a, st);
}

}  // namespace gear
