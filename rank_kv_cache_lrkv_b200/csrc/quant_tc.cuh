// What the tensor-core attention kernels of the 8-bit cache share: tcgen05
// with A from TMEM, TMEM loads and stores, the fp16 tiles of a page and their
// making from codes or from the open block, records of cut tiles.
#pragma once
#include "quant.cuh"
#include "tcgen05.cuh"

namespace lrkv {

constexpr int kStepKeys = kQBlock;              // keys of a step: one page
constexpr int kKHalf = kStepKeys * 128;         // 64 dims of a step's keys
constexpr int kTileBytes = 2 * kKHalf;          // a step's keys, or its values [128][64]
constexpr int kTileRows = 256;                  // rows of a record
// References lag by at most 2^kLazy, weights carry 2^kBoostLog (see
// quant_prefill.cu).
constexpr float kLazy = 5.f;
constexpr float kBoostLog = 8.f;

struct alignas(16) StepScales {
  float sk, sv;
  int ok;       // the page's tokens count (kWideStep: weighed by weigh_wide)
};
// The open block's tokens have powers of two of their own (so that no token takes
// bits from others, least of all from those of queries that do not see it): the
// exponents of their values (NaN: one is not finite), then the powers of their keys,
// all bf16 numbers.
constexpr int kTokValues = 2 * kStepKeys, kTokBytes = 2 * kTokValues;

// Workspace: the counters of the few-row kernel (not used here, and left
// alone), a cut per CTA (sequence, head, row and last CTA of the tile that
// begins in it and goes on elsewhere; last CTA -1: none), two records per CTA
// as in quant_decode.cu, of [33][256] float4: (m, l, M' - m, -) of a row, then its
// 128 sums four at a time, rows side by side.
constexpr size_t kPreRecord = (size_t)33 * kTileRows;
__host__ __device__ inline size_t pre_cuts(int C) { return ((size_t)C * 4 + 255) / 256 * 256; }
__host__ __device__ inline size_t pre_records(int C) {
  return pre_cuts(C) + ((size_t)C * 16 + 255) / 256 * 256;
}

// Shared-memory descriptors in halves: the upper one is the same for every
// 128-byte-swizzled K-major tile, the lower one counts 16-byte units, so a
// step within a tile is one addition (one thread issues all products).
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(alo), "r"(blo), "r"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t blo, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(blo), "r"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}
// fp16 A and B, fp32 D, M = 128, both K-major; N = 64 keys or 128 dims.
constexpr uint32_t kIdescS = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescO = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0;
}
#define LRKV_R32(v, o)                                                                          \
  "=r"(v[o + 0]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]),               \
      "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7]), "=r"(v[o + 8]), "=r"(v[o + 9]),           \
      "=r"(v[o + 10]), "=r"(v[o + 11]), "=r"(v[o + 12]), "=r"(v[o + 13]), "=r"(v[o + 14]),      \
      "=r"(v[o + 15]), "=r"(v[o + 16]), "=r"(v[o + 17]), "=r"(v[o + 18]), "=r"(v[o + 19]),      \
      "=r"(v[o + 20]), "=r"(v[o + 21]), "=r"(v[o + 22]), "=r"(v[o + 23]), "=r"(v[o + 24]),      \
      "=r"(v[o + 25]), "=r"(v[o + 26]), "=r"(v[o + 27]), "=r"(v[o + 28]), "=r"(v[o + 29]),      \
      "=r"(v[o + 30]), "=r"(v[o + 31])
// 32 consecutive columns of this thread's lane, no wait.
template <int kOff, int N>
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[N]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : LRKV_R32(v, kOff)
      : "r"(addr));
}
// Wait for this thread's loads; ties 32 of their registers to the wait.
template <int kOff, int N>
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[kOff + i]));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
// 8 consecutive columns of this thread's lane, and the wait for them.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])::
                   "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 codes -> 32 bytes of fp16 at chunks cc, cc + 1 of a swizzled row.
template <bool kE4M3>
__device__ __forceinline__ void put_codes(uint8_t* rowp, int row, int cc, const uint4& w) {
  uint32_t h[8];
  quant_half4<kE4M3>(w.x, h[0], h[1]);
  quant_half4<kE4M3>(w.y, h[2], h[3]);
  quant_half4<kE4M3>(w.z, h[4], h[5]);
  quant_half4<kE4M3>(w.w, h[6], h[7]);
  *reinterpret_cast<uint4*>(rowp + ((cc ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(rowp + (((cc + 1) ^ (row & 7)) << 4)) =
      make_uint4(h[4], h[5], h[6], h[7]);
}

// ---- the open block's bf16 rows as fp16 under a power of two for each row, by
// the 128 threads ct of the converters.  Real functions: once a sequence at most,
// and in line their registers and instructions cost every page (long calls 2 to 8 %).
// Short ones: code that is run through a single time is waited for, 16 bytes an
// instruction (64 rows of values unrolled, 168 prompts of 189 tokens 150 us, so 92).
__device__ __forceinline__ uint32_t abs_max8(const uint4& w) {  // bf16 bits
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                              __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  return max(m >> 16, m & 0xffffu);
}
// Largest |x| (bf16 bits) of row ct / 2 of the block's rows, nt of them.
static __device__ __noinline__ uint32_t open_row_max(const __nv_bfloat16* rows, int nt, int ct) {
  const uint4* src = reinterpret_cast<const uint4*>(rows + (ct >> 1) * kHeadDim) + 8 * (ct & 1);
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = (ct >> 1) < nt ? src[i] : make_uint4(0, 0, 0, 0);
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max(mx, abs_max8(w[i]));
  return max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
}
// Keys (a row's largest finite element becomes 2^14 ..): writes the tile kb and the
// tokens' powers of two.  Thread = (token, half of the dims).
static __device__ __noinline__ void open_keys(const __nv_bfloat16* rows, int nt, uint8_t* kb, int ct,
                                              uint8_t* tok) {
  const int t = ct >> 1, side = ct & 1;
  uint32_t mx = open_row_max(rows, nt, ct);
  if (__any_sync(0xffffffffu, mx >= 0x7f80u)) {  // what is not finite does not count
    mx = 0;
#pragma unroll 1
    for (int i = 0; i < 64 && t < nt; ++i) {
      const uint32_t x = reinterpret_cast<const uint16_t*>(rows)[t * kHeadDim + 64 * side + i] & 0x7fffu;
      if (x < 0x7f80u) mx = max(mx, x);
    }
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  }
  const int byte = max((int)(mx >> 7) - 14, 13);  // 127 - 14 + the exponent, at least -100
  if (side == 0) reinterpret_cast<uint16_t*>(tok + kTokValues)[t] = (uint16_t)(byte << 7);
  const float up = __uint_as_float((uint32_t)(254 - byte) << 23);
  const uint4* src = reinterpret_cast<const uint4*>(rows + t * kHeadDim) + 8 * side;
#pragma unroll 2
  for (int i = 0; i < 8; ++i) {
    const uint4 w = t < nt ? src[i] : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(kb + side * kKHalf + t * 128 + ((i ^ (t & 7)) << 4)) =
        make_uint4(pack_h2(bf_lo(w.x) * up, bf_hi(w.x) * up),
                   pack_h2(bf_lo(w.y) * up, bf_hi(w.y) * up),
                   pack_h2(bf_lo(w.z) * up, bf_hi(w.z) * up),
                   pack_h2(bf_lo(w.w) * up, bf_hi(w.w) * up));
  }
}
// The exponents of the values (a row's largest element becomes 2^7 ..).
__device__ __forceinline__ void open_value_exponents(const __nv_bfloat16* rows, int nt, int ct, uint8_t* tok) {
  const uint32_t mx = open_row_max(rows, nt, ct);
  const float e = mx < 0x7f80u ? (float)(max((int)(mx >> 7) - 127, -100) - 7) : NAN;
  if (!(ct & 1)) reinterpret_cast<uint16_t*>(tok)[ct >> 1] = (uint16_t)(__float_as_uint(e) >> 16);
}
// Eight of the tokens' numbers.
struct Tok8 {
  uint32_t w[4];
  __device__ __forceinline__ explicit Tok8(const uint8_t* p) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    w[0] = t.x;
    w[1] = t.y;
    w[2] = t.z;
    w[3] = t.w;
  }
  __device__ __forceinline__ float operator[](int k) const { return k & 1 ? bf_hi(w[k >> 1]) : bf_lo(w[k >> 1]); }
};
__device__ __forceinline__ float exp2_whole(float x) {  // 2^x, x whole: in the last bits of x + 1.5 2^23 + 127
  return __uint_as_float(__float_as_uint(x + (12582912.f + 127.f)) << 23);
}
// Values, transposed, by all tokens' exponents: writes the tile vb.  Thread = dim; rows
// with a value that is not finite become 0.
static __device__ __noinline__ void open_values(const __nv_bfloat16* rows, int nt, uint8_t* vb, int ct,
                                                const uint8_t* tok) {
  const __nv_bfloat16* vt = rows + ct;
#pragma unroll 1
  for (int cc = 0; cc < 8; ++cc) {
    const Tok8 ev(tok + 16 * cc);
    uint32_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 8 * cc + 2 * q + e;
        const float x = ev[2 * q + e];
        v[e] = t < nt && x == x ? __bfloat162float(vt[t * kHeadDim]) * exp2_whole(-x) : 0.f;
      }
      h[q] = pack_h2(v[0], v[1]);
    }
    *reinterpret_cast<uint4*>(vb + ct * 128 + ((cc ^ (ct & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// ---- the softmax of the open block, and of a step whose exponents are far apart
//
// A row holds m, the largest score rounded down, and M' - m (M' as in
// quant_decode.cu): whole numbers, exact however large the scores are.  The usual
// step weighs with v = 2^(s f - m) and v (2^(m - M') s_v 2^kBoostLog).  That takes two
// things, and a step that lacks either is weighed by weigh_wide (a real function
// over S in TMEM: it is seldom called):
//  * 2^(m - M') s_v small, as v is flushed under 2^-126.  M' is at most kLazy under m +
//    log2 of the value scale where m was found, so with all scales of a part in
//    [2^-35, 2^35] the factor is at most 2^(70 + kLazy + 1 + kBoostLog), and weights
//    under 2^-42 are flushed (half of fp16's smallest step is 2^-25).  The
//    converters mark a step whose scale is above that range, or whose part had one
//    below it (wide_step).
//  * |m| small: s f is not rounded in the fma, but m comes from it rounded, so v is
//    off by 2 to half an ulp of the score, alike for all tokens of a row; from 2^24
//    on a weight could overflow.  m is looked at where M' moves (it cannot move far
//    alone); a warp with such a row has its factors fcol negated for the rest of the
//    part.
constexpr int kWideStep = 2;
constexpr float kWideRef = 1048576.f;
// StepScales::ok of a full block; low: it, or a block of its part before it, was under the range.
__device__ __forceinline__ int wide_step(float sv, bool& low) {
  low |= sv < 2.9103830456733704e-11f;               // 2^-35
  return low || sv > 34359738368.f ? kWideStep : 1;  // 2^35
}
// Weights of the columns of S up to `last` (0 behind it) to TMEM at tP, which may be
// where S is; returns their sum.  c: log2 of what p is multiplied by, beside fv.
static __device__ __noinline__ float weigh_wide(uint32_t tS, uint32_t tP, int columns, float f, int last,
                                                float ref, float c, float fv) {
  float sum = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < columns; k0 += 16) {
    uint32_t s[16], pk[8];
    tmem_ld16(tS + k0, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float w[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float x = __fmul_rn(__uint_as_float(s[2 * e + u]), f) - ref;
        const bool out = k0 + 2 * e + u > last;
        sum += out ? 0.f : ex2_approx(x);
        w[u] = out ? 0.f : fv * ex2_approx(x + c);
      }
      pk[e] = pack_h2(w[0], w[1]);
    }
    tmem_st8(tP + (k0 >> 1), pk);
  }
  return sum;
}
// A row's state, and the open block's step: the columns of S up to `last`, P, O
// (whose last sums `odone` tells of; nullptr: there are none yet).  tok: the
// columns' tokens, fcol: the row's factor.
struct RowState {
  float m, l, dv;
};
static __device__ __noinline__ RowState open_step(RowState r, uint32_t tS, uint32_t tP, uint32_t tO,
                                                  int columns, const uint8_t* tok, float fcol, int last,
                                                  uint64_t* odone, uint32_t parity, volatile int* fail) {
  // scores, back to where S was (masked: -inf); the largest, and the largest score +
  // exponent of the value, from a whole number `at` that follows the scores
  float mn = -INFINITY, vn = -INFINITY, at = or_zero(r.m);
#pragma unroll 1
  for (int k0 = 0; k0 < columns; k0 += 8) {
    uint32_t s[8];
    tmem_ld8(tS + k0, s);
    const Tok8 ev(tok + 2 * k0), kf(tok + kTokValues + 2 * k0);
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = k0 + k > last ? -INFINITY : __fmul_rn(__uint_as_float(s[k]), fcol * kf[k]);
      mn = fmaxf(mn, x[k]);
      s[k] = __float_as_uint(x[k]);
    }
    tmem_st8(tS + k0, s);
    const float to = floorf(mn);
    if (to > -INFINITY) {
      vn += at - to;
      at = to;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) vn = fmaxf(vn, x[k] - at + ev[k]);
  }
  mn = floorf(mn);
  if (mn > r.m + kLazy) {
    const float sh = r.m - mn;
    r.l *= ex2_approx(sh);
    r.dv += sh;
    r.m = mn;
  }
  const float ref = or_zero(r.m);
  vn += at - ref;
  vn = floorf(vn);
  const bool grow = vn > r.dv + kLazy;
  const float cr = grow ? ex2_approx(r.dv - vn) : 1.f;
  if (grow) r.dv = vn;
  if (__any_sync(0xffffffffu, grow) && odone && quant_wait_warp(odone, parity, fail, threadIdx.x & 31)) {
    tc_fence_after();
#pragma unroll 1
    for (int q4 = 0; q4 < 8; ++q4) {
      uint32_t o[16];
      tmem_ld16(tO + 16 * q4, o);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * cr);
      tmem_st16(tO + 16 * q4, o);
    }
  }
  tmem_wait_st();
  const float c = kBoostLog - or_zero(r.dv);
  float sum = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < columns; k0 += 8) {
    uint32_t s[8], pk[4];
    tmem_ld8(tS + k0, s);
    const Tok8 ev(tok + 2 * k0);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float w[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float x = __uint_as_float(s[k + u]) - ref;
        sum += ex2_approx(x);
        // (NaN of a value that is not finite does not reach what is masked)
        w[u] = k0 + k + u > last ? 0.f : ex2_approx(x + (c + ev[k + u]));
      }
      pk[k >> 1] = pack_h2(w[0], w[1]);
    }
    tmem_st4(tP + (k0 >> 1), pk);
  }
  r.l += sum;
  return r;
}

// Parts of cut tiles, folded (quant_prefill.cu); rows: rows of a tile in use.
int quant_merge_launch(const QuantAttnArgs& a, int C, int rows, cudaStream_t st);

}  // namespace lrkv
