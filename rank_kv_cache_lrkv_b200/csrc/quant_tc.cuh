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
constexpr float kLazy = 6.f;
constexpr float kBoostLog = 8.f;

struct StepScales {
  float sk, sv;
  int ok;       // the page's tokens count
  int minbad;   // first open token whose value row is not finite
};

// Workspace: the counters of the few-row kernel (not used here, and left
// alone), a cut per CTA (sequence, head, row and last CTA of the tile that
// begins in it and goes on elsewhere; last CTA -1: none), two records per CTA
// as in quant_decode.cu, of [33][256] float4: (m, l, M', -) of a row, then its
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

// ---- the open block's bf16 rows as fp16 under a power of two, by the 128
// threads ct of the converters.  Real functions: once a sequence at most, and
// in line their registers and instructions cost every page (long calls 2 to 8 %).
// Largest finite |x| (bf16 bits) of the block's nt rows of one side and the
// first row that is not all finite (64: none).  Every warp looks at all of
// them: no barrier among warps that a failed wait may part.
__device__ __forceinline__ uint32_t scan_open(const __nv_bfloat16* rows, int nt, int lane, int& bad) {
  constexpr int kTogether = 8;  // loads on their way at once (fewer, with every
  // element looked at alone: 168 prompts of 189 tokens 100 us against 62)
  const uint4* src = reinterpret_cast<const uint4*>(rows) + lane;
  uint32_t mx = 0;
#pragma unroll 1
  for (int i0 = 0; 2 * i0 < nt; i0 += kTogether) {
    uint4 w[kTogether];
#pragma unroll
    for (int i = 0; i < kTogether; ++i)
      w[i] = 2 * (i0 + i) + (lane >> 4) < nt ? src[32 * (i0 + i)] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      mx = __vmaxu2(mx, __vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu));
      mx = __vmaxu2(mx, __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
    }
  }
  mx = __reduce_max_sync(0xffffffffu, max(mx >> 16, mx & 0xffffu));
  bad = 64;
  if (mx < 0x7f80u) return mx;
  // something is not finite: once more, element by element
  mx = 0;
#pragma unroll 1
  for (int i = lane; i < nt * kHeadDim; i += 32) {
    const uint32_t x = reinterpret_cast<const uint16_t*>(rows)[i] & 0x7fffu;
    if (x < 0x7f80u) mx = max(mx, x); else bad = min(bad, i / kHeadDim);
  }
  bad = (int)__reduce_min_sync(0xffffffffu, (uint32_t)bad);
  return __reduce_max_sync(0xffffffffu, mx);
}
// Keys (rows: the block's first; the largest becomes 2^14 ..): writes the tile
// kb, returns the scale.  Thread = (token, half of the dims).
static __device__ __noinline__ float open_keys(const __nv_bfloat16* rows, int nt, uint8_t* kb, int ct) {
  int bad;
  const int e = max((int)(scan_open(rows, nt, ct & 31, bad) >> 7) - 127, -100);
  const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
  const int tok = ct >> 1, side = ct & 1;
  const uint4* src = reinterpret_cast<const uint4*>(rows + tok * kHeadDim) + 8 * side;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 w = tok < nt ? src[i] : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(kb + side * kKHalf + tok * 128 + ((i ^ (tok & 7)) << 4)) =
        make_uint4(pack_h2(bf_lo(w.x) * up, bf_hi(w.x) * up),
                   pack_h2(bf_lo(w.y) * up, bf_hi(w.y) * up),
                   pack_h2(bf_lo(w.z) * up, bf_hi(w.z) * up),
                   pack_h2(bf_lo(w.w) * up, bf_hi(w.w) * up));
  }
  return __uint_as_float((uint32_t)(127 - 14 + e) << 23);
}
// The scale of the values (the largest becomes 2^7 ..) and the first token
// with one that is not finite (64: none).
static __device__ __noinline__ float2 open_values_scale(const __nv_bfloat16* rows, int nt, int ct) {
  int bad;
  const int e = (int)(scan_open(rows, nt, ct & 31, bad) >> 7) - 127;
  return make_float2(__uint_as_float((uint32_t)(127 - 7 + max(e, -100)) << 23), __int_as_float(bad));
}
// Values, transposed: writes the tile vb.  Thread = dim; values that are not
// finite become 0 (their tokens were reported).
static __device__ __noinline__ void open_values(const __nv_bfloat16* rows, int nt, uint8_t* vb, int ct,
                                            float sv) {
  const __nv_bfloat16* vt = rows + ct;
  const float up = __uint_as_float((254u << 23) - __float_as_uint(sv));  // 1 / sv, a power of two
#pragma unroll 1
  for (int cc = 0; cc < 8; ++cc) {
    uint32_t h[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 8 * cc + 2 * q + e;
        v[e] = t < nt ? __bfloat162float(vt[t * kHeadDim]) * up : 0.f;
        if (!(fabsf(v[e]) < 1e30f)) v[e] = 0.f;
      }
      h[q] = pack_h2(v[0], v[1]);
    }
    *reinterpret_cast<uint4*>(vb + ct * 128 + ((cc ^ (ct & 7)) << 4)) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// Parts of cut tiles, folded (quant_prefill.cu); rows: rows of a tile in use.
int quant_merge_launch(const QuantAttnArgs& a, int C, int rows, cudaStream_t st);

}  // namespace lrkv
