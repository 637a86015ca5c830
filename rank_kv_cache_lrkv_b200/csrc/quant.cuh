// The full-rank cache held in 8 bits (lrkv_quant_cache): layout, code
// arithmetic and argument blocks shared by its kernels.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace lrkv {

constexpr int kQBlock = LRKV_PAGE_TOKENS;            // tokens per block and page
constexpr int kQTail = LRKV_QUANT_TAIL;              // slots of the bf16 tail ring
constexpr int kQSide = kQBlock * kHeadDim;           // code bytes of one side of a page
constexpr int kQSlab = LRKV_QUANT_SLAB_BYTES;        // one (page, KV head)
constexpr int kErrCapacity = 3;

// What every kernel needs of the cache.
struct QuantView {
  int B, H, maxp, num_pages, e4m3;
  uint8_t* pages;
  const int* bt;
  __nv_bfloat16* tail;
  int *seq_len, *counter, *error;
};

__device__ __forceinline__ void quant_error(const QuantView& c, int code) {
  atomicCAS(c.error, 0, code);
}
// Tokens of sequence b (seq_len is the caller's to set back: kept in range).
__device__ __forceinline__ int quant_len(const QuantView& c, int b) {
  const int L = c.seq_len[b];
  const long long cap = (long long)c.maxp * kQBlock;
  return L < 0 ? 0 : (L > cap ? (int)cap : L);
}
// Slab of block j of (b, h); nullptr when its page is out of range.
__device__ __forceinline__ uint8_t* quant_slab(const QuantView& c, int b, int h, int j) {
  const int page = c.bt[(size_t)b * c.maxp + j];
  if (page < 0 || page >= c.num_pages) return nullptr;
  return c.pages + ((size_t)page * c.H + h) * kQSlab;
}
// Brings bytes (a multiple of 16, from a 16-byte boundary) into L2.
__device__ __forceinline__ void l2_prefetch(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// Row of token t in the tail (side 0: keys, 1: values).
__device__ __forceinline__ __nv_bfloat16* quant_tail(const QuantView& c, int b, int h, int side,
                                                     int t) {
  return c.tail + ((((size_t)b * c.H + h) * 2 + side) * kQTail + t % kQTail) * kHeadDim;
}
// Byte of 16-byte chunk ch of token t in a slab's key codes.
__host__ __device__ __forceinline__ int quant_k_chunk(int t, int ch) {
  return t * kHeadDim + ((ch ^ ((t & 1) << 2)) << 4);
}

__device__ __forceinline__ float or_zero(float x) { return x == -INFINITY ? 0.f : x; }
// a + b on two fp32 lanes at once.
__device__ __forceinline__ float2 add2(const float2 a, const float2 b) {
  unsigned long long dd, aa, bb;
  memcpy(&aa, &a, 8); memcpy(&bb, &b, 8);
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(dd) : "l"(aa), "l"(bb));
  float2 d;
  memcpy(&d, &dd, 8);
  return d;
}

// Value of a stored byte.
template <bool kE4M3>
__device__ __forceinline__ float quant_value(uint32_t byte) {
  if constexpr (kE4M3) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(h)
        : "r"(byte & 0xffu));
    float f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h));
    return f;
  } else {
    return (float)((int)(byte & 0xffu) - 128);
  }
}

// Four stored bytes (one word, lowest byte first) -> two fp16 pairs, exact:
// whole numbers to 127 and e4m3 values (3 mantissa bits, 2^-9 .. 448) are all
// fp16 numbers.  int8: a byte u under the exponent byte 0x64 is 1024 + u;
// taking 1152 away leaves u - 128.
template <bool kE4M3>
__device__ __forceinline__ void quant_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140);
    const uint32_t b = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  }
}

// Bounded mbarrier wait of the attention kernels, which also gives up once the
// CTA has failed.  Kept small: unrolled polls at some twenty places made a
// kernel of 228 KB, and every role waited for its instructions.
__device__ __forceinline__ bool quant_wait(uint64_t* bar, uint32_t parity, volatile int* fail) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (i % 64 == 0) {
      if (*fail) return false;
      if (global_ns() - t0 > 2000000000ull) {
        *fail = 1;
        return false;
      }
    }
  }
}
// The same for a whole warp: every lane looks once, lane 0 goes on waiting.
__device__ __forceinline__ bool quant_wait_warp(uint64_t* bar, uint32_t parity, volatile int* fail,
                                                int lane) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  int ok = 1;
  if (lane == 0) ok = quant_wait(bar, parity, fail) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The slabs last asked for, one a stage of the ring, have landed (or two seconds
// passed): a CTA does not end before its copies, whoever gave up on one.
__device__ __forceinline__ void quant_drain(uint64_t* bars, int issued, int stages) {
  const uint64_t t0 = global_ns();
  for (int k = max(0, issued - stages); k < issued; ++k)
    while (!mbar_try_wait(&bars[k % stages], (k / stages) & 1) && global_ns() - t0 < 2000000000ull) {
    }
}

// Launch arguments of the append, read and attention kernels.
struct QuantAppendArgs {
  QuantView c;
  const __nv_bfloat16 *k, *v;
  int n;
  const int* n_new;
  long long ss, hs, ts;
};
struct QuantReadArgs {
  QuantView c;
  const int* first;
  int n;
  void *k, *v;
  long long ss, hs, ts;
};
struct QuantAttnArgs {
  QuantView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  int Hq, G, n;
  const int* n_q;
  long long qs, qh, qt, os, oh, ot;
  float scale;
  void* ws;
  uint32_t gmul, gshift;  // division by G (group_division)
};
// n / G for 0 <= n < 2^31: with s = ceil(log2 G), mul = floor(2^(31+s) / G) + 1
// exceeds 2^(31+s) / G by at most 1, so n mul / 2^(31+s) exceeds n / G by at most
// n / 2^(31+s) < 1 / G (Granlund and Montgomery, 1994).  mul 0: G is 1.
__device__ __forceinline__ int div_group(const QuantAttnArgs& a, int n) {
  return a.gmul ? (int)(__umulhi((uint32_t)n, a.gmul) >> a.gshift) : n;
}

// Queries of sequence b in this call.
__device__ __forceinline__ int quant_queries(const QuantAttnArgs& a, int b) {
  if (!a.n_q) return a.n;
  const int x = a.n_q[b];
  return x < 0 ? 0 : (x < a.n ? x : a.n);
}

int quant_append_launch(const QuantAppendArgs& a, cudaStream_t st);
int quant_read_launch(const QuantReadArgs& a, int dtype, cudaStream_t st);
size_t quant_attn_workspace(int B, int H, int Hq, int n);
size_t quant_prefill_workspace(int C);
int quant_few_launch(const QuantAttnArgs& a, const DevInfo& info, cudaStream_t st);
int quant_prefill_launch(const QuantAttnArgs& a, const DevInfo& info, cudaStream_t st);
int quant_attn_launch(const QuantAttnArgs& a, cudaStream_t st);

}  // namespace lrkv
