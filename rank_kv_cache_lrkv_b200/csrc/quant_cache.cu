// Writing the 8-bit full-rank cache and reading it back.
//
// Append: a = max |x| over the 64 x 128 values of a block, s = a / M, code =
// rne(M x / a), M = 127 (whole numbers) or 448 (e4m3).  The codes are those
// of exact arithmetic, without a division per value:
//  * y = x * (M / a) in fp32 is off by at most 2^-22.9 of itself;
//  * with x = X 2^p, a = A 2^r (X, A whole, below 256, p <= r) the quotient Q
//    = M x / a is either a midpoint of two codes or at least 2^-16 of itself
//    away from every midpoint.  int8, midpoint m / 2 (m odd): Q - m / 2 =
//    (254 X 2^p - m A 2^r) / (2 A 2^r), a whole number of 2^p / (2 A 2^r) =
//    Q / (254 X).  e4m3, midpoint m 2^t (m < 32): the same way at least
//    Q / (7 X) or Q / (m A);
//  * so y rounded to 19 bits (which moves it by at most 2^-19) is the
//    midpoint itself where Q is one, and lies on Q's side of it otherwise.
#include "quant.cuh"

namespace lrkv {

namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t abs_max8(uint32_t m, const uint4& w) {
  return abs_max2(abs_max2(abs_max2(abs_max2(m, w.x), w.y), w.z), w.w);
}

// x r rounded to 19 bits (r = M / a): Veltkamp's splitting, 24 - 5 bits.
__device__ __forceinline__ float quant_scaled(float x, float r) {
  const float y = __fmul_rn(x, r), z = __fmul_rn(y, 33.f);
  return __fsub_rn(z, __fsub_rn(z, y));
}
// Two values' stored bytes (low byte: lo).
template <bool kE4M3>
__device__ __forceinline__ uint32_t quant_code2(float lo, float hi, float r) {
  const float x = quant_scaled(lo, r), y = quant_scaled(hi, r);
  if constexpr (kE4M3) {
    uint32_t w;
    asm("{\n\t.reg .b16 p;\n\tcvt.rn.satfinite.e4m3x2.f32 p, %1, %2;\n\tcvt.u32.u16 %0, p;\n\t}"
        : "=r"(w)
        : "f"(y), "f"(x));
    return w;
  } else {
    return (uint32_t)(__float2int_rn(x) + 128) | ((uint32_t)(__float2int_rn(y) + 128) << 8);
  }
}
// The 8 bytes of 8 values.
template <bool kE4M3>
__device__ __forceinline__ uint2 quant_code8(const uint4& w, float r) {
  const uint32_t p = quant_code2<kE4M3>(bf_lo(w.x), bf_hi(w.x), r);
  const uint32_t q = quant_code2<kE4M3>(bf_lo(w.y), bf_hi(w.y), r);
  const uint32_t u = quant_code2<kE4M3>(bf_lo(w.z), bf_hi(w.z), r);
  const uint32_t s = quant_code2<kE4M3>(bf_lo(w.w), bf_hi(w.w), r);
  return make_uint2(p | (q << 16), u | (s << 16));
}

// 4 x 4 byte transpose: word i of the result holds byte i of a, b, c, d.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                           uint32_t (&r)[4]) {
  const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
  const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
  r[0] = __byte_perm(ab0, cd0, 0x5410);
  r[1] = __byte_perm(ab0, cd0, 0x7632);
  r[2] = __byte_perm(ab1, cd1, 0x5410);
  r[3] = __byte_perm(ab1, cd1, 0x7632);
}

// One CTA per (block that the call touches, KV head, sequence).
//  * A block that becomes full: thread (token, 16-byte chunk) holds the key
//    rows, thread (4 tokens, chunk) the value rows (so that its codes
//    transpose in registers); maximum over the CTA; codes into shared memory
//    in the slab's layout; one bulk store.
//  * The rows of the call that the tail keeps (the open block and the one
//    before it) are copied by the CTA of the first block, after it has read
//    the open block's old rows: they may take those rows' slots.
// The last CTA of a sequence to finish advances seq_len.
template <bool kE4M3>
__global__ void __launch_bounds__(kAppendThreads) quant_append_kernel(QuantAppendArgs a) {
  __shared__ __align__(128) uint8_t slab[kQSlab];
  __shared__ uint32_t part[2][kAppendThreads / 32];
  pdl_trigger();
  pdl_wait();
  const QuantView& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L0 = quant_len(c, b);
  int n = a.n;
  if (a.n_new) n = max(0, min(n, a.n_new[b]));
  const long long cap = (long long)c.maxp * kQBlock;
  const bool over = L0 + (long long)n > cap;
  if (over) n = (int)(cap - L0);
  const int L1 = L0 + n;
  const int j = L0 / kQBlock + blockIdx.x;
  const __nv_bfloat16* krow = a.k + b * a.ss + h * a.hs;
  const __nv_bfloat16* vrow = a.v + b * a.ss + h * a.hs;
  // row of token t: the tail's for tokens of earlier calls
  auto src = [&](int side, int t) {
    return t < L0 ? quant_tail(c, b, h, side, t)
                  : (side ? vrow : krow) + (long long)(t - L0) * a.ts;
  };
  const bool full = n > 0 && (long long)(j + 1) * kQBlock <= L1;
  uint8_t* out = nullptr;
  if (full) {
    out = quant_slab(c, b, h, j);
    if (!out && tid == 0) quant_error(c, kErrBadPage);
  }
  if (over && tid == 0) quant_error(c, kErrCapacity);

  uint4 kx[4], vx[4];
  if (full) {  // uniform over the CTA
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kx[i] = *reinterpret_cast<const uint4*>(src(0, j * kQBlock + (tid >> 4) + 16 * i) + (tid & 15) * 8);
      vx[i] = *reinterpret_cast<const uint4*>(src(1, j * kQBlock + 4 * (tid & 15) + i) + (tid >> 4) * 8);
    }
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mk = abs_max8(mk, kx[i]);
      mv = abs_max8(mv, vx[i]);
    }
    mk = max(mk >> 16, mk & 0xffffu);
    mv = max(mv >> 16, mv & 0xffffu);
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if (lane == 0) {
      part[0][warp] = mk;
      part[1][warp] = mv;
    }
  }
  __syncthreads();
  if (full && out) {
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) {
      mk = max(mk, part[0][w]);
      mv = max(mv, part[1][w]);
    }
    const bool kbad = mk >= 0x7f80u, vbad = mv >= 0x7f80u;  // an infinity or a NaN
    const float top = kE4M3 ? 448.f : 127.f, least = 7.888609052210118e-31f;  // 2^-100
    const float ak = fmaxf(__uint_as_float(mk << 16), least);
    const float av = fmaxf(__uint_as_float(mv << 16), least);
    const float rk = __fdiv_rn(top, ak), rv = __fdiv_rn(top, av);
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = (tid >> 4) + 16 * i, d8 = tid & 15;
      *reinterpret_cast<uint2*>(slab + quant_k_chunk(t, d8 >> 1) + (d8 & 1) * 8) =
          quant_code8<kE4M3>(kbad ? zero : kx[i], kbad ? 1.f : rk);
    }
    uint2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = quant_code8<kE4M3>(vbad ? zero : vx[i], vbad ? 1.f : rv);
    uint32_t lo[4], hi[4];
    transpose4(w[0].x, w[1].x, w[2].x, w[3].x, lo);
    transpose4(w[0].y, w[1].y, w[2].y, w[3].y, hi);
    uint32_t* vs = reinterpret_cast<uint32_t*>(slab + kQSide);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      vs[((tid >> 4) * 8 + i) * (kQBlock / 4) + (tid & 15)] = lo[i];
      vs[((tid >> 4) * 8 + 4 + i) * (kQBlock / 4) + (tid & 15)] = hi[i];
    }
    if (tid < 8) {
      const float nan = __uint_as_float(0x7fc00000u);
      const float s = tid == 0 ? (kbad ? nan : __fdiv_rn(ak, top))
                               : tid == 1 ? (vbad ? nan : __fdiv_rn(av, top)) : 0.f;
      reinterpret_cast<float*>(slab + 2 * kQSide)[tid] = s;
    }
    proxy_fence_smem();
  }
  if (blockIdx.x == 0 && n > 0) {
    // the call's rows that the tail keeps: 16 threads a row
    const int t0 = max(L0, (L1 / kQBlock - 1) * kQBlock);
    for (int i = tid; i < (L1 - t0) * 32; i += kAppendThreads) {
      const int t = t0 + (i >> 5), side = (i >> 4) & 1, e = (i & 15) * 8;
      *reinterpret_cast<uint4*>(quant_tail(c, b, h, side, t) + e) =
          *reinterpret_cast<const uint4*>((side ? vrow : krow) + (long long)(t - L0) * a.ts + e);
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (full && out) {
      bulk_s2g(out, slab, kQSlab);
      bulk_commit();
    }
    // the last CTA of the sequence: every other has read seq_len
    __threadfence();
    const int last = (int)(gridDim.x * gridDim.y) - 1;
    if (atomicAdd(&c.counter[b], 1) == last) {
      c.seq_len[b] = L1;
      c.counter[b] = 0;
    }
    if (full && out) bulk_wait<0>();
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                 pack_bf16x2(f[6], f[7]));
}

// One CTA per (block of the range, KV head, sequence); threads as in the
// append: keys by (token, chunk), values by (4 tokens, chunk).
template <bool kE4M3, typename T>
__global__ void __launch_bounds__(kAppendThreads) quant_read_kernel(QuantReadArgs a) {
  pdl_trigger();
  pdl_wait();
  const QuantView& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int L = quant_len(c, b);
  const long long f0 = a.first ? a.first[b] : 0;
  const long long lo = max(0ll, f0), hi = min((long long)L, f0 + a.n);
  const long long j = lo / kQBlock + blockIdx.x;
  if (j * kQBlock >= hi) return;
  const int base = (int)j * kQBlock;
  T* krow = static_cast<T*>(a.k) + b * a.ss + h * a.hs;
  T* vrow = static_cast<T*>(a.v) + b * a.ss + h * a.hs;
  auto wanted = [&](int t) { return t >= lo && t < hi; };
  if (base + kQBlock > L) {  // the open block
    for (int i = tid; i < kQBlock * 32; i += kAppendThreads) {
      const int t = base + (i >> 5), side = (i >> 4) & 1, e = (i & 15) * 8;
      if (!wanted(t)) continue;
      float f[8];
      unpack_chunk<__nv_bfloat16>(
          *reinterpret_cast<const uint4*>(quant_tail(c, b, h, side, t) + e), f);
      store8<T>((side ? vrow : krow) + (t - f0) * a.ts + e, f);
    }
    return;
  }
  const uint8_t* slab = quant_slab(c, b, h, (int)j);
  if (!slab && tid == 0) quant_error(c, kErrBadPage);
  float sk = 0.f, sv = 0.f;
  uint2 kw[4];
  uint32_t vw[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) kw[i] = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) vw[i] = 0;
  if (slab) {
    sk = reinterpret_cast<const float*>(slab + 2 * kQSide)[0];
    sv = reinterpret_cast<const float*>(slab + 2 * kQSide)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d8 = tid & 15;
      kw[i] = *reinterpret_cast<const uint2*>(
          slab + quant_k_chunk((tid >> 4) + 16 * i, d8 >> 1) + (d8 & 1) * 8);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      vw[i] = reinterpret_cast<const uint32_t*>(
          slab + kQSide)[((tid >> 4) * 8 + i) * (kQBlock / 4) + (tid & 15)];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = base + (tid >> 4) + 16 * i;
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = quant_value<kE4M3>(kw[i].x >> (8 * e)) * sk;
      f[4 + e] = quant_value<kE4M3>(kw[i].y >> (8 * e)) * sk;
    }
    if (!slab)
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
    if (wanted(t)) store8<T>(krow + (t - f0) * a.ts + (tid & 15) * 8, f);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = base + 4 * (tid & 15) + i;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = slab ? quant_value<kE4M3>(vw[e] >> (8 * i)) * sv : 0.f;
    if (wanted(t)) store8<T>(vrow + (t - f0) * a.ts + (tid >> 4) * 8, f);
  }
}

}  // namespace

int quant_append_launch(const QuantAppendArgs& a, cudaStream_t st) {
  // blocks that n tokens can touch, wherever in a block they start
  const unsigned nb = (unsigned)((a.n + 62ll) / kQBlock + 1);
  const dim3 grid(nb, a.c.H, a.c.B);
  QuantAppendArgs args = a;
  void* p[] = {&args};
  const void* fn = a.c.e4m3 ? (const void*)quant_append_kernel<true>
                            : (const void*)quant_append_kernel<false>;
  return launch_pdl(fn, grid, dim3(kAppendThreads), 0, st, p) == cudaSuccess ? LRKV_OK
                                                                             : LRKV_ERR_CUDA;
}

int quant_read_launch(const QuantReadArgs& a, int dtype, cudaStream_t st) {
  const unsigned nb = (unsigned)((a.n + 62ll) / kQBlock + 1);
  const dim3 grid(nb, a.c.H, a.c.B);
  QuantReadArgs args = a;
  void* p[] = {&args};
  const void* fn;
  if (dtype == LRKV_F32)
    fn = a.c.e4m3 ? (const void*)quant_read_kernel<true, float>
                  : (const void*)quant_read_kernel<false, float>;
  else
    fn = a.c.e4m3 ? (const void*)quant_read_kernel<true, __nv_bfloat16>
                  : (const void*)quant_read_kernel<false, __nv_bfloat16>;
  return launch_pdl(fn, grid, dim3(kAppendThreads), 0, st, p) == cudaSuccess ? LRKV_OK
                                                                             : LRKV_ERR_CUDA;
}

}  // namespace lrkv
