// Writing the 8-bit full-rank cache and reading it back.
//
// Append: a = max |x| over the 64 x 128 values of a block, s = a / M, code =
// rne(M x / a), M = 127 (whole numbers) or 448 (e4m3).  The codes are those
// of exact arithmetic, without a division per value:
//  * M / a is held as r + q, r = M fl(1 / a) and q = (M - r a) fl(1 / a) (the
//    remainder is exact: r a has 32 bits), so y = fl(x r + fl(x q)) is the
//    quotient Q = M x / a off by less than 2^-26 of itself, then rounded once;
//  * with x = X 2^p, a = A 2^e (X, A whole, below 256, p <= e) Q is either a
//    midpoint of two codes or at least 2^-16 of itself away from every one.
//    int8, midpoint m / 2 (m odd): Q - m / 2 = (254 X 2^p - m A 2^e) /
//    (2 A 2^e), a whole number of 2^p / (2 A 2^e) = Q / (254 X).  e4m3,
//    midpoint m 2^t (m < 32): the same way at least Q / (7 X) or Q / (m A);
//  * a midpoint has 8 bits at most, so where Q is one, y is Q; elsewhere y
//    lies on Q's side of it.
#include "quant.cuh"

namespace lrkv {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendCtas = 4;  // resident per SM
constexpr int kAhead = 2;       // blocks in flight per CTA
constexpr int kAppendSmem = kAhead * 4 * kAppendThreads * 16 + 2 * kQSide;

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t abs_max8(uint32_t m, const uint4& w) {
  return abs_max2(abs_max2(abs_max2(abs_max2(m, w.x), w.y), w.z), w.w);
}

// Eight values' stored bytes; rq = (r, q).  A whole number up to 127 is the
// low byte of y + 1.5 2^23 + 128 (the sum rounds half to even).
template <bool kE4M3>
__device__ __forceinline__ uint2 quant_code8(const uint4& w, float2 rq) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  const float2 r = make_float2(rq.x, rq.x), q = make_float2(rq.y, rq.y);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = bf2(in[i]);
    float2 y = mul2(x, q);
    fma2(y, x, r);
    if constexpr (kE4M3) {
      asm("{\n\t.reg .b16 p;\n\tcvt.rn.satfinite.e4m3x2.f32 p, %1, %2;\n\tcvt.u32.u16 %0, p;\n\t}"
          : "=r"(c[i])
          : "f"(y.y), "f"(y.x));
    } else {
      y = add2(y, make_float2(12583040.f, 12583040.f));
      c[i] = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040);
    }
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
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

// CTAs (x, KV head and side, sequence); a CTA takes every gridDim.x-th block
// that the call touches.  A thread's chunks of the next kAhead blocks arrive
// by cp.async in places of its own: no barrier for them, no bank conflicts,
// and more bytes in flight than registers would hold.
//  * A block that becomes full: a thread holds one 16-byte chunk of four
//    tokens (16 apart for keys, consecutive for values: their codes transpose
//    in registers); maximum over the CTA; the key codes go straight to their
//    rows, the value codes turn through shared memory, 16-byte chunks of a
//    row moved by its number against bank conflicts.
//  * The rows of the call that the tail keeps (the open block and the one
//    before it) are copied by the CTA of the first block, after it has read
//    the open block's old rows: they may take those rows' slots.
// The last CTA of a sequence to finish advances seq_len.
// Bound by HBM (512 bytes of a token, head and both sides in, 256 out): 131,072
// tokens x 8 heads (805 MB) in 142 us, 5,700 GB/s.  One token a sequence is a
// launch's latency, 3 us.
template <bool kE4M3>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) quant_append_kernel(QuantAppendArgs a) {
  extern __shared__ __align__(128) uint8_t sm[];
  uint4* ring = reinterpret_cast<uint4*>(sm);  // [kAhead][4][threads]
  uint8_t* codes0 = sm + kAhead * 4 * kAppendThreads * 16;  // [2][kQSide], values only
  __shared__ uint32_t part[2][kAppendThreads / 32];
  pdl_trigger();
  pdl_wait();
  const QuantView& c = a.c;
  const int h = blockIdx.y >> 1, side = blockIdx.y & 1, b = blockIdx.z, tid = threadIdx.x;
  const int L0 = quant_len(c, b);
  int n = a.n;
  if (a.n_new) n = max(0, min(n, a.n_new[b]));
  const long long cap = (long long)c.maxp * kQBlock;
  const bool over = L0 + (long long)n > cap;
  if (over) n = (int)(cap - L0);
  const int L1 = L0 + n;
  const __nv_bfloat16* rows = (side ? a.v : a.k) + b * a.ss + h * a.hs;
  // keys: tokens tid / 16 + 16 i, values: tokens 4 (tid / 16) + i; dims 8 d8 ..
  const int t0 = side ? 4 * (tid >> 4) : tid >> 4, ts = side ? 1 : 16, d8 = tid & 15;
  const int end = n > 0 ? L1 / kQBlock : 0;  // the first block that stays open
  int j = L0 / kQBlock + blockIdx.x, it = 0, s = 0;
  // this thread's first chunk of block j, and the way to its others
  const __nv_bfloat16* src = rows + ((long long)j * kQBlock + t0 - L0) * a.ts + d8 * 8;
  const long long step = (long long)ts * a.ts, jump = (long long)gridDim.x * kQBlock * a.ts;
  const uint32_t mine = smem_u32(ring + tid);
  int ask = j;  // the next block to ask for
  auto load = [&](int st) {
    if (ask < end) {
      const uint32_t to = mine + st * (4 * kAppendThreads * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat16* p = src + i * step;
        // the open block's rows of earlier calls are the tail's
        if (ask * kQBlock < L0) {
          const int t = ask * kQBlock + t0 + ts * i;
          if (t < L0) p = quant_tail(c, b, h, side, t) + d8 * 8;
        }
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * kAppendThreads * 16),
                     "l"(p)
                     : "memory");
      }
    }
    cp_async_commit();
    ask += gridDim.x;
    src += jump;
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) load(i);
  if (blockIdx.x == 0 && n > 0) {
    cp_async_wait<0>();
    __syncthreads();  // the open block's old rows are read
    // the call's rows that the tail keeps, 16 threads a row; all loads of a
    // round in flight at once
    const int k0 = max(L0, (L1 / kQBlock - 1) * kQBlock), e = (tid & 15) * 8;
    for (int r0 = k0 + (tid >> 4); r0 < L1; r0 += 64) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + 16 * i < L1)
          w[i] = *reinterpret_cast<const uint4*>(rows + (long long)(r0 + 16 * i - L0) * a.ts + e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + 16 * i < L1)
          *reinterpret_cast<uint4*>(quant_tail(c, b, h, side, r0 + 16 * i) + e) = w[i];
    }
  }
  // (a sequence that is already full takes no token, n is 0)
  if (over && blockIdx.x == 0 && tid == 0) quant_error(c, kErrCapacity);
#pragma unroll 1
  for (; j < end; j += gridDim.x, it ^= 1) {
    const int pg = __ldg(c.bt + (size_t)b * c.maxp + j);
    uint8_t* codes = codes0 + it * kQSide;
    cp_async_wait<kAhead - 1>();
    uint4 x[4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = ring[(s * 4 + i) * kAppendThreads + tid];
      m = abs_max8(m, x[i]);
    }
    load(s);
    s = s + 1 == kAhead ? 0 : s + 1;
    m = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xffffu));
    if ((tid & 31) == 0) part[it][tid >> 5] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) m = max(m, part[it][w]);
    const bool bad = m >= 0x7f80u;  // an infinity or a NaN
    const float top = kE4M3 ? 448.f : 127.f, least = 7.888609052210118e-31f;  // 2^-100
    const float am = bad ? 1.f : fmaxf(__uint_as_float(m << 16), least);
    const float inv = __frcp_rn(am);
    float2 rq;
    rq.x = top * inv;
    rq.y = __fmaf_rn(-rq.x, am, top) * inv;
    uint2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = quant_code8<kE4M3>(bad ? make_uint4(0, 0, 0, 0) : x[i], rq);
    const bool there = pg >= 0 && pg < c.num_pages;
    uint8_t* out = c.pages + ((size_t)(there ? pg : 0) * c.H + h) * kQSlab;
    if (side == 0) {
      if (there)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint2*>(out + quant_k_chunk(t0 + 16 * i, d8 >> 1) + (d8 & 1) * 8) = w[i];
    } else {
      uint32_t lo[4], hi[4];
      transpose4(w[0].x, w[1].x, w[2].x, w[3].x, lo);
      transpose4(w[0].y, w[1].y, w[2].y, w[3].y, hi);
      // word tid / 16 of rows 8 d8 + i: chunk tid / 64 turned by d8
      uint32_t* vs = reinterpret_cast<uint32_t*>(codes) + d8 * 8 * (kQBlock / 4) +
                     ((((tid >> 6) ^ d8) & 3) << 2) + ((tid >> 4) & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vs[i * (kQBlock / 4)] = lo[i];
        vs[(4 + i) * (kQBlock / 4)] = hi[i];
      }
      __syncthreads();
      if (there)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int k = tid + i * kAppendThreads, d = k >> 2, ch = k & 3;  // row, chunk
          reinterpret_cast<uint4*>(out + kQSide)[k] =
              reinterpret_cast<const uint4*>(codes)[d * 4 + (ch ^ ((d >> 3) & 3))];
        }
    }
    // the side's scale, and its half of the slab's zero bytes
    float* sc = reinterpret_cast<float*>(out + 2 * kQSide);
    if (there && tid == 0) sc[side] = bad ? __uint_as_float(0x7fc00000u) : __fdiv_rn(am, top);
    if (there && tid >= 32 && tid < 35) sc[2 + 3 * side + tid - 32] = 0.f;
    if (!there && tid == 0) quant_error(c, kErrBadPage);
  }
  // A CTA is counted once all its warps have read seq_len: one without a block
  // of its own has met no barrier before this one, and a warp that came after
  // the new length was stored would take the call's tokens for new ones again.
  __syncthreads();
  if (tid == 0) {
    // the last CTA of the sequence: every other has read seq_len
    __threadfence();
    const int last = (int)(gridDim.x * gridDim.y) - 1;
    if (atomicAdd(&c.counter[b], 1) == last) {
      c.seq_len[b] = L1;
      c.counter[b] = 0;
    }
  }
}

// Eight values; kWide: fp32 rows are 32-byte aligned, so that one store fills
// a sector (1.07 GB out in 211 us; two stores of 16 bytes, 284 us).
template <bool kWide>
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  if constexpr (kWide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]),
                 "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}
template <bool kWide>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                 pack_bf16x2(f[6], f[7]));
}

// One CTA per (block of the range, KV head, sequence); threads as in the
// append: keys by (token, chunk), values by (4 tokens, chunk).  Bound by HBM:
// 131,072 tokens x 8 heads to fp32 (1.34 GB moved) in 211 us, 6,360 GB/s, to
// bf16 in 125 us, 6,430.
template <bool kE4M3, typename T, bool kWide>
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
      store8<kWide>((side ? vrow : krow) + (t - f0) * a.ts + e, f);
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
    if (wanted(t)) store8<kWide>(krow + (t - f0) * a.ts + (tid & 15) * 8, f);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = base + 4 * (tid & 15) + i;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = slab ? quant_value<kE4M3>(vw[e] >> (8 * i)) * sv : 0.f;
    if (wanted(t)) store8<kWide>(vrow + (t - f0) * a.ts + (tid >> 4) * 8, f);
  }
}

}  // namespace

int quant_append_launch(const QuantAppendArgs& a, cudaStream_t st) {
  // blocks that n tokens can touch, wherever in a block they start
  const long long nb = (a.n + 62ll) / kQBlock + 1;
  // no more CTAs than are resident at once: the rest is their loops' work
  int dev = 0;
  DevInfo info;
  int rc = current_device_info(dev, info);
  if (rc != LRKV_OK) return rc;
  const long long room = (long long)info.sms * kAppendCtas / (2ll * a.c.H * a.c.B);
  const dim3 grid((unsigned)(nb < room ? nb : room < 1 ? 1 : room), 2 * a.c.H, a.c.B);
  QuantAppendArgs args = a;
  void* p[] = {&args};
  const void* fn = a.c.e4m3 ? (const void*)quant_append_kernel<true>
                            : (const void*)quant_append_kernel<false>;
  rc = prepare_kernel(fn, true);
  if (rc != LRKV_OK) return rc;
  return launch_pdl(fn, grid, dim3(kAppendThreads), kAppendSmem, st, p) == cudaSuccess ? LRKV_OK
                                                                             : LRKV_ERR_CUDA;
}

int quant_read_launch(const QuantReadArgs& a, int dtype, cudaStream_t st) {
  // blocks that n tokens can touch, and a sequence can have
  const long long nb = (a.n + 62ll) / kQBlock + 1;
  const dim3 grid((unsigned)(nb < a.c.maxp ? nb : a.c.maxp), a.c.H, a.c.B);
  QuantReadArgs args = a;
  void* p[] = {&args};
  const bool e = a.c.e4m3;
  const void* fn;
  if (dtype == LRKV_F32) {
    const bool wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 31) == 0 &&
                      ((a.ss | a.hs | a.ts) & 7) == 0;
    fn = wide ? (e ? (const void*)quant_read_kernel<true, float, true>
                   : (const void*)quant_read_kernel<false, float, true>)
              : (e ? (const void*)quant_read_kernel<true, float, false>
                   : (const void*)quant_read_kernel<false, float, false>);
  } else {
    fn = e ? (const void*)quant_read_kernel<true, __nv_bfloat16, true>
           : (const void*)quant_read_kernel<false, __nv_bfloat16, true>;
  }
  return launch_pdl(fn, grid, dim3(kAppendThreads), 0, st, p) == cudaSuccess ? LRKV_OK
                                                                             : LRKV_ERR_CUDA;
}

}  // namespace lrkv
