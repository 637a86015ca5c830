// Attention of few query rows over the 8-bit full-rank cache.
//
// Row r of a unit (sequence, KV head) is query r / G of q head h G + r % G.
// A code is an exact fp16 number, so with q brought to fp16 (exactly: times
// a power of two that puts its row's largest element in [2^14, 2^15); what
// is under 2^-31 of that loses bits) and the block's scales kept outside,
//   score = (q . c_k) (s_k scale 2^e),  acc += (p s_v) c_v
// run on mma.sync m16n8k16 with fp32 accumulation.  Besides the softmax's
// running maximum m a row keeps M', the running maximum of a block's largest
// score + floor(log2 s_v): the weights 2^(score - M') s_v 2^13 are then at
// most 2^15 whatever the blocks' scales, are rounded to fp16 once and keep
// eleven bits down to 2^-27 of the largest.  Within a block p goes by the block's
// own maximum.  Maxima are held rounded down to whole numbers, M' as what it is
// above m: both are exact however large the scores are, and so is every rescaling.
//
// What bounds it (calls over several caches in turn, more than L2 holds, at the
// clock named): HBM for long caches (64 sequences of 12,288 tokens x 8 heads: 1.6 GB
// in 244 us at 1,965 MHz, 280 in a long run at 1,670; 4 of 32,769: 50 us, 5,350 GB/s
// at 1,930), latency for short ones: 8 to 9 us between the launch and the last part
// folded (512 tokens 8.4 us, 4 x 8192 19.8 us, both at 1,965 MHz).  With 9 to 16 rows
// no pipe is full (issue slots 34 %, warp MMAs 18 %, DRAM 40 %): a warp's only slab is
// empty while its next page comes, and its page takes it a chain of products,
// exponentials and products.  8 sequences of 12,288, 16 rows: 57 us int8, 53 e4m3
// (3,530 and 3,810 GB/s, 1,965 MHz).
// Figures of one choice against another, below, are of calls back to back on one
// cache, of which L2 keeps a part.
//
// One launch, persistent, one CTA per SM.  The blocks of all units are laid
// end to end and each CTA takes an equal contiguous range (the caller keeps
// batch x heads x pages under 2^31: the line is counted in 32 bits).
//  * W consumer warps take every W-th block.  Each keeps D page slabs (codes
//    and scales, one bulk copy each) of its own in flight and refills a stage
//    as soon as it has read it, so no warp waits for another's page.
//    S^T = C_k q^T: A fragments are the code bytes themselves, a lane reading 16 bytes of a token's row
//    (which dims form a 16-wide step is free, as long as q agrees) and
//    widening them in registers; V is stored transposed, so acc^T = C_v^T P^T
//    reads its A fragments the same way; P^T moves into the B operand by
//    movmatrix.  Tokens are dealt to A rows so that this lands them in the
//    order of the V bytes: row i of step s is token 16 (i / 2) + 4 s + i % 2
//    (+ 2 for rows 8..15);
//  * tail warp: the open block's bf16 rows, straight from global memory, on
//    bf16 MMAs with the weights split in two bf16 halves.
// At the end of a unit's part the warps' (m, l, acc) are combined in
// shared memory.  A unit in one CTA is finished there; otherwise the parts
// go to the workspace and the unit's last CTA to arrive folds them in order
// (so the result does not depend on which was last) and zeroes the counter.
#include "quant.cuh"
#include "tcgen05.cuh"

namespace lrkv {

namespace {

constexpr int kPad = kHeadDim + 4;              // combine rows: no bank conflicts
constexpr float kBoost = 8192.f;                // 2^13
// What a part's end (its warps' sums, its record) takes, in blocks; the line
// has so many places before a unit's blocks (4 x 8192 tokens 18.3 -> 17.3 us,
// 64 x 300 28.4 -> 24.3; 3 too few, 8 the same).
constexpr int kPartCost = 6;

struct DecPlan {
  int slots, ml, full, start, len, nq, misc, total;
};
__host__ __device__ inline DecPlan dec_plan(int W, int D, int rows, int B) {
  DecPlan p;
  p.slots = W * D * kQSlab;
  p.ml = p.slots + (W + 1) * rows * kPad * 4;
  p.full = p.ml + (W + 1) * rows * 16;
  p.start = p.full + W * D * 8;
  p.len = p.start + (B + 1) * 4;
  p.nq = p.len + B * 4;
  p.misc = p.nq + B * 4;
  p.total = p.misc + 16;
  return p;
}

// Workspace: a counter per CTA, then two records of [16][132] fp32 (m, l, M' - m,
// -, 128 sums) per CTA.  Of the units that a CTA shares with others one at
// most begins in it and one at most began before it: they have record 1 and
// record 0, and the unit's counter is that of the CTA in which it begins.
// Nothing depends on the call's sizes, so any call may follow any other.
constexpr int kMaxRows = 16;
__host__ __device__ inline size_t dec_records(int C) { return ((size_t)C * 4 + 255) / 256 * 256; }
__host__ __device__ inline size_t dec_ws(int C) {
  return dec_records(C) + (size_t)C * 2 * kMaxRows * kPad * 4;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Over the 8 lanes that share lane % 4.
__device__ __forceinline__ float col_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float col_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// A part of a unit: its place, the blocks [i0, i1) of `tiles` in this CTA's
// range, and the line's index of its block 0.
struct Part {
  int b, h, tiles, i0, i1, first;
};

template <bool kE4M3, int NT, int W, int D>
__global__ void __launch_bounds__((W + 1) * 32, 1) quant_decode_kernel(QuantAttnArgs a) {
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t sm[];
  const QuantView& c = a.c;
  const DecPlan pl = dec_plan(W, D, kRows, c.B);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + pl.full);
  float* slots = reinterpret_cast<float*>(sm + pl.slots);
  float4* ml = reinterpret_cast<float4*>(sm + pl.ml);  // [W + 1][kRows] (m, l, M' - m)
  int* start = reinterpret_cast<int*>(sm + pl.start);
  int* slen = reinterpret_cast<int*>(sm + pl.len);
  int* snq = reinterpret_cast<int*>(sm + pl.nq);
  volatile int* fail = reinterpret_cast<volatile int*>(sm + pl.misc);
  volatile int *lastflag = fail + 1, *nunits = fail + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    *fail = 0;
    for (int s = 0; s < W * D; ++s) mbar_init(&full[s], 1);
    mbar_fence_init();
  }
  pdl_trigger();
  pdl_wait();
  if (warp == W) {
    // blocks before each sequence; a sequence without tokens still has one
    // (empty) block for its queries' zeros
    const int per = (c.B + 31) / 32, b0 = min(c.B, lane * per), b1 = min(c.B, b0 + per);
    int own = 0, units = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      slen[b] = quant_len(c, b);
      snq[b] = quant_queries(a, b);
      if (snq[b]) {
        own += (max(1, (slen[b] + kQBlock - 1) / kQBlock) + kPartCost) * c.H;
        units += c.H;
      }
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int e = incl - own;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      start[b] = e;
      if (snq[b]) e += (max(1, (slen[b] + kQBlock - 1) / kQBlock) + kPartCost) * c.H;
    }
    units = __reduce_add_sync(0xffffffffu, units);
    if (lane == 31) {
      start[c.B] = incl;
      *nunits = units;
    }
  }
  __syncthreads();
  const int total = start[c.B];
  // A unit's last CTA adds up its parts: no more of them than about 2 sqrt(the
  // blocks of a unit) (a sequence's only head, 8 rows, 32,768 tokens: 19 us; a
  // part in every CTA 32, 4 sqrt 21; 131,072 tokens 28, 33 and 34; 1 sqrt loses
  // elsewhere, 8 heads of 8192 tokens 12.7 against 10.9).
  const int units = *nunits;
  const float parts = 2.f * sqrtf((float)total / max(units, 1)) + 1.f;
  const int C = (int)min(min((long long)gridDim.x, (long long)total), (long long)(units * parts));
  if ((int)blockIdx.x >= C) return;
  // CTA i takes per blocks, the first `extra` CTAs one more
  const int per = total / C, extra = total - per * C;
  auto range_lo = [&](int i) { return i * per + min(i, extra); };
  auto cta_of = [&](int y) {
    const int big = extra * (per + 1);
    return y < big ? y / (per + 1) : extra + (y - big) / per;
  };
  const int lo = range_lo(blockIdx.x), hi = range_lo(blockIdx.x + 1);

  auto cut = [&](Part& p) {
    p.tiles = max(1, (slen[p.b] + kQBlock - 1) / kQBlock);
    p.i0 = max(0, lo - p.first);
    p.i1 = min(hi - p.first, p.tiles);
  };
  // the part after p, whose first block is the line's block p.first + p.tiles
  auto next_part = [&](Part& p) {
    p.first += p.tiles + kPartCost;
    if (++p.h == c.H) {
      p.h = 0;
      do ++p.b; while (start[p.b + 1] == start[p.b]);
    }
    cut(p);
  };
  // the part that the range begins with
  Part p0;
  {
    int l = 0, r = c.B;
#pragma unroll 1
    while (r - l > 1) {
      const int mid = (l + r) >> 1;
      if (start[mid] <= lo) l = mid; else r = mid;
    }
    p0.b = l;
    const int tiles = max(1, (slen[l] + kQBlock - 1) / kQBlock);
    p0.h = (lo - start[l]) / (tiles + kPartCost);
    p0.first = start[l] + p0.h * (tiles + kPartCost) + kPartCost;
    cut(p0);
  }

  // ---------------- consumer: the loads it has in flight
  uint8_t* ring = sm + warp * D * kQSlab;
  uint64_t* bar = full + warp * D;
  int n_issued = 0, n_read = 0;      // slabs asked for, slabs used
  uint32_t bad = 0;                  // stages whose page was out of range
  int xi = lo + warp;                // next block to ask for
  Part pi = p0;                      // its part
  // next full block at or after xi; its page id is loaded here and first
  // looked at by the issue() after this one
  int npage = -1, nhead = 0;
  auto find_next = [&]() {
    while (xi < hi) {
      while (xi >= pi.first + pi.tiles) next_part(pi);
      const int i = xi - pi.first;
      if (i >= 0 && (i + 1) * kQBlock <= slen[pi.b]) {
        npage = __ldg(c.bt + (size_t)pi.b * c.maxp + i);
        nhead = pi.h;
        return true;
      }
      xi += W;
    }
    return false;
  };
  const uint64_t pol = l2_evict_first_policy();
  bool more = false;
  auto issue = [&]() {
    if (!more) return;
    const int s = n_issued % D;
    if (npage >= 0 && npage < c.num_pages) {
      bad &= ~(1u << s);
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar[s], kQSlab);
        bulk_g2s_hint(ring + s * kQSlab, c.pages + ((size_t)npage * c.H + nhead) * kQSlab, kQSlab,
                      &bar[s], pol);
      }
    } else {
      bad |= 1u << s;
      if (lane == 0) {
        quant_error(c, kErrBadPage);
        mbar_arrive(&bar[s]);
      }
    }
    ++n_issued;
    xi += W;
    more = find_next();
  };

  // r / G for r < 16
  const uint32_t inv = (65536u + a.G - 1) / a.G;
  auto query_of = [&](int r) { return (int)((r * inv) >> 16); };
  // row r of a part's queries
  auto qrow = [&](const Part& p, int r) {
    const int i = query_of(r);
    return a.q + p.b * a.qs + (long long)(p.h * a.G + r - i * a.G) * a.qh + (long long)i * a.qt;
  };
  // a lane's chunks of its rows, as they are
  uint4 qraw[NT][4];
  auto load_q = [&](const Part& p) {
    const int rows = snq[p.b] * a.G;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g;
#pragma unroll
      for (int i = 0; i < 4; ++i) qraw[n][i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(qrow(p, r));
        qraw[n][0] = __ldg(src + 2 * t);
        qraw[n][1] = __ldg(src + 2 * t + 1);
        qraw[n][2] = __ldg(src + 8 + 2 * t);
        qraw[n][3] = __ldg(src + 9 + 2 * t);
      }
    }
  };
  if (warp < W) {
    more = find_next();
    // on its way while the first pages are asked for (4 x 8192 tokens 19.4 ->
    // 18.4 us; two row tiles spill)
    if constexpr (NT == 1) load_q(p0);
#pragma unroll 1
    for (int s = 0; s < D; ++s) issue();
  }

  int* counters = static_cast<int*>(a.ws);
  float* records = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + dec_records(gridDim.x));

  Part p = p0;
  for (int x = lo; x < hi;) {
    if (p.i1 <= 0) break;  // the range ends before the unit's first block
    const int L = slen[p.b], nq = snq[p.b], rows = nq * a.G;  // at most kRows
    const int pos0 = L - nq;  // position of query 0
    float m[2 * NT], l[2 * NT], dv[2 * NT], acc[8][NT][4];
    int pos[2 * NT];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      m[i] = dv[i] = -INFINITY;
      l[i] = 0.f;
      // this lane's columns: row 8 (i / 2) + 2 t + i % 2
      const int r = 8 * (i >> 1) + 2 * t + (i & 1);
      pos[i] = r < rows ? pos0 + query_of(r) : 0x7fffffff;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][n][e] = 0.f;
    float acc_scale = 1.f;  // acc's unit in the end
    bool any = false;

    if (warp < W) {
      // ---------------- quantised blocks
      const int xb = p.first + p.i0;
      int xc = xb + ((warp - (xb - lo) % W) + W) % W;
      const int xend = p.first + p.i1;
      const bool have = xc < xend && (xc - p.first + 1) * kQBlock <= L;
      if (have) {
        any = true;
        // q's B fragments, fp16, and the columns' factors
        uint32_t qf[NT][8][2];
        float fcol[2 * NT];
        if (NT == 2 || x != lo) load_q(p);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4(&w)[4] = qraw[n];
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mx = __vmaxu2(mx, w[i].x & 0x7fff7fffu);
            mx = __vmaxu2(mx, w[i].y & 0x7fff7fffu);
            mx = __vmaxu2(mx, w[i].z & 0x7fff7fffu);
            mx = __vmaxu2(mx, w[i].w & 0x7fff7fffu);
          }
          mx = max(mx >> 16, mx & 0xffffu);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // exponent of the row's largest element; not finite: as it is
          int e = (int)(mx >> 7) - 127;
          e = mx == 0 || e == 128 ? 14 : max(e, -100);
          const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          const float down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              qf[n][2 * i + (k >> 1)][k & 1] = pack_f16x2(bf_lo(v[k]) * up, bf_hi(v[k]) * up);
          }
          fcol[2 * n] = __shfl_sync(0xffffffffu, down, 8 * t) * (a.scale * kLog2e);
          fcol[2 * n + 1] = __shfl_sync(0xffffffffu, down, 8 * t + 4) * (a.scale * kLog2e);
        }
        for (; xc < xend; xc += W) {
          const int i = xc - p.first;
          if ((i + 1) * kQBlock > L) break;
          const int s = n_read % D;
          const bool ok = quant_wait_warp(&bar[s], (n_read / D) & 1, fail, lane);
          const bool use = ok && !((bad >> s) & 1);
          ++n_read;
          if (use) {
            const uint8_t* slab = ring + s * kQSlab;
            const float2 sc = *reinterpret_cast<const float2*>(slab + 2 * kQSide);
            // ---- scores: sacc[s4][n]: tokens 16 (g / 2) + 4 s4 + g % 2 (+ 2)
            float sacc[4][NT][4];
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[s4][n][e] = 0.f;
            // the four token groups side by side: their sums are chains of
            // their own (one group after the other is one long chain)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint4 ka[4], kb[4];
#pragma unroll
              for (int s4 = 0; s4 < 4; ++s4) {
                const uint8_t* rk = slab + (16 * (g >> 1) + 4 * s4 + (g & 1)) * kHeadDim +
                                    ((t ^ (hf << 2) ^ ((g & 1) << 2)) << 4);
                ka[s4] = *reinterpret_cast<const uint4*>(rk);
                kb[s4] = *reinterpret_cast<const uint4*>(rk + 2 * kHeadDim);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int s4 = 0; s4 < 4; ++s4) {
                  const uint32_t wa = k == 0 ? ka[s4].x : k == 1 ? ka[s4].y : k == 2 ? ka[s4].z : ka[s4].w;
                  const uint32_t wb = k == 0 ? kb[s4].x : k == 1 ? kb[s4].y : k == 2 ? kb[s4].z : kb[s4].w;
                  uint32_t a0, a1, a2, a3;
                  quant_half4<kE4M3>(wa, a0, a2);
                  quant_half4<kE4M3>(wb, a1, a3);
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma_f16(sacc[s4][n], a0, a1, a2, a3, qf[n][4 * hf + k][0], qf[n][4 * hf + k][1]);
                }
            }
            // ---- softmax: one maximum per column and block
            const int base = i * kQBlock;
            const bool edge = base + kQBlock - 1 > pos0;
            float corr[2 * NT];
            bool moved = false;
            // s_v = 2^ev fv, 1 <= fv < 2 (a NaN stays in fv)
            const uint32_t vbits = __float_as_uint(sc.y);
            const bool vnan = sc.y != sc.y;
            const float ev = vnan ? 0.f : (float)((int)(vbits >> 23) - 127);
            const float fv = vnan ? sc.y : __uint_as_float((vbits & 0x7fffffu) | 0x3f800000u);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float f = fcol[2 * n + j] * sc.x;
                float mx = -INFINITY;
#pragma unroll
                for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    float& v = sacc[s4][n][2 * u + j];
                    v *= f;
                    if (edge && base + 16 * (g >> 1) + 4 * s4 + (g & 1) + 2 * u > pos[2 * n + j])
                      v = -INFINITY;
                    mx = fmaxf(mx, v);
                  }
                mx = col_max(mx);
                mx = floorf(mx);
                const float mn = fmaxf(mx, m[2 * n + j]);
                const float ref = or_zero(mn), bref = or_zero(mx);
                // from the old maximum and from the block's to the new one
                const float sh = m[2 * n + j] - ref, bsh = mx - ref;
                const float cr = ex2_approx(sh), cb = ex2_approx(bsh);
                const float old = dv[2 * n + j] + sh, dn = fmaxf(old, bsh + ev), dref = or_zero(dn);
                moved |= dn != old;
                corr[2 * n + j] = ex2_approx(old - dref);
                m[2 * n + j] = mn;
                dv[2 * n + j] = dn;
                // p by the block's own maximum, so that one that counts for its
                // values is not flushed; then 2^(maximum - M') s_v 2^13: at most 2^15 in all
                const float wmul = fv * ex2_approx(bsh + ev - dref + 13.f);
                float sum = 0.f;
#pragma unroll
                for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
                  for (int u = 0; u < 2; ++u) {
                    float& v = sacc[s4][n][2 * u + j];
                    const bool out = edge && v == -INFINITY;
                    v = ex2_approx(v - bref);
                    sum += v;
                    v = out ? 0.f : v * wmul;  // a NaN scale does not reach what is masked
                  }
                l[2 * n + j] = l[2 * n + j] * cr + sum * cb;
              }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[j][n][e] *= corr[2 * n + (e & 1)];
            }
            uint32_t pb[4][NT][2];
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                  pb[s4][n][u] =
                      movmatrix_trans(pack_f16x2(sacc[s4][n][2 * u], sacc[s4][n][2 * u + 1]));
            // ---- values: dims 16 j + g (+ 8), tokens 16 t .. 16 t + 15
            const uint8_t* vs = slab + kQSide + g * kQBlock + t * 16;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint4 va = *reinterpret_cast<const uint4*>(vs + 16 * j * kQBlock);
              const uint4 vb = *reinterpret_cast<const uint4*>(vs + (16 * j + 8) * kQBlock);
              const uint32_t wa[4] = {va.x, va.y, va.z, va.w};
              const uint32_t wb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
              for (int s4 = 0; s4 < 4; ++s4) {
                uint32_t a0, a1, a2, a3;
                quant_half4<kE4M3>(wa[s4], a0, a2);
                quant_half4<kE4M3>(wb[s4], a1, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma_f16(acc[j][n], a0, a1, a2, a3, pb[s4][n][0], pb[s4][n][1]);
              }
            }
          }
          __syncwarp();  // the stage is read: refill it
          if (ok) issue();
        }
        acc_scale = 1.f / kBoost;
      }
    } else if (p.i1 == p.tiles && L % kQBlock != 0) {
      // ---------------- the open block, tokens base .. L - 1
      any = true;
      const int base = L / kQBlock * kQBlock;
      const __nv_bfloat16* kt = quant_tail(c, p.b, p.h, 0, base);
      const __nv_bfloat16* vt = quant_tail(c, p.b, p.h, 1, base);
      float sacc[4][NT][4];
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sacc[s4][n][e] = 0.f;
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u4 = 0; u4 < 4; ++u4) {  // dims 32 u4 + 8 t .. + 7 of this lane
        uint4 qw[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          qw[n] = 8 * n + g < rows
                      ? __ldg(reinterpret_cast<const uint4*>(qrow(p, 8 * n + g)) + 4 * u4 + t)
                      : zero;
#pragma unroll
        for (int s4 = 0; s4 < 4; ++s4) {
          const int ta = 16 * (g >> 1) + 4 * s4 + (g & 1), tb = ta + 2;
          const uint4 ka = base + ta < L
                               ? *(reinterpret_cast<const uint4*>(kt + ta * kHeadDim) + 4 * u4 + t)
                               : zero;
          const uint4 kb = base + tb < L
                               ? *(reinterpret_cast<const uint4*>(kt + tb * kHeadDim) + 4 * u4 + t)
                               : zero;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_b16(sacc[s4][n], ka.x, kb.x, ka.y, kb.y, qw[n].x, qw[n].y);
            mma_b16(sacc[s4][n], ka.z, kb.z, ka.w, kb.w, qw[n].z, qw[n].w);
          }
        }
      }
      const float f = a.scale * kLog2e;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = -INFINITY;
          const int last = min(pos[2 * n + j], L - 1);
#pragma unroll
          for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float& v = sacc[s4][n][2 * u + j];
              v = base + 16 * (g >> 1) + 4 * s4 + (g & 1) + 2 * u > last ? -INFINITY : v * f;
              mx = fmaxf(mx, v);
            }
          mx = col_max(mx);
          m[2 * n + j] = mx = floorf(mx);
          dv[2 * n + j] = 0.f;
          const float ref = or_zero(mx);
          float sum = 0.f;
#pragma unroll
          for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float& v = sacc[s4][n][2 * u + j];
              v = ex2_approx(v - ref);
              sum += v;
            }
          l[2 * n + j] = sum;
        }
      int bad = 64;  // first open token whose value row is not finite
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4) {
        uint32_t ph[NT][2], pw[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float x0 = sacc[s4][n][2 * u], x1 = sacc[s4][n][2 * u + 1];
            const uint32_t hi2 = pack_bf16x2(x0, x1);
            ph[n][u] = movmatrix_trans(hi2);
            pw[n][u] = movmatrix_trans(pack_bf16x2(x0 - bf_lo(hi2), x1 - bf_hi(hi2)));
          }
        // dims 8 g + i (half 0) and 64 + 8 g + i (half 1) of tokens 16 t + 4 s4 ..
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {  // 4 dims at a time
          uint2 v[4][2];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int tok = 16 * t + 4 * s4 + k;
              v[k][hf] = base + tok < L
                             ? *reinterpret_cast<const uint2*>(vt + tok * kHeadDim + 64 * hf + 8 * g +
                                                               4 * q2)
                             : make_uint2(0, 0);
              // a weight of 0 must stay 0: such rows count through `bad`
              uint2& w = v[k][hf];
              const uint32_t big = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
              if (max(big >> 16, big & 0xffffu) >= 0x7f80u) {
                bad = min(bad, tok);
                w = make_uint2(0, 0);
              }
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t sel = (i & 1) ? 0x7632 : 0x5410;
            auto pick = [&](int k, int hf) { return (i >> 1) ? v[k][hf].y : v[k][hf].x; };
            const uint32_t a0 = __byte_perm(pick(0, 0), pick(1, 0), sel);
            const uint32_t a1 = __byte_perm(pick(0, 1), pick(1, 1), sel);
            const uint32_t a2 = __byte_perm(pick(2, 0), pick(3, 0), sel);
            const uint32_t a3 = __byte_perm(pick(2, 1), pick(3, 1), sel);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_b16(acc[4 * q2 + i][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
              mma_b16(acc[4 * q2 + i][n], a0, a1, a2, a3, pw[n][0], pw[n][1]);
            }
          }
        }
      }
      bad = (int)__reduce_min_sync(0xffffffffu, (uint32_t)bad);
      if (bad < 64)
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i)
          if (base + bad <= pos[i]) l[i] = NAN;
    }

    // ---------------- combine the warps' (m, l, M' - m, acc)
    __syncthreads();  // the slots of the part before are read
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * n + 2 * t + j;
        const float ls = col_sum(l[2 * n + j]);
        if (g == 0) ml[warp * kRows + r] = make_float4(m[2 * n + j], ls, dv[2 * n + j], 0.f);
        if (any) {
          float* dst = slots + ((size_t)warp * kRows + r) * kPad;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int d0 = warp < W ? 16 * q + g : 8 * g + q;
            dst[d0] = acc[q][n][j] * acc_scale;
            dst[d0 + (warp < W ? 8 : 64)] = acc[q][n][2 + j] * acc_scale;
          }
        }
      }
    __syncthreads();
    const bool whole = p.i0 == 0 && p.i1 == p.tiles;
    // record of this unit's part in CTA cc (begins: in that CTA)
    auto record = [&](int cc, bool begins) {
      return reinterpret_cast<float4*>(records + ((size_t)2 * cc + (begins ? 1 : 0)) * kMaxRows * kPad);
    };
    // a row's result, or zeros where it saw nothing: lane's 4 dims
    auto finish = [&](int r, const float4& st, const float4& o) {
      const int i = query_of(r);
      __nv_bfloat16* dst = a.o + p.b * a.os + (long long)(p.h * a.G + r - i * a.G) * a.oh +
                           (long long)i * a.ot + 4 * lane;
      const float f = st.y == 0.f ? 0.f : ex2_approx(st.z) / st.y;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
    };
    // A part that saw nothing (a NaN sum is something) adds nothing.
    auto nothing = [](const float4& st) { return st.x == -INFINITY && st.y == 0.f; };
    for (int r = warp; r < rows; r += W + 1) {
      float4 st[W + 1], S = make_float4(-INFINITY, 0.f, -INFINITY, 0.f), o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w <= W; ++w) {
        st[w] = ml[w * kRows + r];
        S.x = fmaxf(S.x, st[w].x);
      }
      const float ref = or_zero(S.x);
#pragma unroll
      for (int w = 0; w <= W; ++w) {  // each from the common maximum
        st[w].x -= ref;
        st[w].z += st[w].x;
        S.z = fmaxf(S.z, st[w].z);
      }
      const float zref = or_zero(S.z);
#pragma unroll
      for (int w = 0; w <= W; ++w) {
        if (nothing(st[w])) continue;
        const float f = ex2_approx(st[w].z - zref);
        const float4 v = *reinterpret_cast<const float4*>(slots + (w * kRows + r) * kPad + 4 * lane);
        S.y += st[w].y * ex2_approx(st[w].x);
        o.x += v.x * f;
        o.y += v.y * f;
        o.z += v.z * f;
        o.w += v.w * f;
      }
      if (whole) {
        finish(r, S, o);
      } else {
        float4* dst = record(blockIdx.x, p.i0 == 0) + r * (kPad / 4);
        if (lane == 0) dst[0] = S;
        dst[1 + lane] = o;
      }
    }
    if (!whole) {
      // the CTAs that hold blocks of this unit; the barrier hands all threads'
      // records to thread 0, whose atomic releases them and acquires the others'
      const int c0 = cta_of(p.first), c1 = cta_of(p.first + p.tiles - 1);
      __syncthreads();
      if (threadIdx.x == 0) {
        int before;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                     : "=r"(before)
                     : "l"(counters + c0)
                     : "memory");
        *lastflag = before == c1 - c0;
        if (before == c1 - c0) counters[c0] = 0;
      }
      __syncthreads();
      if (*lastflag) {
        // a lane weighs every 32nd part, then the warp adds them in order (a
        // running maximum over the parts is one long chain: 52 us for the 148
        // parts of a sequence's only head)
        float* wt = slots + warp * kRows * kPad;  // (the slots have been read)
        const int nc = c1 - c0 + 1;
        for (int r = warp; r < rows; r += W + 1) {
          auto place = [&](int k) { return record(c0 + k, k == 0) + r * (kPad / 4); };
          float4 v = make_float4(-INFINITY, 0.f, -INFINITY, 0.f), S = v, o = make_float4(0.f, 0.f, 0.f, 0.f);
          constexpr int kFirst = NT == 1 ? 8 : 4;
          float4 u[kFirst];  // of the first parts, asked for at once (two row tiles: 8 spill)
#pragma unroll
          for (int k = 0; k < kFirst; ++k)
            if (k < nc) u[k] = __ldcg(place(k) + 1 + lane);
          if (lane < nc) v = __ldcg(place(lane));
          auto join = [&](float x, float z) {
            const float xn = fmaxf(S.x, x), r = or_zero(xn);
            S.z = fmaxf(S.x - r + S.z, x - r + z);
            S.x = xn;
          };
          join(v.x, v.z);
          for (int k = lane + 32; k < nc; k += 32) {
            const float4 y = __ldcg(place(k));
            join(y.x, y.z);
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1)
            join(__shfl_xor_sync(0xffffffffu, S.x, d), __shfl_xor_sync(0xffffffffu, S.z, d));
          const float ref = or_zero(S.x), zref = or_zero(S.z);
          for (int k = lane; k < nc; k += 32) {
            if (k >= 32) v = __ldcg(place(k));
            wt[k] = ex2_approx(v.x - ref + v.z - zref);
            S.y += v.y * ex2_approx(v.x - ref);
          }
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) S.y += __shfl_xor_sync(0xffffffffu, S.y, d);
          __syncwarp();
          auto add = [&](const float4& y, float f) {
            o.x += y.x * f;
            o.y += y.y * f;
            o.z += y.z * f;
            o.w += y.w * f;
          };
#pragma unroll
          for (int k = 0; k < kFirst; ++k)
            if (k < nc) add(u[k], wt[k]);
#pragma unroll 8
          for (int k = kFirst; k < nc; ++k) add(__ldcg(place(k) + 1 + lane), wt[k]);
          __syncwarp();
          finish(r, S, o);
        }
      }
    }
    x = p.first + p.i1;
    if (x < hi) next_part(p);
  }
  if (*fail && warp < W && lane == 0) {
    quant_drain(bar, n_issued, D);
    quant_error(c, kErrTimeout);
  }
}

}  // namespace

// Rows per group, and the kernel for them.
template <bool kE4M3, int NT, int W, int D>
static int launch(const QuantAttnArgs& a, const DevInfo& info, cudaStream_t st) {
  const void* fn = (const void*)quant_decode_kernel<kE4M3, NT, W, D>;
  const int smem = dec_plan(W, D, 8 * NT, a.c.B).total;
  if (smem > info.optin) return LRKV_ERR_UNSUPPORTED;
  const int rc = prepare_kernel(fn, true);
  if (rc != LRKV_OK) return rc;
  QuantAttnArgs args = a;
  void* p[] = {&args};
  return launch_pdl(fn, dim3(info.sms), dim3((W + 1) * 32), smem, st, p) == cudaSuccess
             ? LRKV_OK
             : LRKV_ERR_CUDA;
}

size_t quant_attn_workspace(int, int H, int Hq, int n) {
  int dev = 0;
  DevInfo info;
  if (current_device_info(dev, info) != LRKV_OK) return 0;
  // the counters come first in both layouts, the records need no zeros
  return (long long)n * (Hq / H) <= kMaxRows ? dec_ws(info.sms) : quant_prefill_workspace(info.sms);
}

int quant_attn_launch(const QuantAttnArgs& a, cudaStream_t st) {
  int dev = 0;
  DevInfo info;
  const int rc = current_device_info(dev, info);
  if (rc != LRKV_OK) return rc;
  // Six consumer warps with two slabs each: one token of the 32K layer (G 4)
  // 51.7 us, 64 sequences of 12000 239 us; five warps 58.0 and 269, eight with one
  // slab each 57.1 and 261, four with three 53.9 and 254 (this kernel's first form).
  // More sequences than the lengths' place in shared memory allows: five.
  if ((long long)a.n * a.G <= 8) {
    if (dec_plan(6, 2, 8, a.c.B).total <= info.optin)
      return a.c.e4m3 ? launch<true, 1, 6, 2>(a, info, st) : launch<false, 1, 6, 2>(a, info, st);
    return a.c.e4m3 ? launch<true, 1, 5, 2>(a, info, st) : launch<false, 1, 5, 2>(a, info, st);
  }
  // Two row tiles hold twice the registers and combine twice the rows: seven
  // warps of one slab (8 x 12000 tokens, 16 rows: 57.5 us; four of two 58.5,
  // eight of one, which spills, 67.5; the tensor-memory kernel 97).
  if ((long long)a.n * a.G <= kMaxRows)
    return a.c.e4m3 ? launch<true, 2, 7, 1>(a, info, st) : launch<false, 2, 7, 1>(a, info, st);
  // Up to a tile's rows in copies over the tile, against quant_prefill.cu (caches
  // in turn, 1,965 MHz): 4 x 16384 tokens with 20, 64 and 128 rows 53, 58 and 78 us
  // against 80, 82 and 86; 64 x 512 with 32, 64 and 128: 56, 62 and 87 against 72, 72
  // and 73.  (Where a CTA has short units 128 rows lose, 16 x 1024 tokens 46 us
  // against 39.  Lengths are on the device; max_pages_per_seq, a bound on them, is
  // not used for a rule.)
  if ((long long)a.n * a.G <= 128) return quant_few_launch(a, info, st);
  return quant_prefill_launch(a, info, st);
}

}  // namespace lrkv
