// Attention of many query rows over the 8-bit full-rank cache, on the
// fifth-generation tensor cores.
//
// The mathematics is quant_decode.cu's: codes are exact fp16 numbers, q is
// fp16 times a power of two per row, the blocks' scales stay outside the
// products.  Row r of a unit (sequence, KV head) is query r / G of q head
// h G + r % G, so the heads of a group share their keys' tiles.  A tile is
// 256 rows, two groups of 128 (the MMA's M); a step is one page of 64 keys.
//
// Persistent, one CTA per SM, 16 warps:
//  * warps 0-3 and 4-7: softmax of group 0 and 1, one row per thread (its
//    TMEM lane).  S comes from TMEM, P goes back over S's columns as fp16.
//    TMEM holds two S of 64 columns and one O per group, so a group's next
//    scores are ready before its softmax ends.
//  * warps 8-11: converters.  Codes from L2 into registers a step ahead, two
//    bytes to two fp16 numbers, into the 128-byte-swizzled K-major tiles
//    (keys as rows for Q K^T; the stored transpose of V is already K-major
//    for P V).  The open block's rows become fp16 under a power of two each.
//  * warps 12 and 13, one lane each, for group 0 and 1: per step P V (A from
//    TMEM), then Q K^T of the step after the next into the S that P has just
//    left.  (One thread for both needed 2000 clocks a step to issue what takes
//    the tensor cores 1240.)
// What bounds it: a step of 64 keys x 256 rows takes 2350 clocks, in which
// nothing is full (tensor cores 1280, exponentials 1024, issue slots 52 %): it
// is the chain of a step through softmax (2000: TMEM's latency, the row
// maximum, the exponentials, the hand-over) and back through the products.  And
// the card: in a long run it draws 990 W, its limit, at 1.78 GHz of 1.965.
// 2048 queries of 32 heads over 2 x 16,384 tokens: 1.06 ms (970 TFLOP/s) on a
// cool card at 1,965 MHz, 1.16 ms (885) in a long run at 1,800; 8192 over themselves
// 0.61 to 0.65 ms (900 to 845).  A tile's start and end take 12 to 16 thousand
// clocks: 32 prompts of 512 tokens 199 us (346 TFLOP/s, 1,965 MHz).
// Measured against it, the 2048 queries: two threads a row on sixteen softmax
// warps 1.38 ms against 1.09 (what a row costs once is paid twice); sixteen
// warps that take a row's steps in turns 1.17 against 1.12; one S that is given
// back as soon as it is in registers, and P of its own, 1.15 against 1.11 (8K
// prompt 0.65 against 0.66); a part of the exponentials as polynomials on the
// FMA pipe 1.29 against 1.11; the next S loaded ahead into registers 1.43
// against 1.11; the groups started half a step apart: no change, they fall into
// step again; separate converters of keys and of values (quant_few.cu's) 1.25
// against 1.23, 8K prompt 0.72 against 0.66.
// A row keeps its references m (scores) and M' (scores + floor(log2 s_v)) as
// long as they lag by at most 2^kLazy, so O is seldom rescaled; a weight is
// then under 2^(2 + kLazy + kBoostLog) = 2^15 and fp16's floor lies 2^-33
// below the row's largest.
//
// The steps of all tiles are laid end to end and each CTA takes an equal
// contiguous range (causal tiles differ in length, and a few tiles over a
// long cache still fill the GPU).  A tile cut by a range's border goes
// through records in the workspace, which a second launch folds in order.
#include <type_traits>

#include "quant_tc.cuh"

namespace lrkv {

namespace {

constexpr int kRing = 4;                        // key and value tiles in flight
constexpr int kPreThreads = 512;
constexpr int kQHalf = 128 * 128;               // 64 dims of a group's 128 rows of q
constexpr int kQGroup = 2 * kQHalf;
// A step's scales are read until its P is written; the converters are at most
// kRing + 2 steps ahead of that.
constexpr int kScaleRing = 8;
// Steps ahead at which a page is brought into L2 (256 queries over 16K, where
// few tiles share a page: 0.39 ms without, 0.33 with; 2, 3 and 4 alike).
constexpr int kFar = 3;
// A tile's start and end (its rows of q and o, the empty pipeline) take about
// as long as this many steps; the ranges count them.  (5, 8, 12: 168 prompts of
// 189 tokens 89, 94 and 92 us, one of 8192 on a cool card 601, 608 and 624.)
constexpr int kTileSteps = 8;
struct PrePlan {
  int q, k, v, bars, scales, tok, parts, misc, start, len, nq, sum, total;
};
constexpr int kBars = 2 * kRing + 18;
__host__ __device__ inline PrePlan pre_plan(int B) {
  PrePlan p;
  p.q = 0;
  p.k = 2 * kQGroup;
  p.v = p.k + kRing * kTileBytes;
  p.bars = p.v + kRing * kTileBytes;
  p.scales = (p.bars + kBars * 8 + 15) / 16 * 16;
  p.tok = p.scales + kScaleRing * (int)sizeof(StepScales);
  p.parts = p.tok + kScaleRing * kTokBytes;
  p.misc = p.parts + 8 * 48;
  p.start = p.misc + 64;
  p.sum = p.start + (B + 1) * 8;
  p.len = p.sum + B * 4;
  p.nq = p.len + B * 4;
  p.total = (p.nq + B * 4 + 15) / 16 * 16;
  return p;
}

// The line, in shared memory: per sequence its start, what one KV head takes
// of it, its length and its queries.
struct Line {
  const long long* start;
  const int *sum, *len, *nq;
  int B, G;
  const QuantAttnArgs* a;
};
// Steps that group gr of row tile rt of sequence b needs.
__device__ __forceinline__ int group_steps(const Line& n, int b, int rt, int gr) {
  const int R = n.nq[b] * n.G, r = rt * kTileRows + gr * 128;
  if (r >= R) return 0;
  const int maxpos = n.len[b] - n.nq[b] + div_group(*n.a, min(R - 1, r + 127));
  return maxpos < 0 ? 0 : maxpos / kStepKeys + 1;
}
// Steps of a tile (its last group with rows needs most): one at least for
// queries that see nothing (their zeros).
__device__ __forceinline__ int tile_steps(const Line& n, int b, int rt) {
  const int R = n.nq[b] * n.G, r = rt * kTileRows;
  if (r >= R) return 0;
  return max(1, group_steps(n, b, rt, r + 128 < R ? 1 : 0));
}
// What a tile takes of the line.
__device__ __forceinline__ int tile_length(const Line& n, int b, int rt) {
  const int s = tile_steps(n, b, rt);
  return s ? s + kTileSteps : 0;
}

// A part of a tile: steps [j0, j1) of `steps` in this CTA's range (j1 <= j0:
// none), `first` the line's index of its step 0; nt0, nt1: steps that the
// groups need.
struct PrePart {
  int b, h, r0, steps, j0, j1, nt0, nt1;
  long long first;
  __device__ __forceinline__ int ntile(int g) const { return g ? nt1 : nt0; }
};

// The rest of a part whose place (b, h, r0) and first are known.
__device__ __forceinline__ void fill_part(const Line& n, PrePart& p, long long x, long long hi) {
  const int rt = p.r0 / kTileRows;
  p.nt0 = group_steps(n, p.b, rt, 0);
  p.nt1 = group_steps(n, p.b, rt, 1);
  p.steps = max(1, max(p.nt0, p.nt1));
  p.j0 = (int)max(0ll, x - p.first);
  p.j1 = (int)(min(hi, p.first + p.steps) - p.first);
}
// The part that place x of the line belongs to; a whole warp calls, its lanes
// look at 32 heads or tiles at a time.
__device__ __forceinline__ PrePart find_part(const Line& n, long long x, long long hi) {
  const int lane = threadIdx.x & 31;
  PrePart p;
  int l = 0, r = n.B;
#pragma unroll 1
  while (r - l > 1) {
    const int mid = (l + r) >> 1;
    if (n.start[mid] <= x) l = mid; else r = mid;
  }
  p.b = l;
  long long in = x - n.start[l];
  const int sum = n.sum[l];
  p.h = 0;
#pragma unroll 1
  for (;; p.h += 32, in -= 32ll * sum) {
    const uint32_t past = __ballot_sync(0xffffffffu, (lane + 1ll) * sum > in);
    if (past) {
      const int w = __ffs(past) - 1;
      p.h += w;
      in -= (long long)w * sum;
      break;
    }
  }
  int left = (int)in, rt = 0;
#pragma unroll 1
  for (;; rt += 32) {
    const int s = tile_length(n, l, rt + lane);
    int incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, incl > left);
    if (past) {
      const int w = __ffs(past) - 1;
      left -= __shfl_sync(0xffffffffu, incl - s, w);
      rt += w;
      break;
    }
    left -= __shfl_sync(0xffffffffu, incl, 31);
  }
  p.r0 = rt * kTileRows;
  p.first = x - left + kTileSteps;
  fill_part(n, p, x, hi);
  return p;
}
// The part after p, at the place x where p's tile ends on the line.
__device__ __forceinline__ PrePart next_part(const Line& n, const PrePart& p, long long x,
                                             long long hi, int H) {
  PrePart q = p;
  q.r0 += kTileRows;
  if (q.r0 >= n.nq[q.b] * n.G) {
    q.r0 = 0;
    if (++q.h == H) {
      q.h = 0;
      do ++q.b; while (n.sum[q.b] == 0);
    }
  }
  q.first = x + kTileSteps;
  fill_part(n, q, x, hi);
  return q;
}

// The CTA whose range holds the place before x.
__device__ __forceinline__ int last_cta(const Line& n, long long x) {
  const long long total = *static_cast<const volatile long long*>(&n.start[n.B]);
  const int C = (int)min((long long)gridDim.x, total);
  const long long per = total / C, extra = total - per * C, big = extra * (per + 1);
  return (int)(x <= big ? (x - 1) / (per + 1) : extra + (x - 1 - big) / per);
}

template <bool kE4M3>
__global__ void __launch_bounds__(kPreThreads, 1) quant_prefill_kernel(QuantAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  const QuantView& c = a.c;
  const PrePlan pl = pre_plan(c.B);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + pl.bars);
  // sfull, pfull: [group][S buffer]; odone: a step's P V ended, ofull: a part's
  uint64_t *full = bars, *empty = full + kRing, *qfull = empty + kRing, *sfull = qfull + 2, *pfull = sfull + 4, *odone = pfull + 4,
           *ofull = odone + 2, *oempty = ofull + 2, *mdone = oempty + 2, *tokfull = mdone + 1;
  StepScales* scales = reinterpret_cast<StepScales*>(sm + pl.scales);
  PrePart* parts = reinterpret_cast<PrePart*>(sm + pl.parts);  // [8]
  long long* start = reinterpret_cast<long long*>(sm + pl.start);
  int* ssum = reinterpret_cast<int*>(sm + pl.sum);
  int* slen = reinterpret_cast<int*>(sm + pl.len);
  int* snq = reinterpret_cast<int*>(sm + pl.nq);
  volatile int* fail = reinterpret_cast<volatile int*>(sm + pl.misc);
  uint32_t* taddr = reinterpret_cast<uint32_t*>(sm + pl.misc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *fail = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], 4);   // the converters' warps
      mbar_init(&empty[i], 2);  // both groups' issuers
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 2);  // the products' commit and the issuer itself
      mbar_init(&pfull[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 128);
      mbar_init(&odone[i], 1);
      mbar_init(&ofull[i], 1);
      mbar_init(&oempty[i], 128);
    }
    mbar_init(mdone, 2);
    mbar_init(tokfull, 128);
    mbar_fence_init();
  }
  pdl_trigger();
  pdl_wait();
  for (int b = tid; b < c.B; b += kPreThreads) {
    slen[b] = quant_len(c, b);
    snq[b] = quant_queries(a, b);
  }
  if (warp == 12) {
    tmem_alloc(taddr, 512);
    tmem_relinquish();
  }
  __syncthreads();
  const Line line = {start, ssum, slen, snq, c.B, a.G, &a};
  // a warp per sequence: the steps of its tiles
#pragma unroll 1
  for (int b = warp; b < c.B; b += kPreThreads / 32) {
    int s = 0;
#pragma unroll 1
    for (int rt = lane; rt * kTileRows < snq[b] * a.G; rt += 32) s += tile_length(line, b, rt);
    s = (int)__reduce_add_sync(0xffffffffu, (uint32_t)s);
    if (lane == 0) ssum[b] = s;
  }
  __syncthreads();
  if (warp == 0) {
    const int per = (c.B + 31) / 32, b0 = min(c.B, lane * per), b1 = min(c.B, b0 + per);
    long long own = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) own += (long long)ssum[b] * c.H;
    long long incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    long long e = incl - own;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      start[b] = e;
      e += (long long)ssum[b] * c.H;
    }
    if (lane == 31) start[c.B] = incl;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *taddr;
  long long lo = 0, hi = 0;
  {
    const long long total = start[c.B];
    const int C = (int)min((long long)gridDim.x, total);
    if ((int)blockIdx.x < C) {  // the first CTAs of a remainder take one more
      const long long per = total / C;
      const int extra = (int)(total - per * C);
      lo = blockIdx.x * per + min((int)blockIdx.x, extra);
      hi = lo + per + ((int)blockIdx.x < extra ? 1 : 0);
    }
  }

  // the parts of this range, one after the other: `x` is where the part begins
  auto advance = [&](PrePart& p, long long& x) {
    x = p.first + max(p.j1, 0);
    if (x < hi) p = next_part(line, p, x, hi, c.H);
  };

  if (warp < 8) {
    // ================ softmax
    const int gr = warp >> 2, row = tid & 127;  // TMEM lane = row of the group
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + gr * 128, tO = tmem + lane_base + 256 + gr * 128;
    uint8_t* qs = sm + pl.q + gr * kQGroup;
    int4* cuts = reinterpret_cast<int4*>(static_cast<uint8_t*>(a.ws) + pre_cuts(gridDim.x));
    if (tid == 0) cuts[blockIdx.x] = make_int4(0, 0, 0, -1);
    uint32_t ns = 0;          // parity of the S tiles seen, a bit per buffer
    uint32_t nd = 0, np = 0;  // steps of this group in the parts before, and such parts
    uint32_t done = 0;        // steps of the parts before
    // the part lives in shared memory: no registers for it in the loops below
    if (lo < hi) {
      const PrePart p = find_part(line, lo, hi);
      if (lane == 0) parts[warp] = p;
      __syncwarp();
    }
    for (long long x = lo; x < hi;) {
      float m = -INFINITY, l = 0.f, dv = -INFINITY, fcol = 0.f;
      int pos;
      {
        const PrePart p = parts[warp];
        const int nq = snq[p.b], pos0 = slen[p.b] - nq;
        const int rr = p.r0 + gr * 128 + row;
        pos = rr < nq * a.G ? pos0 + div_group(a, rr) : 0x7fffffff;
        const int minpos = pos0 + div_group(a, p.r0 + gr * 128);
        // this group's steps here, and those but the open block's
        int n = min(p.j1, p.ntile(gr)) - p.j0;
        const uint32_t steps = max(0, min(p.j1, max(p.nt0, p.nt1)) - p.j0);
        if (n > 0) {
        // ---- q: the warp copies its 32 rows as they are to where they belong
        // (two rows at a time, chunks of 16 bytes turned by the row), each
        // thread then turns its own row into fp16 with its largest element in
        // [2^14, 2^15)
        {
          const int w0 = row & ~31, R = nq * a.G, ch = lane & 15;
          int r = p.r0 + gr * 128 + w0 + (lane >> 4);
          const int tk = div_group(a, r);
          int hd = r - tk * a.G;
          const __nv_bfloat16* src = a.q + p.b * a.qs + (long long)(p.h * a.G + hd) * a.qh +
                                     (long long)tk * a.qt + 8 * ch;
          const long long two = 2 * a.qh, wrap = a.qt - a.G * a.qh;
          const uint32_t to = smem_u32(qs + (ch >> 3) * kQHalf + (w0 + (lane >> 4)) * 128);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const int rw = i + (lane >> 4);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             to + i * 128 + (((ch & 7) ^ (rw & 7)) << 4)),
                         "l"(r < R ? src : a.q), "r"(r < R ? 16 : 0)
                         : "memory");
            r += 2;
            src += two;
            hd += 2;
            if (hd >= a.G) {
              hd -= a.G;
              src += wrap;
            }
            if (hd >= a.G) {  // G is 1
              hd -= a.G;
              src += wrap;
            }
          }
          cp_async_commit();
          cp_async_wait<0>();
          __syncwarp();
          uint8_t* mine = qs + row * 128;
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(mine + (i >> 3) * kQHalf + (((i & 7) ^ (row & 7)) << 4));
            mx = __vmaxu2(mx, w.x & 0x7fff7fffu);
            mx = __vmaxu2(mx, w.y & 0x7fff7fffu);
            mx = __vmaxu2(mx, w.z & 0x7fff7fffu);
            mx = __vmaxu2(mx, w.w & 0x7fff7fffu);
          }
          mx = max(mx >> 16, mx & 0xffffu);
          int e = (int)(mx >> 7) - 127;
          e = mx == 0 || e == 128 ? 14 : max(e, -100);
          const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23) * (a.scale < 0.f ? -1.f : 1.f);
          fcol = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * (fabsf(a.scale) * kLog2e);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint4* at = reinterpret_cast<uint4*>(mine + (i >> 3) * kQHalf + (((i & 7) ^ (row & 7)) << 4));
            const uint4 w = *at;
            *at = make_uint4(pack_h2(bf_lo(w.x) * up, bf_hi(w.x) * up),
                             pack_h2(bf_lo(w.y) * up, bf_hi(w.y) * up),
                             pack_h2(bf_lo(w.z) * up, bf_hi(w.z) * up),
                             pack_h2(bf_lo(w.w) * up, bf_hi(w.w) * up));
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&qfull[gr]);
        n = min(n, slen[p.b] / kQBlock - p.j0);
        for (int i = 0; i < n; ++i) {
          const int base = (p.j0 + i) * kStepKeys, sb = i & 1;
          if (!quant_wait_warp(&sfull[2 * gr + sb], (ns >> sb) & 1, fail, lane)) break;
          ns ^= 1u << sb;
          tc_fence_after();
          const uint32_t tSb = tS + 64 * sb;
          uint32_t s[64];
          tmem_ld32<0>(tSb, s);
          tmem_ld32<32>(tSb + 32, s);
          const StepScales sc = scales[(done + i) % kScaleRing];
          // s_v = 2^ev fv, 1 <= fv < 2 (a NaN stays in fv)
          const bool vnan = sc.sv != sc.sv;
          const float ev = vnan ? 0.f : (float)((int)(__float_as_uint(sc.sv) >> 23) - 127);
          const float fv = vnan ? sc.sv : __uint_as_float((__float_as_uint(sc.sv) & 0x7fffffu) | 0x3f800000u);
          const float f = fcol * sc.sk;
          tmem_wait_ld32<0>(s);
          tmem_wait_ld32<32>(s);
          const bool edge = base + kStepKeys - 1 > minpos || !sc.ok;
          // twice: masks cost every element two instructions and more
          float x0 = -INFINITY, x1 = -INFINITY;
          if (edge) {
            const int last = sc.ok ? pos - base : -1;
#pragma unroll
            for (int k = 0; k < 64; ++k) {
              if (k > last) s[k] = 0xff800000u;
              x0 = fmaxf(x0, __uint_as_float(s[k]));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
              x0 = fmaxf(x0, fmaxf(__uint_as_float(s[k]), __uint_as_float(s[k + 1])));
              x1 = fmaxf(x1, fmaxf(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])));
            }
            x0 = fmaxf(x0, x1);
          }
          const float mn = x0 == -INFINITY ? x0 : floorf(x0 * fabsf(f));
          if (mn > m + kLazy) {  // also from -inf
            const float sh = m - mn;
            l *= ex2_approx(sh);
            dv += sh;
            m = mn;
          }
          const float ref = or_zero(m), en = mn - ref + ev;
          const bool grow = en > dv + kLazy;
          if (__any_sync(0xffffffffu, grow)) {
            const float cr = grow ? ex2_approx(dv - en) : 1.f;
            if (grow) dv = en;
            if (__any_sync(0xffffffffu, fabsf(ref) > kWideRef)) fcol = -fabsf(fcol);
            // the step before has been added; this one waits for P
            if (i > 0 && quant_wait_warp(&odone[gr], (nd + i - 1) & 1, fail, lane)) {
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
          }
          const float dref = or_zero(dv);
          // 2^(m - M') s_v 2^kBoostLog
          const float wm = fv * ex2_approx(ev - dref + kBoostLog);
          const float2 w2 = make_float2(wm, wm), f2 = make_float2(f, f), nref = make_float2(-ref, -ref);
          float2 sum = make_float2(0.f, 0.f);
          auto weigh = [&](auto edge_c) {
            constexpr bool kEdge = decltype(edge_c)::value;
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              uint32_t pk[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int k = 16 * q4 + 2 * e;
                float2 v = nref;
                fma2(v, make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), f2);
                v.x = ex2_approx(v.x);
                v.y = ex2_approx(v.y);
                float2 w = mul2(v, w2);
                if constexpr (kEdge) {  // a NaN scale does not reach what is not seen
                  if (s[k] == 0xff800000u) v.x = w.x = 0.f;
                  if (s[k + 1] == 0xff800000u) v.y = w.y = 0.f;
                }
                sum = add2(sum, v);
                pk[e] = pack_h2(w.x, w.y);
              }
              tmem_st8(tSb + 8 * q4, pk);
            }
          };
          if (fcol < 0.f || sc.ok == kWideStep)
            sum.x = weigh_wide(tSb, tSb, kStepKeys, fabsf(f), !edge ? kStepKeys : sc.ok ? pos - base : -1, ref,
                               ev - dref + kBoostLog, fv);
          else if (edge)
            weigh(std::true_type());
          else
            weigh(std::false_type());
          l += sum.x + sum.y;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&pfull[2 * gr + sb]);
        }
        }
        done += steps;
      }
      // ---- the open block, and the row's sums (no registers for its place in the
      // loop above)
      PrePart p = parts[warp];
      const int n = min(p.j1, p.ntile(gr)) - p.j0, nopen = slen[p.b] / kQBlock - p.j0;
      if (nopen < n) {
        const int sb = nopen & 1, at = (done - 1) % kScaleRing;
        const uint32_t tSb = tS + 64 * sb;
        if (quant_wait_warp(&sfull[2 * gr + sb], (ns >> sb) & 1, fail, lane)) {
          ns ^= 1u << sb;
          tc_fence_after();
          const RowState r = open_step({m, l, dv}, tSb, tSb, tO, kStepKeys, sm + pl.tok + at * kTokBytes,
                                       fabsf(fcol), pos - (p.j0 + nopen) * kStepKeys,
                                       nopen > 0 ? &odone[gr] : nullptr, (nd + nopen - 1) & 1, fail);
          m = r.m;
          l = r.l;
          dv = r.dv;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&pfull[2 * gr + sb]);
        }
      }
      if (p.j1 > p.j0) {
      float4* records = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.ws) + pre_records(gridDim.x));
      const bool whole = p.j0 == 0 && p.j1 == p.steps;
      const float4 st = make_float4(m, l, dv, 0.f);
      float4* rec = records + ((size_t)2 * blockIdx.x + (p.j0 == 0 ? 1 : 0)) * kPreRecord + gr * 128 + row;
      const float fin = l == 0.f ? 0.f : ex2_approx(dv - kBoostLog) / l;
      if (n > 0) {
        // (a barrier of its own: of odone's phases the last two may still be
        // open here, and a wait by parity tells only one from the one before)
        quant_wait_warp(&ofull[gr], np & 1, fail, lane);
        ++np;
        nd += n;
        tc_fence_after();
      }
#pragma unroll 2
      for (int q4 = 0; q4 < 4; ++q4) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32<0>(tO + 32 * q4, o);
          tmem_wait_ld32<0>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (whole) {
          // rows as bf16 exactly where the same rows of q were (its products
          // have ended): another warp may have its next q in place already
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = l == 0.f ? 0u
                              : pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * fin,
                                            __uint_as_float(o[8 * e + 2 * k + 1]) * fin);
            *reinterpret_cast<uint4*>(qs + (q4 >> 1) * kQHalf + row * 128 +
                                      (((4 * (q4 & 1) + e) ^ (row & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            rec[(size_t)(1 + 8 * q4 + e) * kTileRows] =
                make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        }
      }
      if (n > 0) {
        tc_fence_before();
        mbar_arrive(&oempty[gr]);
      }
      if (whole) {
        __syncwarp();
        // two whole rows of the warp's 32 at a time
        const int w0 = row & ~31, R = snq[p.b] * a.G, ch = lane & 15;
        int r = p.r0 + gr * 128 + w0 + (lane >> 4);
        const int tk = div_group(a, r);
        int hd = r - tk * a.G;
        __nv_bfloat16* dst = a.o + p.b * a.os + (long long)(p.h * a.G + hd) * a.oh +
                             (long long)tk * a.ot + 8 * ch;
        const long long two = 2 * a.oh, wrap = a.ot - a.G * a.oh;
        const uint8_t* from = qs + (ch >> 3) * kQHalf + (w0 + (lane >> 4)) * 128;
#pragma unroll 8
        for (int i = 0; i < 32; i += 2) {
          const int rw = i + (lane >> 4);
          if (r < R)
            *reinterpret_cast<uint4*>(dst) =
                *reinterpret_cast<const uint4*>(from + i * 128 + (((ch & 7) ^ (rw & 7)) << 4));
          r += 2;
          dst += two;
          hd += 2;
          if (hd >= a.G) {
            hd -= a.G;
            dst += wrap;
          }
          if (hd >= a.G) {  // G is 1
            hd -= a.G;
            dst += wrap;
          }
        }
      }
      if (!whole) {
        rec[0] = st;
        // a tile that begins in this CTA and goes on in others: for the merge
        if (tid == 0 && p.j0 == 0)
          cuts[blockIdx.x] = make_int4(p.b, p.h, p.r0, last_cta(line, p.first + p.steps));
      }
      }
      advance(p, x);
      __syncwarp();
      if (lane == 0) parts[warp] = p;
      __syncwarp();
    }
  } else if (warp < 12) {
    // ================ converters
    const int ct = tid - 256;
    const int sub = ct >> 2, ch = ct & 3;  // 32 rows x 4 chunks a round
    uint4 kr[4], vr[4];
    uint32_t cnt = 0, opens = 0;  // steps converted, and open blocks
    const uint8_t* slab;  // slab of a step (nullptr: open, or out of range)
    float2 nsc;           // its scales
    int next = 0, far = 0;  // table entries of the steps j + 1 and j + kFar
    auto entry = [&](const PrePart& p, int j) {
      return (j + 1) * kQBlock <= slen[p.b] ? c.bt[(size_t)p.b * c.maxp + j] : -1;
    };
    auto page = [&](const PrePart& p, int j, int id) {
      slab = nullptr;
      if ((j + 1) * kQBlock <= slen[p.b]) {
        if (id >= 0 && id < c.num_pages) {
          slab = c.pages + ((size_t)id * c.H + p.h) * kQSlab;
          nsc = __ldg(reinterpret_cast<const float2*>(slab + 2 * kQSide));
        } else if (ct == 0) {
          quant_error(c, kErrBadPage);
        }
      }
    };
    // keys: token 32 (i / 2) + sub, chunk ch + 4 (i % 2); a quarter warp then
    // writes two rows' chunks of one half: no bank conflicts
    auto load_k = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        kr[i] = slab ? __ldg(reinterpret_cast<const uint4*>(
                           slab + quant_k_chunk(32 * (i >> 1) + sub, ch + 4 * (i & 1))))
                     : make_uint4(0, 0, 0, 0);
    };
    auto load_v = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vr[i] = slab ? __ldg(reinterpret_cast<const uint4*>(slab + kQSide + (32 * i + sub) * kQBlock + ch * 16))
                     : make_uint4(0, 0, 0, 0);
    };
    bool live = true;
    PrePart p;
    if (lo < hi) p = find_part(line, lo, hi);
    for (long long x = lo; x < hi && live; advance(p, x)) {
      const int L = slen[p.b], last = max(p.nt0, p.nt1);
      const int j1 = min(p.j1, last), jf = min(j1, L / kQBlock);  // full blocks; then the open one
      bool low = false;
      if (p.j0 < jf) {
        page(p, p.j0, entry(p, p.j0));
        load_k();
        load_v();
        next = entry(p, p.j0 + 1);
        far = entry(p, p.j0 + kFar);
      }
      for (int j = p.j0; j < jf; ++j) {
        const int buf = cnt % kRing;
        uint8_t* kb = sm + pl.k + buf * kTileBytes;
        uint8_t* vb = sm + pl.v + buf * kTileBytes;
        const bool there = slab != nullptr;
        float sk = 1.f, sv = 1.f;
        if (there) {
          sk = nsc.x;
          sv = nsc.y;
        }
        if (cnt >= kRing && !quant_wait_warp(&empty[buf], (cnt / kRing - 1) & 1, fail, lane)) { live = false; break; }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 32 * (i >> 1) + sub;
          put_codes<kE4M3>(kb + (i & 1) * kKHalf + row * 128, row, 2 * ch, kr[i]);
        }
        if (j + 1 < jf) {
          page(p, j + 1, next);
          load_k();
          next = entry(p, j + 2);
          if (ct == 0) {
            if (j + kFar < jf && far >= 0 && far < c.num_pages)
              l2_prefetch(c.pages + ((size_t)far * c.H + p.h) * kQSlab, kQSlab);
            far = entry(p, j + 1 + kFar);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          put_codes<kE4M3>(vb + (32 * i + sub) * 128, 32 * i + sub, 2 * ch, vr[i]);
        if (j + 1 < jf) load_v();
        if (ct == 0) {
          StepScales* s = &scales[cnt % kScaleRing];
          s->sk = sk;
          s->sv = sv;
          s->ok = there ? wide_step(sv, low) : 0;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[buf]);
        ++cnt;
      }
      if (live && jf < j1) {  // no pages' registers are held here
        const int buf = cnt % kRing, nt = L - jf * kQBlock;
        uint8_t* tok = sm + pl.tok + cnt % kScaleRing * kTokBytes;
        const __nv_bfloat16 *kt = quant_tail(c, p.b, p.h, 0, jf * kQBlock),
                            *vt = quant_tail(c, p.b, p.h, 1, jf * kQBlock);
        if (cnt >= kRing && !quant_wait_warp(&empty[buf], (cnt / kRing - 1) & 1, fail, lane)) { live = false; break; }
        open_value_exponents(vt, nt, ct, tok);
        mbar_arrive(tokfull);
        open_keys(kt, nt, sm + pl.k + buf * kTileBytes, ct, tok);
        if (!quant_wait_warp(tokfull, opens & 1, fail, lane)) { live = false; break; }
        ++opens;
        open_values(vt, nt, sm + pl.v + buf * kTileBytes, ct, tok);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[buf]);
        ++cnt;
      }
    }
  } else {
    // ================ products
    if (warp < 14) {
      const int gr = warp - 12;
      const uint32_t qa = desc_lo(smem_u32(sm + pl.q)) + gr * (kQGroup >> 4),
                     k0 = desc_lo(smem_u32(sm + pl.k)), v0 = desc_lo(smem_u32(sm + pl.v)),
                     dS = tmem + gr * 128, dO = tmem + 256 + gr * 128;
      // steps of the tiles; parity of this group's P, a bit per buffer; its parts
      uint32_t cnt = 0, np = 0, ns = 0;
      bool live = true;
      PrePart p;
      if (lo < hi) p = find_part(line, lo, hi);
      for (long long x = lo; x < hi && live; advance(p, x)) {
        const int j1 = min(p.j1, max(p.nt0, p.nt1)), n = max(0, j1 - p.j0);
        const int mine = max(0, min(p.j1, p.ntile(gr)) - p.j0);  // this group's steps
        bool ok = true;
        if (n > 0 && elect_one()) {
          // S of step i; the issuer's own arrival hands on what it has seen of
          // the converters (the scales)
          auto scores = [&](int i) {
            const uint32_t d = dS + (i & 1) * 64, kb = k0 + ((cnt + i) % kRing) * (kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ss(d, qa + (((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4),
                     kb + (((kk >> 2) * kKHalf + (kk & 3) * 32) >> 4), kIdescS, kk > 0 ? 1u : 0u);
            tc_commit(&sfull[2 * gr + (i & 1)]);
            mbar_arrive(&sfull[2 * gr + (i & 1)]);
          };
          auto sums = [&](int i) {
            const uint32_t pa = dS + (i & 1) * 64, vb = v0 + ((cnt + i) % kRing) * (kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(dO, pa + 8 * kk, vb + ((kk * 32) >> 4), kIdescO, kk > 0 || i > 0 ? 1u : 0u);
            tc_commit(&odone[gr]);
          };
          // A look at a barrier takes 200 clocks and more here (the tensor
          // cores read shared memory most of the time), so the tile of the
          // scores after these is looked at before this step's products are
          // issued, and waited for only if it was not there yet.
          auto tile = [&](int i, bool wait) {
            uint64_t* bar = &full[(cnt + i) % kRing];
            const uint32_t ph = ((cnt + i) / kRing) & 1;
            return wait ? quant_wait(bar, ph, fail) : mbar_try_wait(bar, ph);
          };
          if (mine > 0) ok = quant_wait(&qfull[gr], ns & 1, fail);
          for (int i = 0; i < 2 && i < n && ok; ++i) {
            ok = tile(i, true);
            if (!ok) break;
            tc_fence_after();
            if (i < mine) scores(i);
          }
          bool seen = false;
          for (int i = 0; i < n && ok; ++i) {
            // an issuer whose group has ended keeps pace with the tiles: each
            // is given back by both, once
            if (!seen && i + 2 < n) ok = tile(i + 2, true);
            if (ok && i < mine) {
              ok = quant_wait(&pfull[2 * gr + (i & 1)], ((np >> (i & 1)) ^ (i >> 1)) & 1, fail);
              // O's last sums have been read
              if (ok && i == 0 && ns > 0) ok = quant_wait(&oempty[gr], (ns - 1) & 1, fail);
            }
            if (!ok) break;
            seen = i + 3 < n && tile(i + 3, false);
            if (i < mine) {
              tc_fence_after();
              sums(i);
              if (i == mine - 1) tc_commit(&ofull[gr]);
              if (i + 2 < mine) scores(i + 2);
            }
            tc_commit(&empty[(cnt + i) % kRing]);
          }
        }
        live = __all_sync(0xffffffffu, ok);
        cnt += n;
        if (mine > 0) {
          np ^= (((mine + 1) >> 1) & 1) | (((mine >> 1) & 1) << 1);
          ++ns;
        }
      }
      // every product has ended before TMEM is freed
      if (lo < hi && elect_one()) {
        tc_commit(mdone);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(mdone, 0) && global_ns() - t0 < kTcTimeoutNs) {
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(*static_cast<volatile uint32_t*>(taddr), 512);
  if (tid == 0 && *fail) quant_error(c, kErrTimeout);
}

// The parts of the tiles that the ranges' borders cut, folded in order: one
// CTA per (CTA in which the tile begins, 8 rows), a warp per row, 4 dims a
// lane.  (Folded by the last CTA to arrive instead, one SM read all parts of
// a tile: 127 us for 64 queries over 16K where the products take 25.)
__global__ void __launch_bounds__(256) quant_merge_kernel(QuantAttnArgs a, int C) {
  pdl_trigger();
  pdl_wait();
  const int c0 = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 cut = __ldcg(reinterpret_cast<const int4*>(static_cast<uint8_t*>(a.ws) + pre_cuts(C)) + c0);
  if (cut.w < 0) return;
  const int b = cut.x, h = cut.y, row = blockIdx.y * 8 + warp, rr = cut.z + row;
  if (rr >= quant_queries(a, b) * a.G) return;
  const float4* records = reinterpret_cast<const float4*>(static_cast<uint8_t*>(a.ws) + pre_records(C)) + row;
  auto part = [&](int cc) { return records + ((size_t)2 * cc + (cc == c0 ? 1 : 0)) * kPreRecord; };
  float M = -INFINITY, Z = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int cc = c0; cc <= cut.w; ++cc) {
    const float4 t = __ldcg(part(cc)), s = __ldcg(part(cc) + (size_t)(1 + lane) * kTileRows);
    if (t.x == -INFINITY && t.y == 0.f) continue;  // saw nothing (a NaN sum is something)
    const float mn = fmaxf(M, t.x), mr = or_zero(mn), a0 = M - mr, a1 = t.x - mr;
    const float z0 = Z + a0, z1 = t.z + a1, zn = fmaxf(z0, z1), zr = or_zero(zn);  // M' from mn
    l = l * ex2_approx(a0) + t.y * ex2_approx(a1);
    const float f0 = ex2_approx(z0 - zr), f1 = ex2_approx(z1 - zr);
    M = mn;
    Z = zn;
    o.x = o.x * f0 + s.x * f1;
    o.y = o.y * f0 + s.y * f1;
    o.z = o.z * f0 + s.z * f1;
    o.w = o.w * f0 + s.w * f1;
  }
  const float f = l == 0.f ? 0.f : ex2_approx(Z - kBoostLog) / l;
  __nv_bfloat16* dst = a.o + b * a.os + (long long)(h * a.G + rr % a.G) * a.oh + (long long)(rr / a.G) * a.ot;
  *reinterpret_cast<uint2*>(dst + 4 * lane) =
      l == 0.f ? make_uint2(0, 0)
               : make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
}

}  // namespace

int quant_merge_launch(const QuantAttnArgs& a, int C, int rows, cudaStream_t st) {
  QuantAttnArgs args = a;
  void* p[] = {&args, &C};
  return launch_pdl((const void*)quant_merge_kernel, dim3(C, (rows + 7) / 8), dim3(256), 0, st, p) ==
                 cudaSuccess
             ? LRKV_OK
             : LRKV_ERR_CUDA;
}

size_t quant_prefill_workspace(int C) {
  return pre_records(C) + (size_t)C * 2 * kPreRecord * 16;
}

int quant_prefill_launch(const QuantAttnArgs& a, const DevInfo& info, cudaStream_t st) {
  const void* fn = a.c.e4m3 ? (const void*)quant_prefill_kernel<true>
                            : (const void*)quant_prefill_kernel<false>;
  const int smem = pre_plan(a.c.B).total + 1024;
  if (smem > info.optin) return LRKV_ERR_UNSUPPORTED;
  const int rc = prepare_kernel(fn, true);
  if (rc != LRKV_OK) return rc;
  QuantAttnArgs args = a;
  void* p[] = {&args};
  if (launch_pdl(fn, dim3(info.sms), dim3(kPreThreads), smem, st, p) != cudaSuccess)
    return LRKV_ERR_CUDA;
  return quant_merge_launch(a, info.sms, kTileRows, st);
}

}  // namespace lrkv
