// Attention of 17 to 128 query rows per KV head over the 8-bit full-rank cache
// (drafted tokens, short follow-ups): as many bytes as one row takes, more
// than quant_decode.cu's registers hold (a warp there has the sums of all
// rows), too few rows to fill a tile of quant_prefill.cu.
//
// The mathematics is quant_prefill.cu's.  The 128 rows of a tcgen05 tile are
// REP copies of up to 128 / REP query rows; S = Q K^T of a page then stands
// REP times in TMEM, and copy c takes the page's tokens 64 c / REP .. alone:
// the exponentials of a few rows are spread over all four sub-partitions, and
// every thread keeps a running maximum and sum of its own.  P is zero outside
// a copy's tokens (written once, at the start), so O of copy c is the sum over
// its tokens; the copies and the two groups are added at the end of a unit.
//
// What bounds it: the latency of a page's way through the roles (codes, tile,
// S, P, O).  Two pages are under way at a time and one leaves every 0.85 us,
// 1.25 with 128 rows; its bytes would take 0.37.  4 x 8 heads x 16,384 tokens
// (134 MB, caches in turn, 1,930 to 1,965 MHz) with 20 rows 54 us, 32 rows 56,
// 64 rows 59, 128 rows 78.
//
// Persistent, one CTA per SM, 18 warps, the pages of all units dealt evenly:
//  * warp 17: one bulk copy per page slab into a ring of NR (44 bytes a
//    nanosecond and SM from HBM want 60 KB and more in flight);
//  * warps 8-11 and 12-15: converters of keys and of values, from the ring to
//    fp16 tiles (one set for both waited for P V before it turned to the next
//    keys: 2900 clocks a page);
//  * warp 16, one lane: Q K^T and P V;
//  * warps 0-3 and 4-7: softmax of even and odd pages, S, P and O of their own.
#include <type_traits>

#include "quant_tc.cuh"

namespace lrkv {

namespace {

constexpr int kFewThreads = 576;
constexpr int kTiles = 3;        // fp16 tiles of keys, and of values, in flight
constexpr int kFewScales = 8;    // a step's scales are read until its P is written
// What a unit's start and end take, in steps (as in quant_prefill.cu): 6, 9,
// 12 and 16 here: 16 x 1024 tokens with 128 rows 50.6, 49.9, 47.8 and 46.0 us,
// 4 x 16384 with 64 62.7, 61.3, 60.9 and 61.2.
constexpr int kUnitSteps = 12;
constexpr uint32_t kTmemP = 128, kTmemO = 256;

struct FewPlan {
  int q, k, v, ml, rowst, fc, scales, tok, vtok, bars, rawok, misc, raw, start, len, nq, total;
};
constexpr int kFewBars = 4 * kTiles + 2 * 8 + 2 + 10;
__host__ __device__ inline FewPlan few_plan(int NR, int B) {
  FewPlan p;
  p.q = 0;
  p.k = 128 * 256;
  p.v = p.k + kTiles * kTileBytes;
  p.ml = p.v + kTiles * kTileBytes;
  p.rowst = p.ml + 256 * 16;
  p.fc = p.rowst + 128 * 16;
  p.scales = p.fc + 128 * 4;
  p.tok = p.scales + kFewScales * (int)sizeof(StepScales);
  p.vtok = p.tok + kFewScales * kTokBytes;
  p.bars = p.vtok + 2 * kTokValues;
  p.rawok = p.bars + kFewBars * 8;
  p.misc = p.rawok + 8 * 4;
  p.raw = (p.misc + 16 + 127) / 128 * 128;
  p.start = p.raw + NR * kQSlab;
  p.len = p.start + (B + 1) * 4;
  p.nq = p.len + B * 4;
  p.total = p.nq + B * 4;
  return p;
}

// A part of a unit: steps [j0, j1) of `steps` in this CTA's range (j1 <= j0:
// none), `first` the line's index of its step 0.
struct FewPart {
  int b, h, steps, j0, j1, first;
};

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t addr, uint32_t (&s)[N]) {
  if constexpr (N == 16) {
    tmem_ld16_async(addr, s);
  } else {
    tmem_ld32<0>(addr, s);
    if constexpr (N == 64) tmem_ld32<32>(addr + 32, s);
  }
}
template <int N>
__device__ __forceinline__ void wait_cols(uint32_t (&s)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(s[i]));
}

template <bool kE4M3, int REP>
__global__ void __launch_bounds__(kFewThreads, 1) quant_few_kernel(QuantAttnArgs a, int NR) {
  constexpr int CW = 64 / REP;        // a thread's columns of S
  constexpr int kCopy = 128 / REP;    // rows of a copy
  extern __shared__ __align__(1024) uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  const QuantView& c = a.c;
  const FewPlan pl = few_plan(NR, c.B);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + pl.bars);
  uint64_t *kfull = bars, *kempty = kfull + kTiles, *vfull = kempty + kTiles, *vempty = vfull + kTiles,
           *rawfull = vempty + kTiles, *rawempty = rawfull + 8, *sfull = rawempty + 8,
           *pfull = sfull + 2, *odone = pfull + 2, *oempty = odone + 2, *qfull = oempty + 2,
           *qempty = qfull + 1, *mdone = qempty + 1, *tokfull = mdone + 1;
  StepScales* scales = reinterpret_cast<StepScales*>(sm + pl.scales);
  volatile int* rawok = reinterpret_cast<volatile int*>(sm + pl.rawok);
  int* start = reinterpret_cast<int*>(sm + pl.start);
  int* slen = reinterpret_cast<int*>(sm + pl.len);
  int* snq = reinterpret_cast<int*>(sm + pl.nq);
  volatile int* fail = reinterpret_cast<volatile int*>(sm + pl.misc);
  uint32_t* taddr = reinterpret_cast<uint32_t*>(sm + pl.misc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *fail = 0;
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&kfull[i], 128);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 128);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&rawfull[i], 1);
      mbar_init(&rawempty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 2);  // the products' commit and the issuer itself
      mbar_init(&pfull[i], 128);
      mbar_init(&odone[i], 1);
      mbar_init(&oempty[i], 128);
    }
    mbar_init(qfull, 128);
    mbar_init(qempty, 1);
    mbar_init(mdone, 1);
    mbar_init(tokfull, 128);
    mbar_fence_init();
  }
  if (warp == 16) {
    tmem_alloc(taddr, 512);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 17) {
    const int per = (c.B + 31) / 32, b0 = min(c.B, lane * per), b1 = min(c.B, b0 + per);
    int own = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      slen[b] = quant_len(c, b);
      snq[b] = quant_queries(a, b);
      if (snq[b]) own += (max(1, (slen[b] + kQBlock - 1) / kQBlock) + kUnitSteps) * c.H;
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
      if (snq[b]) e += (max(1, (slen[b] + kQBlock - 1) / kQBlock) + kUnitSteps) * c.H;
    }
    if (lane == 31) start[c.B] = incl;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *taddr;
  const int total = start[c.B];
  const int C = min((int)gridDim.x, total);
  const bool works = (int)blockIdx.x < C;
  const int per = works ? total / C : 0, extra = works ? total - per * C : 0;
  auto range_lo = [&](int i) { return i * per + min(i, extra); };
  auto cta_of = [&](int y) {
    const int big = extra * (per + 1);
    return y < big ? y / (per + 1) : extra + (y - big) / per;
  };
  const int lo = works ? range_lo(blockIdx.x) : 0, hi = works ? range_lo(blockIdx.x + 1) : 0;

  // the part that the range begins with, and the one after p (x: its place)
  auto fill = [&](FewPart& p, int x) {
    p.steps = max(1, (slen[p.b] + kQBlock - 1) / kQBlock);
    p.j0 = max(0, x - p.first);
    p.j1 = min(hi - p.first, p.steps);
  };
  auto first_part = [&]() {
    FewPart p;
    int l = 0, r = c.B;
#pragma unroll 1
    while (r - l > 1) {
      const int mid = (l + r) >> 1;
      if (start[mid] <= lo) l = mid; else r = mid;
    }
    p.b = l;
    const int len = max(1, (slen[l] + kQBlock - 1) / kQBlock) + kUnitSteps;
    p.h = (lo - start[l]) / len;
    p.first = start[l] + p.h * len + kUnitSteps;
    fill(p, lo);
    return p;
  };
  auto advance = [&](FewPart& p, int& x) {
    x = p.first + max(p.j1, 0);
    if (x < hi) {
      if (++p.h == c.H) {
        p.h = 0;
        do ++p.b; while (start[p.b + 1] == start[p.b]);
      }
      p.first = x + kUnitSteps;
      fill(p, x);
    }
  };
  FewPart p;
  if (lo < hi) p = first_part();

  if (warp < 8) {
    // ================ softmax
    const int gr = warp >> 2, row = tid & 127;  // TMEM lane
    const int r = row % kCopy, copy = row / kCopy;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + gr * 64 + copy * CW;
    const uint32_t tP = tmem + lane_base + kTmemP + gr * 32, tO = tmem + lane_base + kTmemO + gr * 128;
    uint8_t* qs = sm + pl.q;
    float* fc = reinterpret_cast<float*>(sm + pl.fc);
    // 32 sums of the 256 rows, in q's place (its products have ended by then),
    // four at a time turned by the row: no bank conflicts
    float4* comb = reinterpret_cast<float4*>(sm + pl.q);
    float4* ml = reinterpret_cast<float4*>(sm + pl.ml);
    float4* rowst = reinterpret_cast<float4*>(sm + pl.rowst);
    int4* cuts = reinterpret_cast<int4*>(static_cast<uint8_t*>(a.ws) + pre_cuts(gridDim.x));
    if (tid == 0) cuts[blockIdx.x] = make_int4(0, 0, 0, -1);
    {  // P: zeros, of which a copy's tokens are overwritten step by step
      uint32_t z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = 0;
      tmem_st16(tP, z);
      tmem_st16(tP + 16, z);
      tmem_wait_st();
    }
    uint32_t ns = 0, done = 0, np = 0;  // this group's steps; all steps; parts with steps
    for (int x = lo; x < hi; advance(p, x)) {
      const int n = p.j1 - p.j0;
      if (n <= 0) continue;
      const int nq = snq[p.b], R = nq * a.G, pos0 = slen[p.b] - nq;
      const bool valid = r < R;
      const int pos = valid ? pos0 + r / a.G : 0x7fffffff;
      const int mine = (n - gr + 1) >> 1;  // steps of this group
      float m = -INFINITY, l = 0.f, dv = -INFINITY, fcol = 0.f;
      if (gr == 0) {
        // ---- q, as in quant_prefill.cu; a copy's rows are the unit's
        if (np > 0) quant_wait_warp(qempty, (np - 1) & 1, fail, lane);
        const int w0 = row & ~31, ch = lane & 15;
        int rr = w0 % kCopy + (lane >> 4);
        int tk = rr / a.G, hd = rr - tk * a.G;
        const __nv_bfloat16* src = a.q + p.b * a.qs + (long long)(p.h * a.G) * a.qh + 8 * ch;
#pragma unroll 4
        for (int i = 0; i < 32; i += 2) {
          const int rw = w0 + i + (lane >> 4);
          cp_async16(qs + (ch >> 3) * 128 * 128 + rw * 128 + (((ch & 7) ^ (rw & 7)) << 4),
                     rr < R ? src + (long long)hd * a.qh + (long long)tk * a.qt : a.q, rr < R ? 16 : 0);
          rr += 2;
          for (hd += 2; hd >= a.G; hd -= a.G) ++tk;
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
        uint8_t* me = qs + row * 128;
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(me + (i >> 3) * 128 * 128 + (((i & 7) ^ (row & 7)) << 4));
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
        fc[row] = fcol;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint4* at = reinterpret_cast<uint4*>(me + (i >> 3) * 128 * 128 + (((i & 7) ^ (row & 7)) << 4));
          const uint4 w = *at;
          *at = make_uint4(pack_h2(bf_lo(w.x) * up, bf_hi(w.x) * up),
                           pack_h2(bf_lo(w.y) * up, bf_hi(w.y) * up),
                           pack_h2(bf_lo(w.z) * up, bf_hi(w.z) * up),
                           pack_h2(bf_lo(w.w) * up, bf_hi(w.w) * up));
        }
        fence_proxy_async_smem();
        mbar_arrive(qfull);
      }
      // this group's steps but the open block's, which is a part's last
      const int nfull = (min(n, slen[p.b] / kQBlock - p.j0) - gr + 1) >> 1;
      for (int k = 0; k < nfull; ++k) {
        const int i = 2 * k + gr, base = (p.j0 + i) * kStepKeys + copy * CW;
        if (!quant_wait_warp(&sfull[gr], (ns + k) & 1, fail, lane)) break;
        tc_fence_after();
        uint32_t s[CW];
        ld_cols(tS, s);
        if (gr == 1 && k == 0) fcol = fc[row];
        const StepScales sc = scales[(done + i) % kFewScales];
        const bool vnan = sc.sv != sc.sv;
        const float ev = vnan ? 0.f : (float)((int)(__float_as_uint(sc.sv) >> 23) - 127);
        const float fv = vnan ? sc.sv : __uint_as_float((__float_as_uint(sc.sv) & 0x7fffffu) | 0x3f800000u);
        const float f = fcol * sc.sk;
        wait_cols(s);
        const bool edge = (p.j0 + i + 1) * kStepKeys - 1 > pos0 || !sc.ok;
        float x0 = -INFINITY;
        if (edge) {
          const int last = sc.ok ? pos - base : -1;
#pragma unroll
          for (int q = 0; q < CW; ++q) {
            if (q > last) s[q] = 0xff800000u;
            x0 = fmaxf(x0, __uint_as_float(s[q]));
          }
        } else {
          float x1 = -INFINITY;
#pragma unroll
          for (int q = 0; q < CW; q += 4) {
            x0 = fmaxf(x0, fmaxf(__uint_as_float(s[q]), __uint_as_float(s[q + 1])));
            x1 = fmaxf(x1, fmaxf(__uint_as_float(s[q + 2]), __uint_as_float(s[q + 3])));
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
          if (k > 0 && quant_wait_warp(&odone[gr], (ns + k - 1) & 1, fail, lane)) {
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
        const float wm = fv * ex2_approx(ev - dref + kBoostLog);
        const float2 w2 = make_float2(wm, wm), f2 = make_float2(f, f), nref = make_float2(-ref, -ref);
        float2 sum = make_float2(0.f, 0.f);
        auto weigh = [&](auto edge_c) {
          constexpr bool kEdge = decltype(edge_c)::value;
#pragma unroll
          for (int q4 = 0; q4 < CW / 16; ++q4) {
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int q = 16 * q4 + 2 * e;
              float2 v = nref;
              fma2(v, make_float2(__uint_as_float(s[q]), __uint_as_float(s[q + 1])), f2);
              v.x = ex2_approx(v.x);
              v.y = ex2_approx(v.y);
              float2 w = mul2(v, w2);
              if constexpr (kEdge) {  // a NaN scale does not reach what is not seen
                if (s[q] == 0xff800000u) v.x = w.x = 0.f;
                if (s[q + 1] == 0xff800000u) v.y = w.y = 0.f;
              }
              sum = add2(sum, v);
              pk[e] = pack_h2(w.x, w.y);
            }
            tmem_st8(tP + copy * (CW / 2) + 8 * q4, pk);
          }
        };
        if (fcol < 0.f || sc.ok == kWideStep)
          sum.x = weigh_wide(tS, tP + copy * (CW / 2), CW, fabsf(f), !edge ? CW : sc.ok ? pos - base : -1, ref,
                             ev - dref + kBoostLog, fv);
        else if (edge)
          weigh(std::true_type());
        else
          weigh(std::false_type());
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&pfull[gr]);
      }
      if (nfull < mine && quant_wait_warp(&sfull[gr], (ns + nfull) & 1, fail, lane)) {
        const int i = 2 * nfull + gr, at = (done + i) % kFewScales;
        tc_fence_after();
        if (gr == 1 && nfull == 0) fcol = fc[row];
        const RowState st = open_step({m, l, dv}, tS, tP + copy * (CW / 2), tO, CW,
                                      sm + pl.tok + at * kTokBytes + copy * CW * 2, fabsf(fcol),
                                      pos - (p.j0 + i) * kStepKeys - copy * CW,
                                      nfull > 0 ? &odone[gr] : nullptr, (ns + nfull - 1) & 1, fail);
        m = st.m;
        dv = st.dv;
        l = st.l;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&pfull[gr]);
      }
      if (mine > 0) {
        quant_wait_warp(&odone[gr], (ns + mine - 1) & 1, fail, lane);
        tc_fence_after();
      }
      ns += mine;
      done += n;
      ++np;
      // ---- the copies and groups of a row, 32 dims at a time
      ml[tid] = make_float4(m, l, dv, 0.f);
      named_bar(1, 256);
      float M = -INFINITY, Z = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2 * REP; ++i) M = fmaxf(M, ml[i * kCopy + r].x);
      const float mref = or_zero(M);
#pragma unroll
      for (int i = 0; i < 2 * REP; ++i) Z = fmaxf(Z, ml[i * kCopy + r].x - mref + ml[i * kCopy + r].z);
      const float mix = ex2_approx(m - mref + dv - or_zero(Z));
      const bool whole = p.j0 == 0 && p.j1 == p.steps;
      if (tid < kCopy) {
        float ls = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * REP; ++i) {
          const float4 t = ml[i * kCopy + r];
          if (!(t.x == -INFINITY && t.y == 0.f)) ls += t.y * ex2_approx(t.x - mref);
        }
        rowst[r] = make_float4(M, ls, Z, ls == 0.f ? 0.f : ex2_approx(Z - kBoostLog) / ls);
      }
      float4* rec = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.ws) + pre_records(gridDim.x)) +
                    ((size_t)2 * blockIdx.x + (p.j0 == 0 ? 1 : 0)) * kPreRecord;
#pragma unroll 1
      for (int dc = 0; dc < 4; ++dc) {
        uint32_t o[32];
        if (mine > 0) {
          tmem_ld32<0>(tO + 32 * dc, o);
          tmem_wait_ld32<0>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (dc == 3 && mine > 0) {
          tc_fence_before();
          mbar_arrive(&oempty[gr]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          comb[tid * 8 + (e ^ (tid & 7))] =
              make_float4(__uint_as_float(o[4 * e]) * mix, __uint_as_float(o[4 * e + 1]) * mix,
                          __uint_as_float(o[4 * e + 2]) * mix, __uint_as_float(o[4 * e + 3]) * mix);
        named_bar(1, 256);
        for (int it = tid; it < R * 8; it += 256) {
          const int ro = it >> 3, d4 = it & 7;
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 2 * REP; ++i) {
            const float4 u = comb[(i * kCopy + ro) * 8 + (d4 ^ (ro & 7))];
            t.x += u.x;
            t.y += u.y;
            t.z += u.z;
            t.w += u.w;
          }
          const float4 st = rowst[ro];
          if (whole) {
            const int tk = ro / a.G, hd = ro - tk * a.G;
            __nv_bfloat16* out = a.o + p.b * a.os + (long long)(p.h * a.G + hd) * a.oh +
                                 (long long)tk * a.ot + 32 * dc + 4 * d4;
            *reinterpret_cast<uint2*>(out) =
                st.y == 0.f ? make_uint2(0, 0)
                            : make_uint2(pack_bf16x2(t.x * st.w, t.y * st.w),
                                         pack_bf16x2(t.z * st.w, t.w * st.w));
          } else {
            rec[(size_t)(1 + 8 * dc + d4) * kTileRows + ro] = t;
            if (dc == 0 && d4 == 0) rec[ro] = st;
          }
        }
        named_bar(1, 256);
      }
      // a unit that begins in this CTA and goes on in others: for the merge
      if (!whole && tid == 0 && p.j0 == 0)
        cuts[blockIdx.x] = make_int4(p.b, p.h, 0, cta_of(p.first + p.steps - 1));
    }
  } else if (warp < 16) {
    // ================ converters
    const bool keys = warp < 12;
    const int ct = (tid - 256) & 127, sub = ct >> 2, ch = ct & 3;  // 32 rows x 4 chunks a round
    uint64_t* tfull = keys ? kfull : vfull;
    uint64_t* tempty = keys ? kempty : vempty;
    // steps converted, and open blocks; phases of the tiles and the ring
    uint32_t cnt = 0, opens = 0, tph = 1, rph = 0;
    int buf = 0, rs = 0;
    bool live = true;
    for (int x = lo; x < hi && live; advance(p, x)) {
      const int L = slen[p.b];
      bool low = false;
      auto written = [&]() {
        fence_proxy_async_smem();
        mbar_arrive(&tfull[buf]);
        ++cnt;
        if (++buf == kTiles) {
          buf = 0;
          tph ^= 1;
        }
      };
      const int jf = min(p.j1, L / kQBlock);  // full blocks; then the open one
      for (int j = p.j0; j < jf; ++j) {
        const uint8_t* raw = sm + pl.raw + rs * kQSlab;
        uint8_t* tile = sm + (keys ? pl.k : pl.v) + buf * kTileBytes;
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = make_uint4(0, 0, 0, 0);
        float sk = 1.f, sv = 1.f;
        if (!quant_wait_warp(&rawfull[rs], rph, fail, lane)) { live = false; break; }
        const bool there = rawok[rs] != 0;  // if not, zeros under weights of zero
        if (there) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint4*>(
                raw + (keys ? quant_k_chunk(32 * (i >> 1) + sub, ch + 4 * (i & 1))
                            : kQSide + (32 * i + sub) * kQBlock + ch * 16));
          if (keys && ct == 0) {
            const float2 t = *reinterpret_cast<const float2*>(raw + 2 * kQSide);
            sk = t.x;
            sv = t.y;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&rawempty[rs]);  // the codes are in registers
        if (++rs == NR) {
          rs = 0;
          rph ^= 1;
        }
        if (!quant_wait_warp(&tempty[buf], tph, fail, lane)) { live = false; break; }
        if (keys) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 32 * (i >> 1) + sub;
            put_codes<kE4M3>(tile + (i & 1) * kKHalf + row * 128, row, 2 * ch, w[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            put_codes<kE4M3>(tile + (32 * i + sub) * 128, 32 * i + sub, 2 * ch, w[i]);
        }
        if (keys && ct == 0) {
          StepScales* s = &scales[cnt % kFewScales];
          s->sk = sk;
          s->sv = sv;
          s->ok = there ? wide_step(sv, low) : 0;
        }
        written();
      }
      if (live && jf < p.j1) {  // (of an empty sequence too: no rows of it)
        if (!quant_wait_warp(&tempty[buf], tph, fail, lane)) { live = false; break; }
        const int nt = L - jf * kQBlock;
        const __nv_bfloat16 *kt = quant_tail(c, p.b, p.h, 0, jf * kQBlock),
                            *vt = quant_tail(c, p.b, p.h, 1, jf * kQBlock);
        uint8_t* tile = sm + (keys ? pl.k : pl.v) + buf * kTileBytes;
        // (the values' exponents: the keys' converters' for the softmax, the values' own)
        uint8_t* tok = keys ? sm + pl.tok + cnt % kFewScales * kTokBytes : sm + pl.vtok + (opens & 1) * kTokValues;
        open_value_exponents(vt, nt, ct, tok);
        if (keys) {
          open_keys(kt, nt, tile, ct, tok);
        } else {
          mbar_arrive(tokfull);
          if (!quant_wait_warp(tokfull, opens & 1, fail, lane)) { live = false; break; }
          ++opens;
          open_values(vt, nt, tile, ct, tok);
        }
        written();
      }
    }
  } else if (warp == 16) {
    // ================ products
    const uint32_t q0 = desc_lo(smem_u32(sm + pl.q)), k0 = desc_lo(smem_u32(sm + pl.k)),
                   v0 = desc_lo(smem_u32(sm + pl.v));
    uint32_t cnt = 0, nw[2] = {0, 0}, np[2] = {0, 0}, parts = 0;  // steps; P and parts per group
    bool live = true;
    for (int x = lo; x < hi && live; advance(p, x)) {
      const int n = p.j1 - p.j0;
      if (n <= 0) continue;
      bool ok = true;
      if (elect_one()) {
        auto scores = [&](int i) {
          const uint32_t d = tmem + (i & 1) * 64, kb = k0 + ((cnt + i) % kTiles) * (kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(d, q0 + (((kk >> 2) * 128 * 128 + (kk & 3) * 32) >> 4),
                   kb + (((kk >> 2) * kKHalf + (kk & 3) * 32) >> 4), kIdescS, kk > 0 ? 1u : 0u);
          tc_commit(&sfull[i & 1]);
          mbar_arrive(&sfull[i & 1]);
          tc_commit(&kempty[(cnt + i) % kTiles]);
        };
        auto sums = [&](int i) {
          const uint32_t g = i & 1, d = tmem + kTmemO + g * 128, pa = tmem + kTmemP + g * 32,
                         vb = v0 + ((cnt + i) % kTiles) * (kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(d, pa + 8 * kk, vb + ((kk * 32) >> 4), kIdescO, kk > 0 || i > 1 ? 1u : 0u);
          tc_commit(&odone[g]);
          tc_commit(&vempty[(cnt + i) % kTiles]);
        };
        auto tile = [&](uint64_t* bar, int i) {
          return quant_wait(&bar[(cnt + i) % kTiles], ((cnt + i) / kTiles) & 1, fail);
        };
        ok = quant_wait(qfull, parts & 1, fail);
        for (int i = 0; i < 2 && i < n && ok; ++i) {
          ok = tile(kfull, i);
          if (!ok) break;
          tc_fence_after();
          scores(i);
        }
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const int g = i & 1;
          ok = tile(vfull, i);
          if (ok) ok = quant_wait(&pfull[g], ((g ? nw[1] : nw[0]) + (i >> 1)) & 1, fail);
          // O's last sums have been read
          const uint32_t before = g ? np[1] : np[0];
          if (ok && i < 2 && before > 0) ok = quant_wait(&oempty[g], (before - 1) & 1, fail);
          if (!ok) break;
          tc_fence_after();
          sums(i);
          if (i + 2 < n) {
            ok = tile(kfull, i + 2);
            if (!ok) break;
            tc_fence_after();
            scores(i + 2);
          }
        }
        tc_commit(qempty);
      }
      live = __all_sync(0xffffffffu, ok);
      cnt += n;
      nw[0] += (n + 1) >> 1;
      nw[1] += n >> 1;
      ++np[0];
      if (n > 1) ++np[1];
      ++parts;
    }
    // every product has ended before TMEM is freed
    if (works && elect_one()) {
      tc_commit(mdone);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(mdone, 0) && global_ns() - t0 < kTcTimeoutNs) {
      }
    }
    __syncwarp();
  } else if (warp == 17) {
    // ================ loader
    const uint64_t pol = l2_evict_first_policy();
    int rs = 0, issued = 0;
    uint32_t rph = 1;  // an unused stage counts as empty
    bool live = true;
    for (int x = lo; x < hi && live; advance(p, x)) {
      const int end = min(p.j1, slen[p.b] / kQBlock);  // full blocks
      const int* bt = c.bt + (size_t)p.b * c.maxp;
      int next = p.j0 + lane < end ? __ldg(bt + p.j0 + lane) : -1;
      for (int j0 = p.j0; j0 < end && live; j0 += 32) {
        const int page = next;
        next = j0 + 32 + lane < end ? __ldg(bt + j0 + 32 + lane) : -1;
        for (int i = 0; i < 32 && j0 + i < end; ++i) {
          const int pg = __shfl_sync(0xffffffffu, page, i);
          if (!quant_wait_warp(&rawempty[rs], rph, fail, lane)) { live = false; break; }
          if (lane == 0) {
            const bool ok = pg >= 0 && pg < c.num_pages;
            rawok[rs] = ok;
            if (ok) {
              mbar_arrive_expect_tx(&rawfull[rs], kQSlab);
              bulk_g2s_hint(sm + pl.raw + rs * kQSlab, c.pages + ((size_t)pg * c.H + p.h) * kQSlab,
                            kQSlab, &rawfull[rs], pol);
            } else {
              quant_error(c, kErrBadPage);
              mbar_arrive(&rawfull[rs]);
            }
          }
          __syncwarp();
          ++issued;
          if (++rs == NR) {
            rs = 0;
            rph ^= 1;
          }
        }
      }
    }
    if (lane == 0) quant_drain(rawfull, issued, NR);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, 512);
  if (tid == 0 && *fail) quant_error(c, kErrTimeout);
}

template <bool kE4M3, int REP>
int launch(const QuantAttnArgs& a, const DevInfo& info, cudaStream_t st) {
  const void* fn = (const void*)quant_few_kernel<kE4M3, REP>;
  int NR = 5;
  while (NR > 2 && few_plan(NR, a.c.B).total + 1024 > info.optin) --NR;
  const int smem = few_plan(NR, a.c.B).total + 1024;
  if (smem > info.optin) return LRKV_ERR_UNSUPPORTED;
  const int rc = prepare_kernel(fn, true);
  if (rc != LRKV_OK) return rc;
  QuantAttnArgs args = a;
  void* p[] = {&args, &NR};
  if (launch_pdl(fn, dim3(info.sms), dim3(kFewThreads), smem, st, p) != cudaSuccess)
    return LRKV_ERR_CUDA;
  return quant_merge_launch(a, info.sms, 128 / REP, st);
}

}  // namespace

int quant_few_launch(const QuantAttnArgs& a, const DevInfo& info, cudaStream_t st) {
  const long long R = (long long)a.n * a.G;
  if (R <= 32) return a.c.e4m3 ? launch<true, 4>(a, info, st) : launch<false, 4>(a, info, st);
  if (R <= 64) return a.c.e4m3 ? launch<true, 2>(a, info, st) : launch<false, 2>(a, info, st);
  return a.c.e4m3 ? launch<true, 1>(a, info, st) : launch<false, 1>(a, info, st);
}

}  // namespace lrkv
