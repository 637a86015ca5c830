// Attention over the 8-bit full-rank cache: the simplest form.  One CTA per
// (8 rows of a unit's queries, KV head, sequence); blocks of 64 tokens one
// after the other, dequantised into shared memory, one running maximum and
// sum per row.  Row r of a unit is query r / G of q head h G + r % G.
#include "quant.cuh"

namespace lrkv {

namespace {

constexpr int kRows = 8;
constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) quant_attn_simple(QuantAttnArgs a) {
  extern __shared__ float sm[];
  float* kt = sm;                                  // [64][129]
  float* vt = kt + kQBlock * 129;                  // [64][128]
  float* qs = vt + kQBlock * kHeadDim;             // [8][128]
  float* p = qs + kRows * kHeadDim;                // [8][64]
  float* corr = p + kRows * kQBlock;               // [8]
  float* lsum = corr + kRows;                      // [8]
  pdl_trigger();
  pdl_wait();
  const QuantView& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = quant_len(c, b), nq = quant_queries(a, b), R = nq * a.G;
  const int r0 = blockIdx.x * kRows;
  if (r0 >= R) return;
  const int rows = min(kRows, R - r0);
  for (int i = tid; i < kRows * kHeadDim; i += kThreads) {
    const int r = r0 + i / kHeadDim, d = i % kHeadDim;
    qs[i] = i / kHeadDim < rows
                ? __bfloat162float(a.q[b * a.qs + (h * a.G + r % a.G) * a.qh + (r / a.G) * a.qt + d]) *
                      a.scale
                : 0.f;
  }
  const int last = L - nq + (r0 + rows - 1) / a.G;  // the last row's position
  // warp w owns row w: its maximum and sum; thread (row w, 4 dims)
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int pos = L - nq + (r0 + min(warp, rows - 1)) / a.G;
  for (int j = 0; j * kQBlock <= last; ++j) {
    __syncthreads();
    const int base = j * kQBlock;
    const bool open = base + kQBlock > L;
    const uint8_t* slab = open ? nullptr : quant_slab(c, b, h, j);
    if (!open && !slab && tid == 0) quant_error(c, kErrBadPage);
    const float sk = slab ? reinterpret_cast<const float*>(slab + 2 * kQSide)[0] : 0.f;
    const float sv = slab ? reinterpret_cast<const float*>(slab + 2 * kQSide)[1] : 0.f;
    for (int i = tid; i < kQBlock * kHeadDim; i += kThreads) {
      const int t = i / kHeadDim, d = i % kHeadDim;
      float kv = 0.f, vv = 0.f;
      if (open) {
        if (base + t < L) {
          kv = __bfloat162float(quant_tail(c, b, h, 0, base + t)[d]);
          vv = __bfloat162float(quant_tail(c, b, h, 1, base + t)[d]);
        }
      } else if (slab) {
        const uint32_t kb = slab[quant_k_chunk(t, d >> 4) + (d & 15)];
        const uint32_t vb = slab[kQSide + d * kQBlock + t];
        kv = (c.e4m3 ? quant_value<true>(kb) : quant_value<false>(kb)) * sk;
        vv = (c.e4m3 ? quant_value<true>(vb) : quant_value<false>(vb)) * sv;
      }
      kt[t * 129 + d] = kv;
      vt[i] = vv;
    }
    __syncthreads();
    if (!open && !slab) continue;  // a page out of range: its tokens are left out
    if (warp < rows) {
      float s[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = lane + 32 * u;
        s[u] = -INFINITY;
        if (base + t <= pos) {
          float x = 0.f;
          for (int d = 0; d < kHeadDim; ++d) x += qs[warp * kHeadDim + d] * kt[t * 129 + d];
          s[u] = x;
        }
      }
      // NaN scores must not vanish in the maximum
      const bool nan = __any_sync(0xffffffffu, s[0] != s[0] || s[1] != s[1]);
      const float mt = nan ? NAN : fmaxf(m, warp_max(fmaxf(s[0], s[1])));
      const float ref = mt == -INFINITY ? 0.f : mt;
      const float cr = expf(m - ref);
      const float p0 = base + lane <= pos ? expf(s[0] - ref) : 0.f;
      const float p1 = base + lane + 32 <= pos ? expf(s[1] - ref) : 0.f;
      m = mt;
      l = l * cr + warp_sum(p0 + p1);
      p[warp * kQBlock + lane] = p0;
      p[warp * kQBlock + lane + 32] = p1;
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= cr;
      const int seen = min(kQBlock, pos - base + 1);
      for (int t = 0; t < seen; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[e] += p[warp * kQBlock + t] * vt[t * kHeadDim + lane + 32 * e];
      __syncwarp();
    }
  }
  if (warp < rows) {
    const int r = r0 + warp;
    __nv_bfloat16* o = a.o + b * a.os + (h * a.G + r % a.G) * a.oh + (r / a.G) * a.ot;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[lane + 32 * e] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[e] / l);
  }
}

constexpr int kSmem = (kQBlock * 129 + kQBlock * kHeadDim + kRows * kHeadDim + kRows * kQBlock +
                       2 * kRows) * 4;

}  // namespace

size_t quant_attn_workspace(int, int, int, int) { return 256; }

int quant_attn_launch(const QuantAttnArgs& a, cudaStream_t st) {
  const int rc = prepare_kernel((const void*)quant_attn_simple, false);
  if (rc != LRKV_OK) return rc;
  QuantAttnArgs args = a;
  void* p[] = {&args};
  const unsigned nx = (unsigned)(((long long)a.n * a.G + kRows - 1) / kRows);
  return launch_pdl((const void*)quant_attn_simple, dim3(nx, a.c.H, a.c.B), dim3(kThreads), kSmem,
                    st, p) == cudaSuccess
             ? LRKV_OK
             : LRKV_ERR_CUDA;
}

}  // namespace lrkv
