// Attention of one query token per request over its pages: out = softmax(q K^T / sqrt(d)) V.
#include <cuda_fp16.h>

#include "pages.h"
#include "rtvla.h"

namespace rtvla {

namespace {
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }
}  // namespace

// One CTA per request and query head; a warp takes every fourth key, with its own running
// maximum, sum and output, joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(128) k_pages_attend(PagedAttnParams p) {
  constexpr int E = D / 32;
  const PageGeom g = p.g;
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / (p.n_q_heads / g.n_kv_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false;
  const int len = pg_len(p.lens[b], g, &bad);
  const int n = pg_list_len(len, p.sel_width, p.sel != nullptr, g);
  const int32_t *sel = p.sel ? p.sel + ((size_t)b * g.n_kv_heads + h) * p.sel_width : nullptr;
  const size_t q0 = ((size_t)b * p.n_q_heads + hq) * D;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = to_f(static_cast<const T *>(p.q)[q0 + lane + 32 * i]) * p.scale_log2;
    o[i] = 0.f;
  }
  for (int j = warp; j < n; j += 4) {
    const int row = pg_key_row(p.table + (size_t)b * g.width, sel, j, n, len, g, &bad);
    if (row < 0) continue;
    const size_t at = pg_elem(p.layer, row, h, g) + lane;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += q[i] * to_f(static_cast<const T *>(p.k)[at + 32 * i]);
    s = warp_sum(s);
    const float nm = fmaxf(m, s), ref = nm == -INFINITY ? 0.f : nm;
    const float a = exp2f(m - ref), w = exp2f(s - ref);
    m = nm;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * a + w * to_f(static_cast<const T *>(p.v)[at + 32 * i]);
  }
  __shared__ float so[4][D], sm[4], sl[4];
#pragma unroll
  for (int i = 0; i < E; ++i) so[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_ATTEND);
  __syncthreads();
  const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int w = 0; w < 4; ++w) L += sl[w] * exp2f(sm[w] - ref);
  for (int i = threadIdx.x; i < D; i += 128) {
    float v = 0.f;
    for (int w = 0; w < 4; ++w) v += so[w][i] * exp2f(sm[w] - ref);
    put(static_cast<T *>(p.out) + q0 + i, L > 0.f ? v / L : 0.f);
  }
}

namespace {
template <typename T>
cudaError_t attend(const PagedAttnParams &p, cudaStream_t st) {
  const dim3 grid(p.n_q_heads, p.batch);
  if (p.g.head_dim == 64) k_pages_attend<T, 64><<<grid, 128, 0, st>>>(p);
  else if (p.g.head_dim == 128) k_pages_attend<T, 128><<<grid, 128, 0, st>>>(p);
  else k_pages_attend<T, 256><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_pages_attend(const PagedAttnParams &p, int dtype, cudaStream_t st) {
  return dtype == RTVLA_DTYPE_BF16 ? attend<bf16>(p, st) : attend<__half>(p, st);
}

}  // namespace rtvla
