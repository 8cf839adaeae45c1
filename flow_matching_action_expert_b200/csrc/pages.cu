// Kernels of the paged KV cache's bookkeeping: the plan (pages, slots and positions of a step's
// new tokens), the write of new rows into their slots, and the choice of pages for sparse
// attention.  The attention itself is in paged_attn.cu.
#include <cuda_fp16.h>

#include "pages.h"
#include "rtvla.h"

namespace rtvla {

namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<bf16>(bf16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// ---------------------------------------------------------------------------------------
// plan

constexpr int PT = 256;  // threads of the plan kernel

// Exclusive scan of one value per thread over the block; *total receives the sum.
__device__ long long block_scan(long long v, long long *total, long long *warp_sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  __syncthreads();  // warp_sums free again
  if (lane == 31) warp_sums[w] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < PT / 32; ++i) {
    if (i < w) before += warp_sums[i];
    all += warp_sums[i];
  }
  *total = all;
  return before + inc - v;
}

// Last index b with cum[b] <= i (cum[0] = 0, i < cum[n]): the request that owns item i.
__device__ __forceinline__ int owner(const int *cum, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

// Scans over the requests give the rows, the pages pushed and the pages popped before each
// request; everything else follows from those three sums without any order among threads.  A
// popped page may be one pushed in the same step, so a pop looks its page up where the push would
// read it instead of in the free list (pages pushed in this step lie at or above the old top, so
// the pushes never touch an entry a pop reads).
__global__ void __launch_bounds__(PT) k_pages_plan(PlanParams p) {
  extern __shared__ int sm[];
  __shared__ long long warp_sums[PT / 32];
  __shared__ int first_refused;
  const PageGeom g = p.g;
  const int B = p.batch, cap = g.width << g.shift;
  int *s_len = sm;                  // length before the step; ~length: refused alone
  int *s_rows = s_len + B;          // [B + 1] rows before request b, at most n_rows
  int *s_take = s_rows + B + 1;     // [B + 1] pages popped before request b
  int *s_back = s_take + B + 1;     // [B + 1] pages pushed before request b
  const int per = (B + PT - 1) / PT;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  bool bad = false;
  if (threadIdx.x == 0) first_refused = B;

  long long sum = 0, total;
  for (int b = b0; b < b1; ++b) sum += max(p.delta[b], 0);
  long long rows = block_scan(sum, &total, warp_sums);
  if (threadIdx.x == 0) s_rows[B] = (int)min(total, (long long)p.n_rows);
  long long take = 0, back = 0;
  for (int b = b0; b < b1; ++b) {
    const int raw = p.lens[b], delta = p.delta[b];
    bool alone = false;
    const int len = pg_len(raw, g, &alone);
    s_rows[b] = (int)min(rows, (long long)p.n_rows);
    if (delta > 0) {
      rows += delta;
      if (rows > p.n_rows || (long long)len + delta > cap) alone = true;
    }
    s_len[b] = alone ? ~len : len;
    bad |= alone;
    if (!alone) {
      const int held = pg_pages(len, g), after = pg_pages((int)max(0ll, (long long)len + delta), g);
      take += max(0, after - held);
      back += max(0, held - after);
    }
  }
  long long all_take, all_back;
  take = block_scan(take, &all_take, warp_sums);
  back = block_scan(back, &all_back, warp_sums);
  const int raw_free = p.n_free[0];
  const int nf = min(max(raw_free, 0), g.n_pages);
  // a table that gives back more pages than the pool has is the caller's fault
  const int n_back = (int)min(all_back, (long long)(g.n_pages - nf));
  if (raw_free != nf || all_back > n_back) bad = true;
  const int top = nf + n_back;
  for (int b = b0; b < b1; ++b) {
    s_take[b] = (int)take;
    s_back[b] = (int)min(back, (long long)n_back);
    const int len = s_len[b];
    if (len >= 0) {
      const int held = pg_pages(len, g), after = pg_pages((int)max(0ll, (long long)len + p.delta[b]), g);
      if (after > held && take + (after - held) > top) atomicMin(&first_refused, b);
      take += max(0, after - held);
      back += max(0, held - after);
    }
  }
  if (threadIdx.x == 0) {
    s_take[B] = (int)all_take;
    s_back[B] = n_back;
  }
  __syncthreads();
  const int stop = first_refused;
  const int n_take = s_take[stop];
  if (threadIdx.x == 0 && stop < B) set_error(p.ctl, DEVERR_NO_PAGES, PG_AT_PLAN);

  auto given_back = [&](int e) {  // page pushed as the e-th of this step
    const int b = owner(s_back, B, e);
    const int held = pg_pages(s_len[b], g), n = s_back[b + 1] - s_back[b];
    return p.table[(size_t)b * g.width + held - n + (e - s_back[b])];
  };
  auto popped = [&](int i) {  // page popped as the i-th of this step
    const int at = top - 1 - i;
    return at < nf ? p.free_pages[at] : given_back(at - nf);
  };
  for (int i = threadIdx.x; i < n_take; i += PT) {
    const int b = owner(s_take, B, i);
    p.table[(size_t)b * g.width + pg_pages(s_len[b], g) + (i - s_take[b])] = popped(i);
  }
  for (int e = threadIdx.x; e < n_back; e += PT) p.free_pages[nf + e] = given_back(e);
  for (int r = threadIdx.x; r < p.n_rows; r += PT) {
    int slot = -1, pos = 0;
    if (r < s_rows[B]) {
      const int b = owner(s_rows, B, r), len = s_len[b];
      if (len >= 0 && (b < stop || s_take[b + 1] == s_take[b])) {
        pos = len + (r - s_rows[b]);
        const int e = pos >> g.shift, held = pg_pages(len, g);
        const int page = e < held ? p.table[(size_t)b * g.width + e] : popped(s_take[b] + e - held);
        if (page >= 0 && page < g.n_pages) {
          slot = (page << g.shift) + (pos & ((1 << g.shift) - 1));
        } else {
          bad = true;
          pos = 0;
        }
      }
    }
    p.slots[r] = slot;
    p.positions[r] = pos;
  }
  __syncthreads();  // lens_out may be lens, n_free_out n_free
  for (int b = threadIdx.x; b < B; b += PT) {
    const int len = s_len[b];
    int n = len < 0 ? ~len : len;
    if (len >= 0 && (b < stop || s_take[b + 1] == s_take[b])) n = (int)max(0ll, (long long)len + p.delta[b]);
    p.lens_out[b] = n;
    p.row_start[b] = s_rows[b];
  }
  if (threadIdx.x == 0) {
    p.row_start[B] = s_rows[B];
    p.n_free_out[0] = top - n_take;
  }
  if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_PLAN);
}

namespace {
size_t plan_smem(int batch) { return (size_t)(4 * batch + 3) * sizeof(int); }

// ---------------------------------------------------------------------------------------
// write

// cos and sin of a position as the product of two table entries, e^{i(256 h + l)f} =
// e^{i 256 h f} e^{i l f}: both tables hold fp64 angles rounded once, so the product is within
// 2e-7 of the exact value at every position, and 2^24 positions need two tables of at most 2^16
// rows instead of one of 2^24.
__device__ __forceinline__ float2 rope_at(const float2 *lo, const float2 *hi, int pos, int i, int half) {
  const float2 a = lo[(size_t)(pos & 255) * half + i], b = hi[(size_t)(pos >> 8) * half + i];
  return make_float2(a.x * b.x - a.y * b.y, a.y * b.x + a.x * b.y);
}

}  // namespace

// One CTA per row.
template <typename T, typename S>
__global__ void __launch_bounds__(128) k_pages_write(WriteParams p) {
  const PageGeom g = p.g;
  const int r = blockIdx.x, d = g.head_dim, half = d / 2;
  const int hq = p.n_q_heads, hkv = g.n_kv_heads, ld = (hq + 2 * hkv) * d;
  bool bad = false;
  const int slot = pg_slot(p.slots[r], g, &bad), pos = p.positions[r];
  if (slot >= 0 && (pos < 0 || pos >= g.width << g.shift)) bad = true;
  if (bad && threadIdx.x == 0) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_WRITE);
  if (slot < 0 || bad) return;
  const S *src = static_cast<const S *>(p.qkv);
  T *k = static_cast<T *>(p.k), *v = static_cast<T *>(p.v), *q = static_cast<T *>(p.q_out);
  // the rotated, rounded pair i of head h of row `row` at position `at`
  auto pair = [&](int row, int at, int h, int i, T &y1, T &y2) {
    const S *x = src + (size_t)row * ld + h * d;
    const float x1 = to_f(x[i]), x2 = to_f(x[i + half]);
    const float2 cs = p.rope_lo ? rope_at(p.rope_lo, p.rope_hi, at, i, half) : make_float2(1.f, 0.f);
    y1 = from_f<T>(x1 * cs.x - x2 * cs.y);
    y2 = from_f<T>(x2 * cs.x + x1 * cs.y);
  };
  for (int u = threadIdx.x; u < (hq + hkv) * half; u += blockDim.x) {
    const int h = u / half, i = u % half;
    T y1, y2;
    pair(r, pos, h, i, y1, y2);
    T *dst = h < hq ? q + (size_t)r * hq * d + h * d : k + pg_elem(p.layer, slot, h - hq, g);
    dst[i] = y1;
    dst[i + half] = y2;
  }
  for (int u = threadIdx.x; u < hkv * d; u += blockDim.x)
    v[pg_elem(p.layer, slot, u / d, g) + u % d] = from_f<T>(to_f(src[(size_t)r * ld + (hq + hkv) * d + u]));
  const int ps = 1 << g.shift;
  if (!p.k_mean || (slot & (ps - 1)) != ps - 1) return;
  // this row fills its page: its keys are this call's rows r, r - 1, ... as far as their slots run
  // on downwards (other CTAs write those, so they are computed again here), and the pool's below
  __shared__ int run;
  if (threadIdx.x == 0) run = min(ps, r + 1);
  __syncthreads();
  for (int i = threadIdx.x; i < min(ps, r + 1); i += blockDim.x)
    if (p.slots[r - i] != slot - i) atomicMin(&run, i);
  __syncthreads();
  const int from = ps - run;
  T *mean = static_cast<T *>(p.k_mean);
  for (int u = threadIdx.x; u < hkv * half; u += blockDim.x) {
    const int h = u / half, i = u % half;
    float s1 = 0.f, s2 = 0.f;
    for (int o = 0; o < ps; ++o) {
      T y1, y2;
      if (o < from) {
        const T *x = k + pg_elem(p.layer, slot - (ps - 1) + o, h, g);
        y1 = x[i];
        y2 = x[i + half];
      } else {
        const int row = r - (ps - 1 - o);
        const int at = min(max(p.positions[row], 0), (g.width << g.shift) - 1);
        pair(row, at, hq + h, i, y1, y2);
      }
      s1 += to_f(y1);
      s2 += to_f(y2);
    }
    T *dst = mean + pg_mean_elem(p.layer, slot >> g.shift, h, g);
    dst[i] = from_f<T>(s1 / ps);
    dst[i + half] = from_f<T>(s2 / ps);
  }
}

// ---------------------------------------------------------------------------------------
// select

namespace {
// Order-preserving map of a score to an integer; 0 and 1 and the all-ones word are kept free.
__device__ __forceinline__ unsigned long long score_key(double s) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(s);
  const unsigned long long k = (u >> 63) ? ~u : u | 0x8000000000000000ull;
  return min(max(k, 2ull), ~1ull);
}
constexpr unsigned long long KEY_BAD = 1, KEY_TAKEN = ~0ull;
}  // namespace

// One CTA per request and KV head: every page's score, then the best page, budget times over.
template <typename T>
__global__ void __launch_bounds__(256) k_pages_select(SelectParams p) {
  const PageGeom g = p.g;
  const int h = blockIdx.x, b = blockIdx.y, d = g.head_dim, G = p.n_q_heads / g.n_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ double qs[256];
  __shared__ unsigned long long best_key[8];
  __shared__ int best_page[8], counts[8];
  bool bad = false;
  const int held = pg_pages(pg_len(p.lens[b], g, &bad), g);
  if (bad && threadIdx.x == 0 && h == 0) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_SELECT);
  int *sel = p.sel + ((size_t)b * g.n_kv_heads + h) * p.budget;
  const int n = min(held, p.budget);
  if (held <= p.budget) {
    for (int i = threadIdx.x; i < p.budget; i += 256) sel[i] = i < n ? i : -1;
    return;
  }
  const T *q = static_cast<const T *>(p.q) + ((size_t)b * p.n_q_heads + h * G) * d;
  for (int i = threadIdx.x; i < d; i += 256) {
    double s = 0.0;
    for (int j = 0; j < G; ++j) s += (double)to_f(q[j * d + i]);
    qs[i] = s;
  }
  __syncthreads();
  unsigned long long *keys = p.keys + ((size_t)b * g.n_kv_heads + h) * g.width;
  const int lo = p.keep_first, hi = held - p.keep_last;
  for (int e = warp; e < held; e += 8) {
    unsigned long long key = KEY_TAKEN;
    if (e >= lo && e < hi) {
      const int page = pg_page(p.table + (size_t)b * g.width, e, g);
      if (page < 0) {
        key = KEY_BAD;
        if (lane == 0) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_SELECT);
      } else {
        const T *m = static_cast<const T *>(p.k_mean) + pg_mean_elem(p.layer, page, h, g);
        double s = 0.0;
        for (int i = lane; i < d; i += 32) s += qs[i] * (double)to_f(m[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        key = score_key(s);
      }
    }
    if (lane == 0) keys[e] = key;
  }
  __syncthreads();
  for (int left = p.budget - lo - p.keep_last; left > 0; --left) {
    unsigned long long k = 0;
    int at = 0;
    for (int e = lo + threadIdx.x; e < hi; e += 256)
      if (keys[e] != KEY_TAKEN && keys[e] > k) {
        k = keys[e];
        at = e;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, k, o);
      const int a2 = __shfl_xor_sync(0xffffffffu, at, o);
      if (k2 > k || (k2 == k && a2 < at)) {
        k = k2;
        at = a2;
      }
    }
    if (lane == 0) {
      best_key[warp] = k;
      best_page[warp] = at;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int w = 0;
      for (int i = 1; i < 8; ++i)
        if (best_key[i] > best_key[w] || (best_key[i] == best_key[w] && best_page[i] < best_page[w])) w = i;
      keys[best_page[w]] = KEY_TAKEN;
    }
    __syncthreads();
  }
  int done = 0;
  for (int e0 = 0; e0 < held; e0 += 256) {
    const int e = e0 + threadIdx.x;
    const bool mine = e < held && keys[e] == KEY_TAKEN;
    const unsigned m = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) counts[warp] = __popc(m);
    __syncthreads();
    int before = done;
    for (int i = 0; i < 8; ++i) {
      if (i < warp) before += counts[i];
      done += counts[i];
    }
    if (mine) sel[before + __popc(m & ((1u << lane) - 1))] = e;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------------
// launchers

cudaError_t pages_init_attributes() {
  return cudaFuncSetAttribute(k_pages_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(4096));
}

cudaError_t launch_pages_plan(const PlanParams &p, cudaStream_t st) {
  k_pages_plan<<<1, PT, plan_smem(p.batch), st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_write(const WriteParams &p, int dtype, int src_dtype, cudaStream_t st) {
  if (p.n_rows == 0) return cudaSuccess;
  if (dtype == RTVLA_DTYPE_BF16) {
    if (src_dtype == RTVLA_DTYPE_F32) k_pages_write<bf16, float><<<p.n_rows, 128, 0, st>>>(p);
    else k_pages_write<bf16, bf16><<<p.n_rows, 128, 0, st>>>(p);
  } else {
    if (src_dtype == RTVLA_DTYPE_F32) k_pages_write<__half, float><<<p.n_rows, 128, 0, st>>>(p);
    else k_pages_write<__half, __half><<<p.n_rows, 128, 0, st>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_pages_select(const SelectParams &p, int dtype, cudaStream_t st) {
  const dim3 grid(p.g.n_kv_heads, p.batch);
  if (dtype == RTVLA_DTYPE_BF16) k_pages_select<bf16><<<grid, 256, 0, st>>>(p);
  else k_pages_select<__half><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace rtvla
