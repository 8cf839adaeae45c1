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
//
// A decode step is one CTA: a chain of two scans and three dependent loads.  With more rows every
// CTA repeats the scans and takes a share of the rows and pages; the last one to finish writes the
// lengths and the new top, which the others still read (they may be updated in place).
__global__ void __launch_bounds__(PT) k_pages_plan(PlanParams p) {
  extern __shared__ int sm[];
  __shared__ long long warp_sums[PT / 32];
  __shared__ int first_refused, is_last;
  const PageGeom g = p.g;
  const int B = p.batch, cap = g.width << g.shift;
  int *s_len = sm;                  // length before the step; ~length: refused alone
  int *s_delta = s_len + B;
  int *s_rows = s_delta + B;        // [B + 1] rows before request b, at most n_rows
  int *s_take = s_rows + B + 1;     // [B + 1] pages popped before request b
  int *s_back = s_take + B + 1;     // [B + 1] pages pushed before request b
  const int per = (B + PT - 1) / PT;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  const int first = blockIdx.x * PT + threadIdx.x, stride = gridDim.x * PT;  // shares of rows and pages
  bool bad = false;
  if (threadIdx.x == 0) first_refused = B;
  for (int b = threadIdx.x; b < B; b += PT) {
    s_len[b] = p.lens[b];
    s_delta[b] = p.delta[b];
  }
  const int raw_free = p.n_free[0];
  __syncthreads();

  long long sum = 0, total;
  for (int b = b0; b < b1; ++b) sum += max(s_delta[b], 0);
  long long rows = block_scan(sum, &total, warp_sums);
  if (threadIdx.x == 0) s_rows[B] = (int)min(total, (long long)p.n_rows);
  long long take = 0, back = 0;
  for (int b = b0; b < b1; ++b) {
    const int raw = s_len[b], delta = s_delta[b];
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
      const int held = pg_pages(len, g), after = pg_pages((int)max(0ll, (long long)len + s_delta[b]), g);
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
  for (int i = first; i < n_take; i += stride) {
    const int b = owner(s_take, B, i);
    p.table[(size_t)b * g.width + pg_pages(s_len[b], g) + (i - s_take[b])] = popped(i);
  }
  for (int e = first; e < n_back; e += stride) p.free_pages[nf + e] = given_back(e);
  for (int r = first; r < p.n_rows; r += stride) {
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
  if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_PLAN);
  if (gridDim.x > 1) {
    __syncthreads();  // this CTA has read its lengths
    if (threadIdx.x == 0) {
      __threadfence();
      is_last = atomicAdd(p.done, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last) return;
    if (threadIdx.x == 0) *p.done = 0;  // for the next call
  }
  for (int b = threadIdx.x; b < B; b += PT) {
    const int len = s_len[b];
    int n = len < 0 ? ~len : len;
    if (len >= 0 && (b < stop || s_take[b + 1] == s_take[b])) n = (int)max(0ll, (long long)len + s_delta[b]);
    p.lens_out[b] = n;
    p.row_start[b] = s_rows[b];
  }
  if (threadIdx.x == 0) {
    p.row_start[B] = s_rows[B];
    p.n_free_out[0] = top - n_take;
  }
}

namespace {
size_t plan_smem(int batch) { return (size_t)(5 * batch + 3) * sizeof(int); }

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

constexpr int ST = 512;            // threads of a select CTA
constexpr int SC = 8;              // CTAs of a cluster: they score, the first one chooses
constexpr int RUN = 16;            // pages a warp scores at a time
constexpr int BITS = 11, BINS = 1 << BITS;
constexpr int SELECT_SMEM_KEYS = 8192;  // keys held in shared memory; longer tables use the workspace

// Order-preserving map of a score to an integer; 0 and 1 are kept for pages outside the pool.
__device__ __forceinline__ unsigned long long score_key(double s) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(s);
  return max((u >> 63) ? ~u : u | 0x8000000000000000ull, 2ull);
}
constexpr unsigned long long KEY_BAD = 1;

__device__ __forceinline__ void add8(double (&a)[8], const uint4 &v, bf16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[2 * i] += (double)__uint_as_float(w[i] << 16);
    a[2 * i + 1] += (double)__uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void add8(double (&a)[8], const uint4 &v, __half) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    a[2 * i] += (double)f.x;
    a[2 * i + 1] += (double)f.y;
  }
}

// Exclusive scan of a pair of counts over the block.
__device__ uint2 scan_pair(uint2 v, uint2 *warp_sums, uint2 *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint2 inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) {
      inc.x += x;
      inc.y += y;
    }
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = inc;
  __syncthreads();
  uint2 before = make_uint2(0, 0), all = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < ST / 32; ++i) {
    const uint2 x = warp_sums[i];
    if (i < w) {
      before.x += x.x;
      before.y += x.y;
    }
    all.x += x.x;
    all.y += x.y;
  }
  *total = all;
  return make_uint2(before.x + inc.x - v.x, before.y + inc.y - v.y);
}

}  // namespace

// One cluster per request and KV head.  Its CTAs share the scoring (16 bytes of a page's mean per
// lane, fp64 sums: the means of a long request are a few hundred KB, so this is latency, not
// bandwidth) and put order-preserving integer keys into the first CTA's shared memory.  That CTA
// finds the lowest key taken by radix passes from the top bits, which stop as soon as the pages
// in the deciding bin fit one comparison of all pairs: two passes for ordinary scores.  Selected is
// then every key above that one, and of the keys equal to it the first few in page order.
template <typename T, int D>
__global__ void __cluster_dims__(SC, 1, 1) __launch_bounds__(ST) k_pages_select(SelectParams p) {
  extern __shared__ unsigned long long smem_keys[];
  __shared__ int bins[BINS];
  __shared__ uint2 warp_sums[ST / 32];
  __shared__ unsigned long long near_key[ST];
  __shared__ int bin_s, above_s, n_near, near_eq;
  __shared__ unsigned long long cut_s;
  const PageGeom g = p.g;
  const int rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z, G = p.n_q_heads / g.n_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false;
  const int held = pg_pages(pg_len(p.lens[b], g, &bad), g);
  if (bad && threadIdx.x == 0 && rank == 0 && h == 0) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_SELECT);
  int *sel = p.sel + ((size_t)b * g.n_kv_heads + h) * p.budget;
  if (held <= p.budget) {  // the whole cluster leaves here
    for (int i = rank * ST + threadIdx.x; i < p.budget; i += SC * ST) sel[i] = i < held ? i : -1;
    return;
  }
  // candidates: logical pages lo .. lo + n - 1, of which `need` are chosen
  const int lo = p.keep_first, n = held - p.keep_last - lo, need = p.budget - lo - p.keep_last;
  const bool in_smem = g.width <= SELECT_SMEM_KEYS;
  unsigned long long *keys = in_smem ? smem_keys : p.keys + ((size_t)b * g.n_kv_heads + h) * g.width;
  {
    unsigned long long *dst = keys;
    if (in_smem) {
      uint64_t at;
      asm("mapa.u64 %0, %1, %2;" : "=l"(at) : "l"(reinterpret_cast<uint64_t>(smem_keys)), "r"(0));
      dst = reinterpret_cast<unsigned long long *>(at);
    }
    constexpr int LPP = D / 8, PPW = 32 / LPP;  // lanes per page, pages per load
    const int sub = lane / LPP, ln = lane % LPP;
    double qs[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const T *q = static_cast<const T *>(p.q) + ((size_t)b * p.n_q_heads + h * G) * D + ln * 8;
    for (int j = 0; j < G; ++j) add8(qs, *reinterpret_cast<const uint4 *>(q + (size_t)j * D), T());
    for (int c0 = (rank * (ST / 32) + warp) * RUN; c0 < n; c0 += SC * (ST / 32) * RUN) {
      const int mine = lane < RUN && c0 + lane < n ? pg_page(p.table + (size_t)b * g.width, lo + c0 + lane, g) : -1;
      if (lane < RUN && c0 + lane < n && mine < 0) bad = true;
      constexpr int LOADS = RUN / PPW, AHEAD = LOADS < 8 ? LOADS : 8;
#pragma unroll
      for (int i0 = 0; i0 < LOADS; i0 += AHEAD) {
        uint4 v[AHEAD];
        int page[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          page[i] = __shfl_sync(0xffffffffu, mine, (i0 + i) * PPW + sub);
          v[i] = make_uint4(0, 0, 0, 0);
          if (page[i] >= 0)
            v[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k_mean) +
                                                    pg_mean_elem(p.layer, page[i], h, g) + ln * 8);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          double m[8] = {0, 0, 0, 0, 0, 0, 0, 0}, s = 0.0;
          add8(m, v[i], T());
#pragma unroll
          for (int u = 0; u < 8; ++u) s += qs[u] * m[u];
#pragma unroll
          for (int o = LPP / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          const int c = c0 + (i0 + i) * PPW + sub;
          if (ln == 0 && c < n) dst[c] = page[i] < 0 ? KEY_BAD : score_key(s);
        }
      }
    }
    if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_SELECT);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank != 0) return;

  // cut: the lowest key taken; eq: how many of the keys equal to it are taken
  unsigned long long cut = 0, prefix = 0;
  int eq = 0, left = need, shift = 64;
  while (left > 0) {
    const int width = min(BITS, shift), next = shift - width;
    for (int i = threadIdx.x; i < BINS; i += ST) bins[i] = 0;
    if (threadIdx.x == 0) n_near = 0;
    __syncthreads();
    for (int c0 = 0; c0 < n; c0 += ST) {
      const int c = c0 + threadIdx.x;
      const bool in = c < n && (shift == 64 || keys[c] >> shift == prefix);
      // neighbours in score share their top bits, so that lanes are counted together
      const int digit = in ? (int)((keys[c] >> next) & ((1 << width) - 1)) : -1;
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&bins[digit], __popc(same));
    }
    __syncthreads();
    // the bin that holds the `left`-th highest: bins are scanned from the top
    constexpr int PER = BINS / ST;
    uint2 mine = make_uint2(0, 0), all;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine.x += bins[BINS - 1 - (threadIdx.x * PER + i)];
    int above = (int)scan_pair(mine, warp_sums, &all).x;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int bin = BINS - 1 - (threadIdx.x * PER + i), count = bins[bin];
      if (above < left && left <= above + count) {
        bin_s = bin;
        above_s = above;
      }
      above += count;
    }
    __syncthreads();
    const int count = bins[bin_s];
    prefix = shift == 64 ? (unsigned long long)bin_s : (prefix << width) | (unsigned long long)bin_s;
    shift = next;
    left -= above_s;
    if (left == count || shift == 0) {
      cut = prefix << shift;
      eq = left;  // shift 0: `left` of the keys equal to the cut; otherwise every key of the bin
      if (shift > 0) {  // one below the bin (no key is 0)
        cut = cut ? cut - 1 : 0;
        eq = 0;
      }
      break;
    }
    if (count <= ST) {  // few enough to compare all pairs
      for (int c = threadIdx.x; c < n; c += ST)
        if (keys[c] >> shift == prefix) near_key[atomicAdd(&n_near, 1)] = keys[c];
      __syncthreads();
      if ((int)threadIdx.x < count) {
        const unsigned long long k = near_key[threadIdx.x];
        int over = 0, same = 0;
        for (int i = 0; i < count; ++i) {
          over += near_key[i] > k;
          same += near_key[i] == k;
        }
        if (over < left && left <= over + same) {  // equal keys write equal values
          cut_s = k;
          near_eq = left - over;
        }
      }
      __syncthreads();
      cut = cut_s;
      eq = near_eq;
      break;
    }
    __syncthreads();
  }
  if (need == 0) {
    cut = ~0ull;
    eq = 0;
  }
  // the chosen pages in order: every thread takes a run of pages
  const int per = (n + ST - 1) / ST, c0 = min(n, (int)threadIdx.x * per), c1 = min(n, c0 + per);
  uint2 mine = make_uint2(0, 0), all;
  for (int c = c0; c < c1; ++c) {
    mine.x += keys[c] > cut;
    mine.y += keys[c] == cut;
  }
  const uint2 before = scan_pair(mine, warp_sums, &all);
  int equal = (int)before.y, at = lo + (int)before.x + min(equal, eq);
  for (int c = c0; c < c1; ++c) {
    const bool take = keys[c] > cut || (keys[c] == cut && equal < eq);
    equal += keys[c] == cut;
    if (take) sel[at++] = lo + c;
  }
  for (int i = threadIdx.x; i < lo; i += ST) sel[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += ST) sel[p.budget - p.keep_last + i] = held - p.keep_last + i;
}

// ---------------------------------------------------------------------------------------
// launchers

cudaError_t launch_pages_plan(const PlanParams &p, int sm_count, cudaStream_t st) {
  // four rows per thread: the scans cost every CTA about 4 us, as much as a thread's four rows
  const int want = (p.n_rows + 4 * PT - 1) / (4 * PT);
  k_pages_plan<<<want < 1 ? 1 : want < sm_count ? want : sm_count, PT, plan_smem(p.batch), st>>>(p);
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

namespace {
size_t select_smem(const PageGeom &g) { return g.width <= SELECT_SMEM_KEYS ? (size_t)g.width * 8 : 0; }

template <typename T, int D>
cudaError_t select_attributes() {
  return cudaFuncSetAttribute(k_pages_select<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SELECT_SMEM_KEYS * 8);
}

template <typename T>
cudaError_t select(const SelectParams &p, cudaStream_t st) {
  const dim3 grid(SC, p.g.n_kv_heads, p.batch);
  const size_t sm = select_smem(p.g);
  if (p.g.head_dim == 64) k_pages_select<T, 64><<<grid, ST, sm, st>>>(p);
  else if (p.g.head_dim == 128) k_pages_select<T, 128><<<grid, ST, sm, st>>>(p);
  else k_pages_select<T, 256><<<grid, ST, sm, st>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t pages_init_attributes() {
  cudaError_t e =
      cudaFuncSetAttribute(k_pages_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(4096));
  if (e == cudaSuccess) e = select_attributes<bf16, 64>();
  if (e == cudaSuccess) e = select_attributes<bf16, 128>();
  if (e == cudaSuccess) e = select_attributes<bf16, 256>();
  if (e == cudaSuccess) e = select_attributes<__half, 64>();
  if (e == cudaSuccess) e = select_attributes<__half, 128>();
  if (e == cudaSuccess) e = select_attributes<__half, 256>();
  return e;
}

bool pages_select_needs_keys(const PageGeom &g) { return g.width > SELECT_SMEM_KEYS; }

cudaError_t launch_pages_select(const SelectParams &p, int dtype, cudaStream_t st) {
  return dtype == RTVLA_DTYPE_BF16 ? select<bf16>(p, st) : select<__half>(p, st);
}

}  // namespace rtvla
