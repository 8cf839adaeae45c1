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

// Exclusive scan of one value per thread over a block of PT; *total receives the sum.
template <int PT>
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
  long long sums = lane < PT / 32 ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += n;
  }
  const long long before = __shfl_sync(0xffffffffu, sums, (w + 31) & 31);
  *total = __shfl_sync(0xffffffffu, sums, 31);
  return (w ? before : 0) + inc - v;
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
// A decode step is one CTA: a chain of three scans and three dependent loads.  With more rows every
// CTA repeats the scans and takes a share of the rows and pages; the last one to finish writes the
// lengths and the new top, which the others still read (they may be updated in place).  Measured:
// 64 requests of one token 4.9 us; 2000 requests and 91 thousand rows 13.9 us (one CTA: 1173 us).
template <int PT>
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
  long long rows = block_scan<PT>(sum, &total, warp_sums);
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
  take = block_scan<PT>(take, &all_take, warp_sums);
  back = block_scan<PT>(back, &all_back, warp_sums);
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
  for (int e = first; e < n_back; e += stride) {
    const int page = given_back(e);
    bad |= !pg_in_pool(page, g);
    p.free_pages[nf + e] = page;
  }
  for (int r = first; r < p.n_rows; r += stride) {
    int slot = -1, pos = 0;
    if (r < s_rows[B]) {
      const int b = owner(s_rows, B, r), len = s_len[b];
      if (len >= 0 && (b < stop || s_take[b + 1] == s_take[b])) {
        pos = len + (r - s_rows[b]);
        const int e = pos >> g.shift, held = pg_pages(len, g);
        const int page = e < held ? p.table[(size_t)b * g.width + e] : popped(s_take[b] + e - held);
        if (pg_in_pool(page, g)) {
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

}  // namespace

// ---------------------------------------------------------------------------------------
// write

namespace {

constexpr int WT = 256;       // threads of a write CTA
constexpr int MEAN_CTAS = 2;  // per SM, that look for filled pages
constexpr int HEADS = 4;      // heads a thread moves: their loads are in flight together

// eight consecutive values as they lie in memory, and in fp32
template <typename S>
struct Raw8 {
  uint4 v[sizeof(S) / 2];
  __device__ __forceinline__ void load(const S *p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(S) / 2; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void to(float (&f)[8]) const {
    const S *x = reinterpret_cast<const S *>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f(x[i]);
  }
};
template <typename S>
__device__ __forceinline__ void load8(float (&f)[8], const S *p) {
  Raw8<S> r;
  r.load(p);
  r.to(f);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
  uint4 v;
  T *x = reinterpret_cast<T *>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = from_f<T>(f[i]);
  *reinterpret_cast<uint4 *>(p) = v;
}

// cos and sin of pairs 8 i8 .. 8 i8 + 7 at a position: the product of two table entries,
// e^{i(256 h + l)f} = e^{i 256 h f} e^{i l f}.  Both tables hold fp64 angles rounded once, so the
// product is within 2e-7 of the exact value at every position, and 2^24 positions need two tables
// of at most 2^16 rows instead of one of 2^24.
__device__ __forceinline__ void rope8(float (&c)[8], float (&s)[8], const WriteParams &p, int pos, int i8, int half) {
  const float4 *lo = reinterpret_cast<const float4 *>(p.rope_lo + (size_t)(pos & 255) * half + i8 * 8);
  const float4 *hi = reinterpret_cast<const float4 *>(p.rope_hi + (size_t)(pos >> 8) * half + i8 * 8);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float4 a = lo[u], b = hi[u];
    c[2 * u] = a.x * b.x - a.y * b.y;
    s[2 * u] = a.y * b.x + a.x * b.y;
    c[2 * u + 1] = a.z * b.z - a.w * b.w;
    s[2 * u + 1] = a.w * b.z + a.z * b.w;
  }
}
__device__ __forceinline__ void rotate8(float (&x1)[8], float (&x2)[8], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float y = x1[u] * c[u] - x2[u] * s[u];
    x2[u] = x2[u] * c[u] + x1[u] * s[u];
    x1[u] = y;
  }
}

}  // namespace

// Moves bytes: a row is read once and written once, with two table rows of 8 bytes per pair that
// its heads share through L1.  A thread takes eight pairs (16 bytes of each half) of HEADS heads.
// Measured: 4348 rows of 10 heads of 256 (44 MB) 13.8 us, 3.2 TB/s: two waves of CTAs, each as long as
// its chain of loads (slot, then table row); 9465 rows 23.6 us, 4.1 TB/s.  Two heads per thread take
// 13.6 us; 64 registers instead of 80 spill (14.9).  A decode step of 16 rows: 4.3 us.
// The first CTAs look for rows that fill their page, one KV head each, several small pages at a time; a
// CTA's further pages follow one another, at 1.7 us each, so it takes as few rows as the grid allows (16
// rows that fill four pages of 16: 3.3 us, with eight rows to a CTA 8.6; 32 + 16 heads of 128: 3.5, with
// all heads and pages in turn 78).  The mean of such a page needs the rows of this call that other CTAs
// write, so it is computed from their sources again; the page's earlier keys come from the pool.
template <typename T, typename S>
__global__ void __launch_bounds__(WT) k_pages_write(WriteParams p, int mean_ctas, int mean_rows) {
  const PageGeom g = p.g;
  const int d = g.head_dim, half = d / 2, blocks = d / 16;  // blocks of eight pairs
  const int hq = p.n_q_heads, hkv = g.n_kv_heads, heads = hq + 2 * hkv, cap = g.width << g.shift;
  const size_t ld = (size_t)heads * d;
  const S *src = static_cast<const S *>(p.qkv);
  T *k = static_cast<T *>(p.k), *v = static_cast<T *>(p.v), *q = static_cast<T *>(p.q_out);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the attention may be launched
  if ((int)blockIdx.x >= mean_ctas) {
    const int groups = (heads + HEADS - 1) / HEADS;
    const uint32_t item = (blockIdx.x - mean_ctas) * (uint32_t)WT + threadIdx.x;  // at least 32 bytes of qkv each
    const uint32_t at = item / (uint32_t)blocks, r = at / (uint32_t)groups;
    const int i8 = (int)(item % (uint32_t)blocks), h0 = (int)(at - r * groups);  // heads h0, h0 + groups, ...
    if (r >= (uint32_t)p.n_rows) return;
    // the row's values are requested before its slot is known
    const int want = p.slots[r], pos = p.positions[r];
    Raw8<S> raw1[HEADS], raw2[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
      const S *x = src + r * ld + (size_t)min(h0 + u * groups, heads - 1) * d + i8 * 8;
      raw1[u].load(x);
      raw2[u].load(x + half);
    }
    bool bad = false;
    const int slot = pg_slot(want, g, &bad);
    if (slot >= 0 && (pos < 0 || pos >= cap)) bad = true;
    if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_WRITE);
    if (slot < 0 || bad) return;
    float c[8], s[8];
    if (p.rope_lo) rope8(c, s, p, pos, i8, half);
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
      const int h = h0 + u * groups;
      if (h >= heads) break;
      float x1[8], x2[8];
      raw1[u].to(x1);
      raw2[u].to(x2);
      if (p.rope_lo && h < hq + hkv) rotate8(x1, x2, c, s);
      T *dst = h < hq ? q + ((size_t)r * hq + h) * d
                      : h < hq + hkv ? k + pg_elem(p.layer, slot, h - hq, g)
                                     : v + pg_elem(p.layer, slot, h - hq - hkv, g);
      store8(dst + i8 * 8, x1);
      store8(dst + i8 * 8 + half, x2);
    }
    return;
  }
  // ---- page means
  __shared__ float sums[WT * 16];  // [WT / blocks][d]
  __shared__ int slot_s[WT / 4];
  const int ps = 1 << g.shift, i8 = threadIdx.x % blocks, lane_r = threadIdx.x / blocks, n_lanes = WT / blocks;
  // `team` row lanes add the keys of a page, `teams` pages at a time
  const int team = min(ps, n_lanes), teams = n_lanes / team, my_team = lane_r / team;
  // this CTA's KV head, and its rows; every warp looks at 32 of them at a time, one per lane
  const int h = (int)blockIdx.x % hkv, r0 = (int)blockIdx.x / hkv * mean_rows, r1 = min(p.n_rows, r0 + mean_rows);
  const int lane = threadIdx.x & 31;
  for (int g0 = r0; g0 < r1; g0 += 32) {
    int my_slot = -1;  // of a row that fills its page
    if (g0 + lane < r1) {
      bool bad = false;
      my_slot = pg_slot(p.slots[g0 + lane], g, &bad);
      const int at = p.positions[g0 + lane];
      if (at < 0 || at >= cap || (my_slot & (ps - 1)) != ps - 1) my_slot = -1;
    }
    unsigned fills = __ballot_sync(0xffffffffu, my_slot >= 0);
    while (fills) {
      unsigned mine = fills;  // this team's page is the my_team-th
      for (int t = 0; t < teams && fills; ++t) {
        if (t < my_team) mine &= mine - 1;
        fills &= fills - 1;
      }
      const int i = mine ? __ffs(mine) - 1 : 0, r = g0 + i;
      int slot = __shfl_sync(0xffffffffu, my_slot, i);
      if (!mine) slot = -1;
      float a1[8] = {0, 0, 0, 0, 0, 0, 0, 0}, a2[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (slot >= 0) {
#pragma unroll 2
        for (int o = lane_r % team; o < ps; o += team) {
          float x1[8], x2[8];
          // the key `back` tokens before: of this call's row as far before, if that has its slot and is
          // written there (its position may be none)
          const int back = ps - 1 - o, row = r - back, pos = row >= 0 ? p.positions[row] : -1;
          if (pos >= 0 && pos < cap && p.slots[row] == slot - back) {
            const S *x = src + row * ld + (size_t)(hq + h) * d + i8 * 8;
            load8(x1, x);
            load8(x2, x + half);
            if (p.rope_lo) {
              float c[8], s[8];
              rope8(c, s, p, pos, i8, half);
              rotate8(x1, x2, c, s);
            }
          } else {
            const T *x = k + pg_elem(p.layer, slot - back, h, g) + i8 * 8;
            load8(x1, x);
            load8(x2, x + half);
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {  // keys as stored
            a1[u] += to_f(from_f<T>(x1[u]));
            a2[u] += to_f(from_f<T>(x2[u]));
          }
        }
      }
      if (lane_r % team == 0 && i8 == 0) slot_s[my_team] = slot;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sums[lane_r * d + i8 * 8 + u] = a1[u];
        sums[lane_r * d + half + i8 * 8 + u] = a2[u];
      }
      __syncthreads();
      for (int at = threadIdx.x; at < teams * d; at += WT) {
        const int t = at / d, x = at % d;
        if (slot_s[t] < 0) continue;
        float sum = 0.f;
        for (int l = 0; l < team; ++l) sum += sums[(t * team + l) * d + x];
        static_cast<T *>(p.k_mean)[pg_mean_elem(p.layer, slot_s[t] >> g.shift, h, g) + x] = from_f<T>(sum / ps);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------------------
// select

namespace {

constexpr int ST = 512;            // threads of a select CTA
constexpr int SC = 8;              // CTAs of a cluster: they score, the first one chooses
constexpr int RUN = 16;            // pages a warp scores at a time
constexpr int BITS = 9, BINS = 1 << BITS;  // one bin per thread
constexpr int NEAR = 64;           // pages scored again and compared in all pairs
constexpr int SELECT_SMEM_KEYS = 16384;  // candidates whose keys fit shared memory

// Order-preserving maps of scores to integers; 0 (fp32) and 1 (fp64) are kept for pages outside
// the pool, 0 (fp64) for pages that are out already.
__device__ __forceinline__ uint32_t key32(float s) {
  const uint32_t u = __float_as_uint(s);
  return max((u >> 31) ? ~u : u | 0x80000000u, 1u);
}
__device__ __forceinline__ float score32(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long key64(double s) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(s);
  return min(max((u >> 63) ? ~u : u | 0x8000000000000000ull, 2ull), ~1ull);
}

// the eight 16-bit values of v in fp32 (exact)
__device__ __forceinline__ void unpack8(float (&f)[8], const uint4 &v, bf16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(float (&f)[8], const uint4 &v, __half) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// Exclusive scan of one count per thread over the block; total receives the sum.
__device__ int scan_count(int v, int *warp_sums, int &total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto inclusive = [lane](int x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += a;
    }
    return x;
  };
  const int inc = inclusive(v);
  __syncthreads();
  if (lane == 31) warp_sums[w] = inc;
  __syncthreads();
  const int sums = inclusive(lane < ST / 32 ? warp_sums[lane] : 0);
  const int before = __shfl_sync(0xffffffffu, sums, (w + 31) & 31);
  total = __shfl_sync(0xffffffffu, sums, 31);
  return (w ? before : 0) + inc - v;
}

}  // namespace

// One cluster per request and KV head.  The choice is defined by fp64 scores, but fp64 sums are slow
// (with them throughout, selection and attention of 64 of 2040 pages took 23.0 us instead of 21.5),
// so the cluster scores in fp32, 16 bytes of a page's mean per lane, and puts order-preserving
// integer keys into the first CTA's shared memory.  An fp32 score is within
//   E = 16 * 2^-24 * sum_i |q_i| * max |mean|
// of the exact one (8 products and sums in a lane, at most 5 sums over lanes, one rounding of q:
// 14 roundings); where an fp32 sum is not finite, though the exact one may be, E counts as infinite.
// With t the `need`-th highest fp32 score, the `need`-th highest exact one lies within E of t: pages
// above t + 2E are in, pages below t - 2E are out, and only those between are scored again in fp64 -
// with ordinary scores the page at t alone.
//
// t is found by one histogram over equal steps of the score and a comparison of all pairs in the
// deciding step; where that step holds too many (or a bound is not finite), radix passes over the
// keys' bits find it for any values.  If more than NEAR pages lie within 2E of t (equal means,
// scores near zero, NaN), the same radix passes run over fp64 keys in a workspace.
//
// Bound by the chain of loads and barriers, not by bytes: 2040 pages of 256 components (1 MB) take
// about 8 us behind the launch (scores 4300 cycles, the cut 6300, the list 2500), 32 such requests
// of up to 2048 pages about 14.
template <typename T, int D>
__global__ void __cluster_dims__(SC, 1, 1) __launch_bounds__(ST, 2) k_pages_select(SelectParams p) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ double q_sum[D];
  __shared__ float q_32[D];
  __shared__ int bins[BINS], warp_sums[ST / 32];
  __shared__ uint32_t ends[2][ST / 32], big_mean[SC * (ST / 32)], near_key[NEAR];
  __shared__ unsigned long long near_key64[NEAR];
  __shared__ int near_c[NEAR];
  __shared__ float q_size[ST / 32];
  __shared__ int found[3], n_near, n_over;
  __shared__ uint32_t cut_s;
  const PageGeom g = p.g;
  const int rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z, G = p.n_q_heads / g.n_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the attention may be launched
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has started
  constexpr int LPP = D / 8, PPW = 32 / LPP;  // lanes per page, pages per load
  const int sub = lane / LPP, ln = lane % LPP;
  // the sum of the group's query heads, one component per thread; loads that need no length first
  const int32_t *row = p.table + (size_t)b * g.width;
  const int lo = p.keep_first, my_c0 = (warp * SC + rank) * RUN;
  const int raw_page = lane < RUN && lo + my_c0 + lane < g.width ? row[lo + my_c0 + lane] : -1;
  if (threadIdx.x < D) {
    const T *q = static_cast<const T *>(p.q) + ((size_t)b * p.n_q_heads + h * G) * D + threadIdx.x;
    double sum = 0.0;
    for (int j0 = 0; j0 < G; j0 += 8) {
      T v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j0 + j < G ? q[(size_t)(j0 + j) * D] : from_f<T>(0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += (double)to_f(v[j]);
    }
    q_sum[threadIdx.x] = sum;
    q_32[threadIdx.x] = (float)sum;
    const float size = warp_sum(fabsf((float)sum));
    if (lane == 0) q_size[warp] = size;
  }
  bool bad = false;
  const int held = pg_pages(pg_len(p.lens[b], g, &bad), g);
  if (bad && threadIdx.x == 0 && rank == 0 && h == 0) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_SELECT);
  int *sel = p.sel + ((size_t)b * g.n_kv_heads + h) * p.budget;
  // the first CTA's shared memory is written only once all of the cluster's CTAs have started
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (held <= p.budget) {  // the whole cluster leaves here
    for (int i = rank * ST + threadIdx.x; i < p.budget; i += SC * ST) sel[i] = i < held ? i : -1;
    return;
  }
  // candidates: logical pages lo .. lo + n - 1, of which `need` are chosen
  const int n = held - p.keep_last - lo, need = p.budget - lo - p.keep_last;
  // fp32 keys: in shared memory, or for long tables in the lower halves of the workspace's words
  const bool in_smem = g.width <= SELECT_SMEM_KEYS;
  unsigned long long *wide = p.keys + ((size_t)b * g.n_kv_heads + h) * g.width;
  uint32_t *keys = in_smem ? smem_keys : reinterpret_cast<uint32_t *>(wide);
  const int ks = in_smem ? 1 : 2;
  {
    auto in_first = [](void *x) {  // the same variable of the cluster's first CTA
      uint64_t at;
      asm("mapa.u64 %0, %1, %2;" : "=l"(at) : "l"(reinterpret_cast<uint64_t>(x)), "r"(0));
      return reinterpret_cast<void *>(at);
    };
    uint32_t *dst = in_smem ? static_cast<uint32_t *>(in_first(smem_keys)) : keys;
    __syncthreads();  // q_32
    float q[8], big = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) q[u] = q_32[ln * 8 + u];
    for (int c0 = my_c0; c0 < n; c0 += SC * (ST / 32) * RUN) {
      int mine = c0 == my_c0 ? raw_page : lane < RUN && c0 + lane < n ? row[lo + c0 + lane] : -1;
      if (lane >= RUN || c0 + lane >= n) mine = -1;
      else if (!pg_in_pool(mine, g)) {
        bad = true;
        mine = -1;
      }
      // the page's number among all layers' and heads' means; in place of a missing one the run's first
      // (its score is not used, but what is read takes part in the bound)
      const int first = max(__shfl_sync(0xffffffffu, mine, 0), 0), there = mine >= 0 ? mine : first;
      const uint32_t mean_at = ((uint32_t)p.layer * g.n_pages + (uint32_t)there) * g.n_kv_heads + h;
      constexpr int LOADS = LPP / 2 < 8 ? LPP / 2 : 8, STEP = LOADS * PPW;  // loads in flight, their pages
      static_assert(RUN % STEP == 0, "whole steps");
#pragma unroll
      for (int i0 = 0; i0 < RUN; i0 += STEP) {
        uint4 v[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          const uint32_t m = __shfl_sync(0xffffffffu, mean_at, i0 + i * PPW + sub);
          v[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k_mean) + (size_t)m * D + ln * 8);
        }
        float s[LOADS];  // this lane's share of the scores of pages i0 + i * PPW + sub
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          float f[8];
          unpack8(f, v[i], T());
          s[i] = 0.f;
#pragma unroll
          for (int u = 0; u < 8; u += 2) {
            s[i] = fmaf(q[u], f[u], s[i]);
            s[i] = fmaf(q[u + 1], f[u + 1], s[i]);
            big = fmaxf(big, fmaxf(fabsf(f[u]), fabsf(f[u + 1])));
          }
        }
        // sums over the LPP lanes of a page; the first steps halve the pages a lane holds
        int i = 0;
#pragma unroll
        for (int o = LPP / 2, w = LOADS / 2; o > 0; o >>= 1, w >>= 1) {
          if (w > 0) {
            const bool up = lane & o;
            if (up) i += w;
#pragma unroll
            for (int u = 0; u < w; ++u) {
              const float give = up ? s[u] : s[u + w], keep = up ? s[u + w] : s[u];
              s[u] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
          } else {
            s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
          }
        }
        if (!(fabsf(s[0]) < INFINITY)) big = INFINITY;  // no bound: all pages go by fp64
        const int at = i0 + i * PPW + sub, page = __shfl_sync(0xffffffffu, mine, at);
        if (!(lane & (LPP / LOADS - 1)) && c0 + at < n) dst[(c0 + at) * ks] = page < 0 ? 0 : key32(s[0]);
      }
    }
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(big));  // not negative: ordered as bits
    if (lane == 0) static_cast<uint32_t *>(in_first(big_mean))[rank * (ST / 32) + warp] = most;
    if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_SELECT);
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank != 0) return;

  // histogram of digit_of(c) (-1: none); the bin that holds the `left`-th highest, the number in
  // the bins above it and in it
  int above, count;
  auto find = [&](int left, bool together, auto digit_of) {
    bins[threadIdx.x] = 0;
    if (threadIdx.x == 0) n_near = n_over = 0;
    __syncthreads();
    for (int c0 = 0; c0 < n; c0 += ST) {
      const int c = c0 + threadIdx.x, digit = c < n ? digit_of(c) : -1;
      if (together) {  // top bits are shared by many keys: equal lanes are counted at once
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (digit >= 0 && lane == __ffs(same) - 1) atomicAdd(&bins[digit], __popc(same));
      } else if (digit >= 0) {
        atomicAdd(&bins[digit], 1);
      }
    }
    __syncthreads();
    static_assert(BINS == ST, "one bin per thread");
    int total;
    const int bin = BINS - 1 - threadIdx.x, have = bins[bin], over = scan_count(have, warp_sums, total);
    if (over < left && left <= over + have) {
      found[0] = bin;
      found[1] = over;
      found[2] = have;
    }
    __syncthreads();
    above = found[1];
    count = found[2];
    return found[0];
  };

  // chosen are the candidates with keys from `cut` on
  uint32_t cut = ~0u;
  if (need > 0) {
    uint32_t kmin = ~0u, kmax = 0;
    for (int c = threadIdx.x; c < n; c += ST) {
      const uint32_t k = keys[c * ks];
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) {
      ends[0][warp] = kmin;
      ends[1][warp] = kmax;
    }
    __syncthreads();
    kmin = __reduce_min_sync(0xffffffffu, ends[0][lane % (ST / 32)]);
    kmax = __reduce_max_sync(0xffffffffu, ends[1][lane % (ST / 32)]);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < SC * (ST / 32) / 32; ++i) most = max(most, big_mean[i * 32 + lane]);
    most = __reduce_max_sync(0xffffffffu, most);
    const float size = warp_sum(lane < D / 32 ? q_size[lane] : 0.f);
    // (the last term: products below the smallest normal fp32 number)
    const float E = 16.f * 5.9604645e-8f * size * __uint_as_float(most) + 1e-42f;

    // t, the `need`-th highest fp32 key
    uint32_t t = 0;
    auto settle = [&](int left, auto is_near) {  // the `left`-th highest of the `count` <= NEAR keys picked
      for (int c = threadIdx.x; c < n; c += ST)
        if (is_near(c)) near_key[atomicAdd(&n_near, 1)] = keys[c * ks];
      __syncthreads();
      if ((int)threadIdx.x < count) {
        const uint32_t k = near_key[threadIdx.x];
        int over = 0, same = 0;
        for (int i = 0; i < count; ++i) {
          over += near_key[i] > k;
          same += near_key[i] == k;
        }
        if (over < left && left <= over + same) cut_s = k;  // equal keys write equal values
      }
      __syncthreads();
      t = cut_s;
    };
    const float low = score32(kmin), scale = (BINS - 1) / (score32(kmax) - low);
    bool done = false;
    if (low - low == 0.f && scale > 0.f && scale - scale == 0.f) {  // all finite, and not all equal
      // (s - low) * scale rises with s, rounded or not
      auto step = [&](int c) { return min(BINS - 1, (int)((score32(keys[c * ks]) - low) * scale)); };
      const int bin = find(need, false, step);
      if (count <= NEAR) {
        settle(need - above, [&](int c) { return step(c) == bin; });
        done = true;
      }
    }
    uint32_t prefix = 0;
    for (int left = need, shift = 32; !done;) {
      const int width = min(BITS, shift), next = shift - width;
      const int bin = find(left, true, [&](int c) {
        const uint32_t k = keys[c * ks];
        return shift == 32 || k >> shift == prefix ? (int)(k >> next & ((1u << width) - 1)) : -1;
      });
      prefix = shift == 32 ? (uint32_t)bin : prefix << width | (uint32_t)bin;
      shift = next;
      left -= above;
      done = shift == 0 || count <= NEAR;
      if (shift == 0) t = prefix;
      else if (count <= NEAR) settle(left, [&](int c) { return keys[c * ks] >> shift == prefix; });
      __syncthreads();
    }

    // pages within 2E of t (all of them, if there is no bound)
    const float ts = score32(t), reach = 2.f * E;
    const bool bounded = t != 0 && ts - ts == 0.f && reach - reach == 0.f;
    cut = bounded ? key32(__fadd_rd(ts, -reach)) : 0;
    const uint32_t top = bounded ? key32(__fadd_ru(ts, reach)) : ~0u;
    if (threadIdx.x == 0) n_near = n_over = 0;
    __syncthreads();
    for (int c0 = 0; c0 < n; c0 += ST) {
      const int c = c0 + threadIdx.x;
      const uint32_t k = c < n ? keys[c * ks] : 0;
      const bool over = c < n && k > top, within = c < n && k >= cut && !over;
      const unsigned all = __ballot_sync(0xffffffffu, over);
      if (lane == 0 && all) atomicAdd(&n_over, __popc(all));
      if (within) {
        const int at = atomicAdd(&n_near, 1);
        if (at < NEAR) near_c[at] = c;
      }
    }
    __syncthreads();
    const int zone = n_near, left = need - n_over;
    // a whole warp: the exact score of candidate c
    auto exact = [&](int c) {
      const int page = pg_page(row, lo + c, g);
      if (page < 0) return 1ull;
      const T *m = static_cast<const T *>(p.k_mean) + pg_mean_elem(p.layer, page, h, g);
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) s += q_sum[lane + 32 * i] * (double)to_f(m[lane + 32 * i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return key64(s);
    };
    if (zone == left) {
      // all of them
    } else if (zone <= NEAR) {
      for (int i = warp; i < zone; i += ST / 32) {
        const unsigned long long k = exact(near_c[i]);
        if (lane == 0) near_key64[i] = k;
      }
      __syncthreads();
      if ((int)threadIdx.x < zone) {
        const unsigned long long k = near_key64[threadIdx.x];
        const int c = near_c[threadIdx.x];
        int better = 0;
        for (int i = 0; i < zone; ++i)
          better += near_key64[i] > k || (near_key64[i] == k && near_c[i] < c);
        if (better >= left) keys[c * ks] = 0;
        else if (cut == 0) keys[c * ks] = 1;
      }
      cut = max(cut, 1u);
      __syncthreads();
    } else {
      // fp64 keys of the pages between in the workspace (all ones for those in, 0 for those out),
      // then the same passes: the cut, and of the pages equal to it the first ones
      for (int c = warp; c < n; c += ST / 32) {
        const uint32_t k = keys[c * ks];
        const unsigned long long w = k > top ? ~0ull : k >= cut ? exact(c) : 0;
        __syncwarp();
        if (lane == 0) wide[c] = w;
        __syncwarp();
      }
      __syncthreads();
      unsigned long long pre = 0;
      int eq = need, total = 0;
      for (int shift = 64; shift > 0;) {
        const int width = min(BITS, shift), next = shift - width;
        const int bin = find(eq, true, [&](int c) {
          const unsigned long long k = wide[c];
          return k && (shift == 64 || k >> shift == pre) ? (int)(k >> next & ((1u << width) - 1)) : -1;
        });
        pre = shift == 64 ? (unsigned long long)bin : pre << width | (unsigned long long)bin;
        shift = next;
        eq -= above;
        total = count;
        __syncthreads();
      }
      int last = n - 1;  // the last index taken of those equal to the cut
      if (total > eq) {
        unsigned pre_i = 0;
        int want = eq;
        constexpr int IDX_BITS = 27;  // three passes over the complement of the index
        for (int shift = IDX_BITS; shift > 0; shift -= BITS) {
          const int next = shift - BITS;
          const int bin = find(want, true, [&](int c) {
            const unsigned i = (1u << IDX_BITS) - 1 - (unsigned)c;
            return wide[c] == pre && (shift == IDX_BITS || i >> shift == pre_i) ? (int)(i >> next & (BINS - 1)) : -1;
          });
          pre_i = pre_i << BITS | (unsigned)bin;
          want -= above;
          __syncthreads();
        }
        last = (int)((1u << IDX_BITS) - 1 - pre_i);
      }
      // 1: chosen, 0: not
      for (int c = threadIdx.x; c < n; c += ST) {
        const unsigned long long w = wide[c];
        keys[c * ks] = w > pre || (w == pre && c <= last);
      }
      cut = 1;
      __syncthreads();
    }
  }
  // the chosen pages in order: 32 flags to a word, a word to a thread
  if (need > 0) {
    int done = lo;
    for (int base = 0; base < n; base += ST * 32) {
      for (int c0 = base; c0 < min(n, base + ST * 32); c0 += ST) {
        const int c = c0 + threadIdx.x;
        const unsigned word = __ballot_sync(0xffffffffu, c < n && keys[c * ks] >= cut);
        if (lane == 0) bins[(c - base) >> 5] = (int)word;
      }
      __syncthreads();
      const int words = (min(n - base, ST * 32) + ST - 1) / ST * (ST / 32);
      unsigned word = (int)threadIdx.x < words ? (unsigned)bins[threadIdx.x] : 0u;
      int total, at = done + scan_count(__popc(word), warp_sums, total);
      for (; word; word &= word - 1) sel[at++] = lo + base + threadIdx.x * 32 + __ffs(word) - 1;
      done += total;
      __syncthreads();
    }
  }
  for (int i = threadIdx.x; i < lo; i += ST) sel[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += ST) sel[p.budget - p.keep_last + i] = held - p.keep_last + i;
}

// ---------------------------------------------------------------------------------------
// launchers

namespace {
// (cos, sin) of positions step * row, angle = position * theta^(-2 i / d) in fp64, rounded once
__global__ void k_rope_table(float2 *dst, int rows, int step, int half, double theta) {
  const size_t n = (size_t)rows * half;
  for (size_t at = (size_t)blockIdx.x * blockDim.x + threadIdx.x; at < n; at += (size_t)gridDim.x * blockDim.x) {
    double s, c;
    sincos((double)(at / half) * step * pow(theta, -(double)(at % half) / half), &s, &c);
    dst[at] = make_float2((float)c, (float)s);
  }
}
}  // namespace

cudaError_t launch_rope_table(float2 *dst, int rows, int step, int head_dim, double theta, cudaStream_t st) {
  k_rope_table<<<592, 256, 0, st>>>(dst, rows, step, head_dim / 2, theta);
  return cudaGetLastError();
}

cudaError_t launch_pages_plan(const PlanParams &p, int sm_count, cudaStream_t st) {
  // A CTA's time is the scans over the requests: 1024 threads from 256 requests on (2000 requests and
  // 91 thousand rows: 13.9 us, with 256 threads 17.1).  Two rows per thread: every CTA repeats the
  // scans, so more of them only help until each SM has one.
  const bool many = p.batch > 256;
  const int threads = many ? 1024 : 256, want = (p.n_rows + 2 * threads - 1) / (2 * threads);
  const int ctas = want < 1 ? 1 : want < sm_count ? want : sm_count;
  if (many) k_pages_plan<1024><<<ctas, threads, plan_smem(p.batch), st>>>(p);
  else k_pages_plan<256><<<ctas, threads, plan_smem(p.batch), st>>>(p);
  return cudaGetLastError();
}

namespace {
template <typename T, typename S>
cudaError_t write(const WriteParams &p, int sm_count, cudaStream_t st) {
  const int heads = p.n_q_heads + 2 * p.g.n_kv_heads;
  const long long items = (long long)p.n_rows * ((heads + HEADS - 1) / HEADS) * (p.g.head_dim / 16);
  const long long move = (items + WT - 1) / WT;
  // the means' CTAs search one row each, or as many (a power of two) as let at most MEAN_CTAS fall to an SM
  // (one per SM: 4348 rows 13.9 -> 15.1 us, 2365 rows 9.6 -> 9.0)
  int rows = 1;
  const long long most = (long long)MEAN_CTAS * sm_count;
  while (rows < p.n_rows && (long long)((p.n_rows + rows - 1) / rows) * p.g.n_kv_heads > most) rows *= 2;
  const int mean = p.k_mean ? (p.n_rows + rows - 1) / rows * p.g.n_kv_heads : 0;
  k_pages_write<T, S><<<(unsigned)(move + mean), WT, 0, st>>>(p, mean, rows);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_pages_write(const WriteParams &p, int dtype, int src_dtype, int sm_count, cudaStream_t st) {
  if (p.n_rows == 0) return cudaSuccess;
  const bool f32 = src_dtype == RTVLA_DTYPE_F32;
  if (dtype == RTVLA_DTYPE_BF16) return f32 ? write<bf16, float>(p, sm_count, st) : write<bf16, bf16>(p, sm_count, st);
  return f32 ? write<__half, float>(p, sm_count, st) : write<__half, __half>(p, sm_count, st);
}

namespace {
size_t select_smem(const PageGeom &g) { return g.width <= SELECT_SMEM_KEYS ? (size_t)g.width * 4 : 0; }

template <typename T>
cudaError_t select_attributes(int head_dim) {
  const auto kernel = head_dim == 64    ? k_pages_select<T, 64>
                      : head_dim == 128 ? k_pages_select<T, 128>
                                        : k_pages_select<T, 256>;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SELECT_SMEM_KEYS * 4);
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

cudaError_t pages_init_attributes(int dtype, int head_dim) {
  const cudaError_t e =
      cudaFuncSetAttribute(k_pages_plan<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(4096));
  if (e != cudaSuccess) return e;
  return dtype == RTVLA_DTYPE_BF16 ? select_attributes<bf16>(head_dim) : select_attributes<__half>(head_dim);
}

cudaError_t launch_pages_select(const SelectParams &p, int dtype, cudaStream_t st) {
  return dtype == RTVLA_DTYPE_BF16 ? select<bf16>(p, st) : select<__half>(p, st);
}

}  // namespace rtvla
