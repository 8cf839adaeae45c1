// Attention of one query token per request over its pages: out = softmax(q K^T / sqrt(d)) V.
//
// Every key and value is read once and used by the G = n_q_heads / n_kv_heads heads that share
// it, 4 G d flops per 4 d bytes: far below the tensor cores' 250 flops per byte, so the kernel is
// built to keep HBM busy, and the products run on mma.sync m16n8k16 tiles because those take the
// G heads as the narrow side (N = 8): S^T = K Q^T with 16 keys as M, O^T = V^T P^T with 16
// components of d as M.  (A tcgen05 tile has M >= 64 and its operands in one shared buffer per
// CTA; with 8 query rows it would only add barriers.)
//
// One warp owns a 16-key tile and a private ring filled by cp.async, K and V tiles in turn, so that
// nothing in the main loop waits for another warp; each warp keeps its own running maximum, sum and
// O^T in registers.  At the end of a request's keys the four warps' results are joined in shared
// memory.  Three tiles per warp and two CTAs per SM (d = 256) keep 128 KB per SM in flight; three
// pairs of tiles and one CTA per SM keep as much but leave an SM idle at the end of each request
// (16 requests of 800 tokens: 13.8 us, with two CTAs 11.8; 64 of up to 32768: 178.7 and 181.3).
//
// The work is split evenly whatever the lengths (k_pages_attend): the 64-key chunks of all (request,
// KV head) pairs, in order, are cut into one contiguous range per CTA.  A pair that lies inside one
// range is finished there; of one that is cut each part goes to a workspace in fp32 and k_pages_join
// adds the parts.  Both kernels find their place by summing the lengths themselves, so no plan has
// to be made on the host and a captured graph stays valid when the lengths change.  (Adding the parts
// in the attention kernel, by the CTA that finishes last, leaves one SM to do it: 16 requests of 800
// tokens 14.3 us instead of 11.3, one of 131071 38.4 instead of 32.0.)  A few pairs of bounded length
// go to k_pages_attend_cluster, which joins through shared memory.
//
// Measured: 64 requests of up to 32768 tokens, 8 heads of 256 on one KV head (1.13 GB of K and V),
// 179 to 181 us, 6.3 TB/s, 96% of the GPU's measured copy rate; 24 ragged requests, 32/8 heads of 128
// in f16 (351 MB) 65 us, 5.4 TB/s; one request of 131071 tokens (134 MB) 33 us, of which the reading
// takes 21 and the start, the last tiles and the join the rest.  Short calls are latency: 7.9 us
// for one request of 544 tokens, 9.9 for 16 of 800.
//
// Weights are split into two 16-bit parts, p = hi + lo, and multiplied twice: the products cost
// nothing next to the loads, and the weights then count to 2^-16 (bf16) or 2^-22 (f16) instead of
// 2^-8 or 2^-11.  f16 has no numbers below 2^-24, so its parts are those of 2^15 p (at most 32768, of
// 65504): what is lost of a small weight is at most 2^-40 of the largest.
#include <cuda_fp16.h>

#include <algorithm>

#include "pages.h"
#include "rtvla.h"

namespace rtvla {

namespace {

constexpr int WARPS = 4;
constexpr int CHUNK = 64;  // keys per unit of work: one 16-key tile per warp
constexpr int SETUP = 1;   // units that starting a pair and joining its warps count in the split
constexpr int SLOTS = 3;   // ring of a warp: tiles of 16 rows, K and V in turn
constexpr int MAX_CTAS = 1024;  // of one launch
constexpr int CLUSTER = 8;      // CTAs that share a pair, when there are few pairs

__device__ __forceinline__ void put(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half *p, float v) { *p = __float2half_rn(v); }

// two weights as (first in the low half) 16-bit hi parts and the 16-bit rest, of P_SCALE times each
template <typename T>
constexpr float P_SCALE = 1.f;
template <>
constexpr float P_SCALE<__half> = 32768.f;
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo, bf16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - __low2float(h), b - __high2float(h));
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo, __half) {
  a *= P_SCALE<__half>;
  b *= P_SCALE<__half>;
  const __half2 h = __floats2half2_rn(a, b);
  const __half2 l = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&l);
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bf16) {
  mma_16816(c, a[0], a[1], a[2], a[3], b0, b1);
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// transposes an 8 x 8 tile of 16-bit values spread over the warp as an mma accumulator row pair
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// 16 bytes global -> shared, zeros when !take (nothing is read then)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// units of work of request b (of each of its KV heads): its chunks, behind SETUP units for what
// every pair costs besides
__device__ __forceinline__ int units_of(const PagedAttnParams &p, int b) {
  bool bad = false;
  const int len = pg_len(p.lens[b], p.g, &bad);
  const int n = pg_list_len(len, p.sel_width, p.sel != nullptr, p.g);
  return n > 0 ? (n + CHUNK - 1) / CHUNK + SETUP : 0;
}

// a / b (a >= 0, b > 0), in 32 bits where they suffice: a 64-bit division takes a hundred
// instructions on the way to the first load
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((unsigned long long)(a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// byte offset of 16-byte chunk c of row r in a tile of D-wide 16-bit rows: chunks are XORed with
// the row so that the 8 rows of an ldmatrix fall on different banks
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

template <int D, int NT>
struct Smem {
  static constexpr int TILE = 16 * D * 2;                 // bytes of 16 rows
  static constexpr int RING = SLOTS * TILE;               // one warp's ring
  static constexpr int Q = NT * 8 * D * 2;
  static constexpr int OLD = D + 4;                       // floats per head of a warp's result
  static constexpr int TOTAL = WARPS * RING + Q;
  static_assert(NT * 8 * OLD * 4 <= RING, "a warp's result fits its ring");
};

// the same variable of the cluster's CTA `rank`
__device__ __forceinline__ const void *in_cta(const void *x, int rank) {
  uint64_t at;
  asm("mapa.u64 %0, %1, %2;" : "=l"(at) : "l"(reinterpret_cast<uint64_t>(x)), "r"(rank));
  return reinterpret_cast<const void *>(at);
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CTAs that fit on an SM by shared memory (227 KB, 1 KB of it per CTA reserved)
template <int D, int NT>
constexpr int ctas_per_sm() {
  const int fit = (227 * 1024) / (Smem<D, NT>::TOTAL + 2048);
  return fit < 4 ? fit : 4;
}

// Chunks [c0, c1) of request b and KV head h, of the n keys it attends to: every warp takes the tiles
// `warp`, `warp` + 4, ...  Leaves each warp's result in its ring ([head][OLD] floats, unnormalised) and
// its maximum (log2 units) and sum in ml_s, behind a barrier.
template <typename T, int D, int NT>
__device__ __forceinline__ void attend_chunks(const PagedAttnParams &p, uint8_t *smem, float2 (*ml_s)[NT * 8], int b,
                                              int h, int len, int n, int c0, int c1, bool &bad) {
  using S = Smem<D, NT>;
  const PageGeom &g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t4 = lane & 3;
  const int G = p.n_q_heads / g.n_kv_heads;
  uint8_t *ring = smem + warp * S::RING;
  const uint32_t ring_a = smem_u32(ring), q_a = smem_u32(smem + WARPS * S::RING);
  const T *kp = static_cast<const T *>(p.k), *vp = static_cast<const T *>(p.v);
  const int32_t *trow = p.table + (size_t)b * g.width;
  const int32_t *sel = p.sel ? p.sel + ((size_t)b * g.n_kv_heads + h) * p.sel_width : nullptr;
  const int tiles_end = min(c1 * 4, (n + 15) >> 4);

  // row of the cache (all layers, pages and heads counted together) of key j, or ~0
  auto row_of = [&](int j) -> uint32_t {
    const int r = pg_key_row(trow, sel, j, n, len, g, &bad);
    if (r < 0) return ~0u;
    return (uint32_t)(((((size_t)p.layer * g.n_pages + (r >> g.shift)) * g.n_kv_heads + h) << g.shift) +
                      (r & ((1 << g.shift) - 1)));
  };
  // requests the tile of K or V rows (lanes 0..15 hold them) into a slot, as one group
  auto load = [&](const T *src, int slot, uint32_t rows) {
    constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte chunks per row, rows per instruction
    const int c = lane % CPR;
#pragma unroll
    for (int i = 0; i < 16 / RPI; ++i) {
      const int r = i * RPI + lane / CPR;
      const uint32_t at = __shfl_sync(0xffffffffu, rows, r);
      const bool take = at != ~0u;
      copy16(ring_a + slot * S::TILE + tile_at<D>(r, c), src + (take ? (size_t)at * D : 0) + c * 8, take);
    }
  };
  auto rows_of = [&](int t) { return lane < 16 && t < tiles_end ? row_of(t * 16 + lane) : ~0u; };

  // the ring holds K and V of this tile in slots `slot` and `slot` + 1
  int tile = c0 * 4 + warp, slot = 0;
  uint32_t row = rows_of(tile);
  if (tile < tiles_end) load(kp, 0, row);
  copy_commit();
  if (tile < tiles_end) load(vp, 1, row);
  copy_commit();
  uint32_t live = __ballot_sync(0xffffffffu, row != ~0u);
  row = rows_of(tile + WARPS);
  // the group's query heads, zero rows past G
  {
    const T *q = static_cast<const T *>(p.q) + ((size_t)b * p.n_q_heads + h * G) * D;
    for (int i = threadIdx.x; i < NT * 8 * (D / 8); i += WARPS * 32) {
      const int r = i / (D / 8), c = i % (D / 8);
      const uint4 v = r < G ? *reinterpret_cast<const uint4 *>(q + (size_t)r * D + c * 8) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(smem + WARPS * S::RING + tile_at<D>(r, c)) = v;
    }
  }
  __syncthreads();

  float o[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
  }

#pragma unroll 1
  for (; tile < tiles_end; tile += WARPS) {
    const int slot1 = slot == SLOTS - 1 ? 0 : slot + 1, slot2 = slot1 == SLOTS - 1 ? 0 : slot1 + 1;
    const bool more = tile + WARPS < tiles_end;
    const uint32_t ka = ring_a + slot * S::TILE, va = ring_a + slot1 * S::TILE;
    copy_wait<1>();  // this tile's K
    __syncwarp();    // and every lane is done with slot2, the last tile's V
    if (more) load(kp, slot2, row);
    copy_commit();

    // S^T = K Q^T: rows (keys) gq and gq + 8, columns (heads) 2 t4 and 2 t4 + 1
    float s[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][0][e] = s[nt][1][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; kk += 2) {
      uint32_t a[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        ldsm_x4(a[u][0], a[u][1], a[u][2], a[u][3],
                ka + tile_at<D>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * (kk + u) + (lane >> 4)));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t q0, q1, q2, q3;
        ldsm_x4(q0, q1, q2, q3, q_a + tile_at<D>(nt * 8 + (lane & 7), 2 * kk + (lane >> 3)));
        mma(s[nt][0], a[0], q0, q1, T());
        mma(s[nt][1], a[1], q2, q3, T());
      }
    }
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = (live >> (gq + (e >> 1) * 8)) & 1 ? (s[nt][0][e] + s[nt][1][e]) * p.scale_log2 : -INFINITY;
      float a[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float cm = fmaxf(x[e], x[e + 2]);
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, w));
        const float nm = fmaxf(m[nt][e], cm), ref = nm == -INFINITY ? 0.f : nm;
        a[e] = exp2f(m[nt][e] - ref);
        m[nt][e] = nm;
        x[e] = exp2f(x[e] - ref);
        x[e + 2] = exp2f(x[e + 2] - ref);
        l[nt][e] = l[nt][e] * a[e] + (x[e] + x[e + 2]);
      }
      if (__any_sync(0xffffffffu, a[0] != 1.f || a[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][nt][0] *= a[0];
          o[i][nt][1] *= a[1];
          o[i][nt][2] *= a[0];
          o[i][nt][3] *= a[1];
        }
      }
      split2(x[0], x[1], hi[nt][0], lo[nt][0], T());
      split2(x[2], x[3], hi[nt][1], lo[nt][1], T());
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        hi[nt][e] = transpose8(hi[nt][e]);
        lo[nt][e] = transpose8(lo[nt][e]);
      }
    }
    copy_wait<1>();  // this tile's V
    __syncwarp();    // and every lane is done with this tile's K
    if (more) load(vp, slot, row);
    copy_commit();
    live = __ballot_sync(0xffffffffu, row != ~0u);
    row = rows_of(tile + 2 * WARPS);
    // O^T += V^T P^T: rows (components) 16 i + gq and + 8, columns (heads) 2 t4 and 2 t4 + 1
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      ldsm_x4_t(a[0], a[1], a[2], a[3],
                va + tile_at<D>((lane & 7) + (lane >> 4) * 8, 2 * i + ((lane >> 3) & 1)));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma(o[i][nt], a, hi[nt][0], hi[nt][1], T());
        mma(o[i][nt], a, lo[nt][0], lo[nt][1], T());
      }
    }
    slot = slot2;
  }
  __syncwarp();

  // ---- join the warps: each puts its result into its own ring
  float *so = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[nt][e];
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      const int head = nt * 8 + 2 * t4 + e;
      if (gq == 0) ml_s[warp][head] = make_float2(m[nt][e], sum);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        so[head * S::OLD + 16 * i + gq] = o[i][nt][e] * (1.f / P_SCALE<T>);
        so[head * S::OLD + 16 * i + gq + 8] = o[i][nt][e + 2] * (1.f / P_SCALE<T>);
      }
    }
  __syncthreads();
}

// components d .. d + 3 of one head over the four warps' results; M and L: their maximum and sum
template <int D, int NT>
__device__ __forceinline__ float4 warps_sum(const uint8_t *smem, const float2 (*ml_s)[NT * 8], int head, int d,
                                            float &M, float &L) {
  using S = Smem<D, NT>;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml_s[w][head].x);
  const float ref = M == -INFINITY ? 0.f : M;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  L = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const float f = exp2f(ml_s[w][head].x - ref);
    const float4 x =
        *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * S::RING) + head * S::OLD + d);
    L += f * ml_s[w][head].y;
    v.x += f * x.x;
    v.y += f * x.y;
    v.z += f * x.z;
    v.w += f * x.w;
  }
  return v;
}

// four components of the output from their weighted sum and the sum of the weights
template <typename T>
__device__ __forceinline__ void put4(T *out, const float4 &v, float L) {
  const float inv = L > 0.f ? 1.f / L : 0.f;
  put(out, v.x * inv);
  put(out + 1, v.y * inv);
  put(out + 2, v.z * inv);
  put(out + 3, v.w * inv);
}

}  // namespace

// NT: query heads in tiles of 8 (1: G <= 8, 2: G <= 16)
template <typename T, int D, int NT>
__global__ void __launch_bounds__(WARPS * 32, ctas_per_sm<D, NT>()) k_pages_attend(PagedAttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long warp_sum_s[WARPS];
  __shared__ long long first_at;
  __shared__ int first_b;
  __shared__ float2 ml_s[WARPS][NT * 8];
  const PageGeom g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.n_q_heads / g.n_kv_heads, B = p.batch;
  // Launched while the kernel before it may still run (rtvla_pages_write and _select let it), so
  // nothing is read before this; the join is launched likewise.
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's range of units, and the request it starts in
  const int per = (B + WARPS * 32 - 1) / (WARPS * 32);
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  long long mine = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    mine += units_of(p, b);
    if (blockIdx.x == 0) pg_len(p.lens[b], g, &bad);
  }
  if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_ATTEND);
  if (threadIdx.x == 0) {
    first_b = 0;
    first_at = 0;
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) warp_sum_s[warp] = inc;
  __syncthreads();
  long long before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += warp_sum_s[w];
    total += warp_sum_s[w];
  }
  total *= g.n_kv_heads;
  before *= g.n_kv_heads;
  const long long ctas = min(total, (long long)gridDim.x);  // those with work: every range holds a unit
  if (blockIdx.x >= ctas) return;
  const long long start = quotient(total * blockIdx.x, ctas), end = quotient(total * (blockIdx.x + 1), ctas);
  if (before <= start && start < before + mine * g.n_kv_heads) {
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const long long n = (long long)units_of(p, b) * g.n_kv_heads;
      if (start < before + n) break;
      before += n;
    }
    first_b = b;
    first_at = start - before;
  }
  __syncthreads();
  int b = first_b, n_units = max(units_of(p, b), 1);
  int h = min((int)quotient(first_at, n_units), g.n_kv_heads - 1), u0 = (int)(first_at - (long long)h * n_units);
  long long at = start;  // unit of the whole work

  while (true) {
    // ---- one segment: chunks [c0, c1) of (b, h)
    const int u1 = (int)min((long long)n_units, u0 + (end - at));
    const int c0 = max(u0 - SETUP, 0), c1 = u1 - SETUP, n_chunks = n_units - SETUP;
    if (c1 > c0) {
      const int len = pg_len(p.lens[b], g, &bad);
      const int n = pg_list_len(len, p.sel_width, p.sel != nullptr, g);
      attend_chunks<T, D, NT>(p, smem, ml_s, b, h, len, n, c0, c1, bad);
      const bool whole = c0 == 0 && c1 == n_chunks;
      // a CTA's parts: of a pair that began before it, and of one that goes on after it
      const size_t part = (size_t)blockIdx.x * 2 + (c0 == 0 ? 1 : 0);
      for (int i = threadIdx.x; i < G * (D / 4); i += WARPS * 32) {
        const int head = i / (D / 4), d = (i % (D / 4)) * 4;
        float M, L;
        const float4 v = warps_sum<D, NT>(smem, ml_s, head, d, M, L);
        if (whole) {
          put4(static_cast<T *>(p.out) + ((size_t)b * p.n_q_heads + h * G + head) * D + d, v, L);
        } else {
          *reinterpret_cast<float4 *>(p.part_o + (part * G + head) * D + d) = v;
          if (d == 0) p.part_ml[part * G + head] = make_float2(M, L);
        }
      }
    }
    at += u1 - u0;
    if (at >= end) break;
    __syncthreads();
    u0 = 0;
    if (++h == g.n_kv_heads) {  // the next request that holds anything
      h = 0;
      for (++b; b < B; b += 32) {
        const int c = b + lane < B ? units_of(p, b + lane) : 0;
        const unsigned some = __ballot_sync(0xffffffffu, c > 0);
        if (some) {
          const int to = __ffs(some) - 1;
          n_units = __shfl_sync(0xffffffffu, c, to);
          b += to;
          break;
        }
      }
      if (b >= B) break;  // only if the lengths changed under the kernel
    }
  }
  if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_ATTEND);
}

// The same for few pairs of bounded length: a cluster per (request, KV head), its CTAs share the
// chunks evenly and add their results through each other's shared memory, so that there is neither
// a workspace nor a second kernel.
template <typename T, int D, int NT>
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(WARPS * 32, ctas_per_sm<D, NT>())
    k_pages_attend_cluster(PagedAttnParams p) {
  using S = Smem<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 ml_s[WARPS][NT * 8], sum_s[NT * 8];
  const PageGeom g = p.g;
  const int rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z, G = p.n_q_heads / g.n_kv_heads;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // as k_pages_attend
  bool bad = false;
  const int len = pg_len(p.lens[b], g, &bad);
  const int n = pg_list_len(len, p.sel_width, p.sel != nullptr, g), chunks = (n + CHUNK - 1) / CHUNK;
  const int c0 = chunks * rank / CLUSTER, c1 = chunks * (rank + 1) / CLUSTER;
  if (c1 > c0) {
    attend_chunks<T, D, NT>(p, smem, ml_s, b, h, len, n, c0, c1, bad);
    // the warps' sum takes the place of warp 0's result: a thread reads and writes its own components
    for (int i = threadIdx.x; i < G * (D / 4); i += WARPS * 32) {
      const int head = i / (D / 4), d = (i % (D / 4)) * 4;
      float M, L;
      const float4 v = warps_sum<D, NT>(smem, ml_s, head, d, M, L);
      *reinterpret_cast<float4 *>(reinterpret_cast<float *>(smem) + head * S::OLD + d) = v;
      if (d == 0) sum_s[head] = make_float2(M, L);
    }
  } else if (threadIdx.x < NT * 8) {
    sum_s[threadIdx.x] = make_float2(-INFINITY, 0.f);
  }
  if (bad) set_error(p.ctl, DEVERR_BOUNDS, PG_AT_ATTEND);
  cluster_barrier();
  // each CTA adds a share of the components over all of them
  for (int i = rank * WARPS * 32 + threadIdx.x; i < G * (D / 4); i += CLUSTER * WARPS * 32) {
    const int head = i / (D / 4), d = (i % (D / 4)) * 4;
    float2 ml[CLUSTER];
    float4 x[CLUSTER];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r) {
      ml[r] = *static_cast<const float2 *>(in_cta(&sum_s[head], r));
      x[r] = *static_cast<const float4 *>(in_cta(reinterpret_cast<float *>(smem) + head * S::OLD + d, r));
      M = fmaxf(M, ml[r].x);
    }
    const float ref = M == -INFINITY ? 0.f : M;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r) {
      if (ml[r].x == -INFINITY && ml[r].y == 0.f) continue;  // no keys: its shared memory holds no result
      const float f = exp2f(ml[r].x - ref);
      L += f * ml[r].y;
      v.x += f * x[r].x;
      v.y += f * x[r].y;
      v.z += f * x[r].z;
      v.w += f * x[r].w;
    }
    put4(static_cast<T *>(p.out) + ((size_t)b * p.n_q_heads + h * G + head) * D + d, v, L);
  }
  cluster_barrier();  // no CTA leaves while others read its shared memory
}

// Adds the parts of one (request, query head) that was cut across CTAs of k_pages_attend, and
// writes the zeros of a request that holds nothing.  A CTA joins W of the D components: W / 4
// threads side by side, the others share the parts.  Launched before the parts are complete; it
// finds its place meanwhile.
template <typename T, int D, int JOIN_THREADS, int W>
__global__ void __launch_bounds__(JOIN_THREADS) k_pages_join(PagedAttnParams p, int grid) {
  constexpr int COLS = W / 4, ROWS = JOIN_THREADS / COLS;
  __shared__ long long sum_s[2][JOIN_THREADS / 32];
  __shared__ float red_s[2][JOIN_THREADS / 32];
  __shared__ float4 acc_s[ROWS][COLS];
  __shared__ float2 part_s[MAX_CTAS];  // per part: maximum (then weight) and sum
  const PageGeom g = p.g;
  const int hq = blockIdx.x / (D / W), b = blockIdx.y, G = p.n_q_heads / g.n_kv_heads, h = hq / G;
  const int d0 = blockIdx.x % (D / W) * W;  // first component
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long before = 0, total = 0;
  for (int i = threadIdx.x; i < p.batch; i += JOIN_THREADS) {
    const long long c = units_of(p, i);
    total += c;
    if (i < b) before += c;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, w);
    total += __shfl_xor_sync(0xffffffffu, total, w);
  }
  if (lane == 0) {
    sum_s[0][warp] = before;
    sum_s[1][warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < JOIN_THREADS / 32; ++w) {
    before += sum_s[0][w];
    total += sum_s[1][w];
  }
  const long long n = units_of(p, b);
  T *out = static_cast<T *>(p.out) + ((size_t)b * p.n_q_heads + hq) * D + d0;
  total *= g.n_kv_heads;
  const long long x0 = before * g.n_kv_heads + n * h, x1 = x0 + n;
  const long long ctas = max(min(total, (long long)grid), 1ll);
  // unit x belongs to the CTA c with total c / ctas <= x < total (c + 1) / ctas
  const int from = n ? (int)quotient((x0 + SETUP + 1) * ctas - 1, total) : 0;
  const int to = n ? (int)quotient(x1 * ctas - 1, total) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n == 0) {
    for (int i = threadIdx.x; i < W; i += JOIN_THREADS) put(out + i, 0.f);
    return;
  }
  const int parts = to - from + 1;
  if (parts == 1) return;  // finished where it was computed
  const int head = hq - h * G;
  auto part = [&](int i) {  // the i-th part's place in the workspace
    return ((size_t)(from + i) * 2 + (i == 0 ? 1 : 0)) * G + head;
  };
  // eight loads in flight, the first ones before the weights are known
  const int col = threadIdx.x % COLS, row = threadIdx.x / COLS;
  float4 x[8];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * ROWS;
      x[u] = i < parts ? *reinterpret_cast<const float4 *>(p.part_o + part(i) * D + d0 + col * 4)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(row);
  // weight of every part: 2^(m_i - M) / sum_i 2^(m_i - M) l_i
  float M = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += JOIN_THREADS) {
    const float2 ml = p.part_ml[part(i)];
    part_s[i] = ml;
    M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  if (lane == 0) red_s[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < JOIN_THREADS / 32; ++w) M = fmaxf(M, red_s[0][w]);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int i = threadIdx.x; i < parts; i += JOIN_THREADS) {
    const float f = exp2f(part_s[i].x - ref);
    L += f * part_s[i].y;
    part_s[i].x = f;
  }
  L = warp_sum(L);
  if (lane == 0) red_s[1][warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < JOIN_THREADS / 32; ++w) L += red_s[1][w];
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = row; i0 < parts;) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float f = i0 + u * ROWS < parts ? part_s[i0 + u * ROWS].x : 0.f;
      v.x += f * x[u].x;
      v.y += f * x[u].y;
      v.z += f * x[u].z;
      v.w += f * x[u].w;
    }
    i0 += 8 * ROWS;
    if (i0 < parts) load(i0);
  }
  acc_s[row][col] = v;
  __syncthreads();
  if (row != 0) return;
#pragma unroll
  for (int r = 1; r < ROWS; ++r) {
    const float4 x = acc_s[r][col];
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  put4(out + col * 4, v, L);
}

namespace {

template <typename T, int D, int NT>
cudaError_t attend(const PagedAttnParams &p, int sm_count, cudaStream_t st) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = Smem<D, NT>::TOTAL;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const long long keys = (long long)(p.sel && p.sel_width < p.g.width ? p.sel_width : p.g.width) << p.g.shift;
  const long long wave = std::min(sm_count * ctas_per_sm<D, NT>(), MAX_CTAS);
  const long long pairs = (long long)p.batch * p.g.n_kv_heads, chunks = (keys + CHUNK - 1) / CHUNK;
  // Clusters save the parts and the second launch, about 2.5 us, but give a CTA up to chunks / CLUSTER
  // chunks where an even split over the whole wave gives fewer; one more costs 1.4 us at d = 256 and
  // 0.8 below.  One request of 1000 tokens: 7.5 us (split 8.1), of 2000: 10.4 (8.7) at d = 256, 8.0
  // (8.3) at d = 128; 16 requests of 1000: 10.1 (12.7).  Past half a wave clusters no longer fit at once
  // (37 requests of 1000: 20.3, split 17.6).  The lengths are on the GPU, so the rule goes by what the
  // table rows or the lists have room for; the figures are for rows just as long as the requests.  With
  // rows for 8192 tokens one request of 544 takes the split form and 0.9 us more, 16 of 800 1.0 more.
  const long long most_c = (chunks + CLUSTER - 1) / CLUSTER, most_s = (pairs * (chunks + SETUP) + wave - 1) / wave;
  if (pairs * CLUSTER * 2 <= wave && most_c - most_s <= (D == 256 ? 1 : 3)) {
    cfg.gridDim = dim3(CLUSTER, p.g.n_kv_heads, p.batch);
    return cudaLaunchKernelEx(&cfg, k_pages_attend_cluster<T, D, NT>, p);
  }
  // otherwise one wave of CTAs, but no more than there can be units
  const long long most = pairs * (chunks + SETUP);
  const int ctas = (int)(most < wave ? most : wave);
  cfg.gridDim = dim3(ctas);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_pages_attend<T, D, NT>, p);
  if (e != cudaSuccess) return e;
  // Few (request, head) pairs have many parts each and take 512 threads; many pairs have few parts,
  // and most of their CTAs only find that there is nothing to do: smaller ones pass faster (24 x 32
  // pairs: 64.2 us with 256 threads, 71.2 with 512; one pair of 148 parts: 49.0 and 36.7 us).
  const bool few = (long long)p.n_q_heads * p.batch * (D / 64) <= sm_count;
  cfg.gridDim = dim3(p.n_q_heads * (few ? D / 64 : 1), p.batch);
  cfg.blockDim = dim3(few ? 512 : 256);
  cfg.dynamicSmemBytes = 0;
  return few ? cudaLaunchKernelEx(&cfg, k_pages_join<T, D, 512, 64>, p, ctas)
             : cudaLaunchKernelEx(&cfg, k_pages_join<T, D, 256, D>, p, ctas);
}

template <typename T, int D>
cudaError_t attend(const PagedAttnParams &p, int sm_count, cudaStream_t st) {
  return p.n_q_heads / p.g.n_kv_heads <= 8 ? attend<T, D, 1>(p, sm_count, st) : attend<T, D, 2>(p, sm_count, st);
}

template <typename T>
cudaError_t attend(const PagedAttnParams &p, int sm_count, cudaStream_t st) {
  if (p.g.head_dim == 64) return attend<T, 64>(p, sm_count, st);
  return p.g.head_dim == 128 ? attend<T, 128>(p, sm_count, st) : attend<T, 256>(p, sm_count, st);
}

template <typename T, int D, int NT>
cudaError_t allow_smem() {
  const cudaError_t e =
      cudaFuncSetAttribute(k_pages_attend<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, NT>::TOTAL);
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(k_pages_attend_cluster<T, D, NT>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, NT>::TOTAL);
}

template <typename T, int D>
cudaError_t allow_smem(int group) {
  return group <= 8 ? allow_smem<T, D, 1>() : allow_smem<T, D, 2>();
}

template <typename T>
cudaError_t allow_smem(int head_dim, int group) {
  if (head_dim == 64) return allow_smem<T, 64>(group);
  return head_dim == 128 ? allow_smem<T, 128>(group) : allow_smem<T, 256>(group);
}

}  // namespace

int pages_attend_parts(int head_dim, int group, int sm_count) {
  const int at = head_dim == 64 ? 0 : head_dim == 128 ? 1 : 2;
  const int one[] = {ctas_per_sm<64, 1>(), ctas_per_sm<128, 1>(), ctas_per_sm<256, 1>()};
  const int two[] = {ctas_per_sm<64, 2>(), ctas_per_sm<128, 2>(), ctas_per_sm<256, 2>()};
  return 2 * std::min((group <= 8 ? one : two)[at] * sm_count, MAX_CTAS);
}

cudaError_t pages_attend_init_attributes(int dtype, int head_dim, int group) {
  return dtype == RTVLA_DTYPE_BF16 ? allow_smem<bf16>(head_dim, group) : allow_smem<__half>(head_dim, group);
}

cudaError_t launch_pages_attend(const PagedAttnParams &p, int dtype, int sm_count, cudaStream_t st) {
  return dtype == RTVLA_DTYPE_BF16 ? attend<bf16>(p, sm_count, st) : attend<__half>(p, sm_count, st);
}

}  // namespace rtvla
