// C ABI of the paged KV cache (rtvla_pages_*): argument checks, the context with its RoPE tables
// and workspaces, and the launches.
#include <cmath>
#include <cstdlib>
#include <new>
#include <vector>

#include "kernels.h"
#include "pages.h"
#include "rtvla.h"

using namespace rtvla;

struct rtvla_pages_ctx {
  rtvla_pages_config cfg;
  PageGeom g;
  int device = 0, sm_count = 148;
  unsigned char *arena = nullptr;  // one allocation holds every buffer
  size_t mem_cap = 0;
  bool checked = false;
  std::vector<GuardRegion> guards;
  GuardRegion *d_guards = nullptr;
  DevCtl *ctl = nullptr;
  float2 *rope_lo = nullptr, *rope_hi = nullptr;
  int *done = nullptr;  // plan: CTAs finished
  float *part_o = nullptr;
  float2 *part_ml = nullptr;
  unsigned long long *keys = nullptr;  // select: [max_batch][n_kv_heads][table_width]
};

namespace {

// Makes the context's device current for a call and restores the caller's.
struct OnDevice {
  int before = -1, want;
  bool ok;
  explicit OnDevice(int device) : want(device) {
    ok = cudaGetDevice(&before) == cudaSuccess && (before == want || cudaSetDevice(want) == cudaSuccess);
  }
  ~OnDevice() {
    if (ok && before != want) cudaSetDevice(before);
  }
};

// Hands out 256-byte aligned buffers of an arena (of a null one, to find its size).  In checked mode
// each lies between two guard bands, as the denoise context's buffers do.
struct Carve {
  rtvla_pages_ctx *c;
  unsigned char *base;
  size_t at = 0;
  template <typename T>
  void operator()(T *&p, size_t n) {
    const size_t bytes = (n * sizeof(T) + 255) & ~size_t(255);
    if (c->checked) {
      if (base) c->guards.push_back(GuardRegion{base + at, (unsigned long long)bytes});
      at += GUARD_BYTES;
    }
    if (base) p = reinterpret_cast<T *>(base + at);
    at += bytes + (c->checked ? GUARD_BYTES : 0);
  }
};

void p_free(rtvla_pages_ctx *c) {
  if (c->arena) cudaFree(c->arena);
  delete c;
}

rtvla_status check_cfg(const rtvla_pages_config *g) {
  if (g->n_layers < 1 || g->n_layers > 256 || g->n_q_heads < 1 || g->n_kv_heads < 1 || g->n_kv_heads > 64 ||
      g->page_size < 1 || g->n_pages < 1 || g->table_width < 1 || g->max_batch < 1 || g->max_batch > 4096 ||
      !(g->rope_theta >= 0.f) || !std::isfinite(g->rope_theta))
    return RTVLA_ERR_INVALID_ARG;
  if ((long long)g->n_pages * g->page_size >= (1ll << 31) || (long long)g->table_width * g->page_size > (1ll << 24))
    return RTVLA_ERR_INVALID_ARG;
  // a row of the cache (layer, page, head, token) is numbered in 32 bits; more would not fit a GPU
  if ((double)g->n_layers * g->n_pages * g->n_kv_heads * g->page_size >= 4294967295.0) return RTVLA_ERR_INVALID_ARG;
  if (g->n_q_heads % g->n_kv_heads) return RTVLA_ERR_INVALID_ARG;
  if (g->dtype != RTVLA_DTYPE_BF16 && g->dtype != RTVLA_DTYPE_F16) return RTVLA_ERR_UNSUPPORTED;
  if (g->head_dim != 64 && g->head_dim != 128 && g->head_dim != 256) return RTVLA_ERR_UNSUPPORTED;
  if (g->n_q_heads / g->n_kv_heads > 16) return RTVLA_ERR_UNSUPPORTED;
  if (g->page_size > 1024 || (g->page_size & (g->page_size - 1))) return RTVLA_ERR_UNSUPPORTED;
  return RTVLA_OK;
}

rtvla_status p_create(rtvla_pages_ctx *c) {
  const rtvla_pages_config &g = c->cfg;
  if (cudaGetDevice(&c->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess)
    return RTVLA_ERR_CUDA;
  const int group = g.n_q_heads / g.n_kv_heads;
  if (pages_init_attributes(g.dtype, g.head_dim) != cudaSuccess ||
      pages_attend_init_attributes(g.dtype, g.head_dim, group) != cudaSuccess)
    return RTVLA_ERR_CUDA;
  const bool rope = g.rope_theta > 0.f;
  const size_t half = g.head_dim / 2, hi = ((size_t)g.table_width * g.page_size + 255) / 256;
  const size_t parts = (size_t)pages_attend_parts(g.head_dim, group, c->sm_count) * group;
  auto layout = [&](unsigned char *base) {
    Carve take{c, base};
    take(c->ctl, 1);
    take(c->done, 1);
    take(c->part_o, parts * g.head_dim);
    take(c->part_ml, parts);
    if (rope) {
      take(c->rope_lo, 256 * half);
      take(c->rope_hi, hi * half);
    }
    if (g.has_select) take(c->keys, (size_t)g.max_batch * g.n_kv_heads * g.table_width);
    if (c->checked) take(c->d_guards, 16);  // one entry per buffer
    return take.at;
  };
  const size_t bytes = layout(nullptr);
  if (c->mem_cap && bytes > c->mem_cap) return RTVLA_ERR_OOM;
  if (cudaMalloc(&c->arena, bytes) != cudaSuccess) {
    c->arena = nullptr;
    return RTVLA_ERR_OOM;
  }
  layout(c->arena);
  if (c->checked) {
    for (const GuardRegion &r : c->guards)
      if (cudaMemset(r.base, GUARD_FILL, GUARD_BYTES) != cudaSuccess ||
          cudaMemset(r.base + GUARD_BYTES + r.bytes, GUARD_FILL, GUARD_BYTES) != cudaSuccess)
        return RTVLA_ERR_CUDA;
    if (cudaMemcpy(c->d_guards, c->guards.data(), c->guards.size() * sizeof(GuardRegion), cudaMemcpyHostToDevice) !=
        cudaSuccess)
      return RTVLA_ERR_CUDA;
  }
  if (cudaMemset(c->ctl, 0, sizeof(DevCtl)) != cudaSuccess || cudaMemset(c->done, 0, sizeof(int)) != cudaSuccess)
    return RTVLA_ERR_CUDA;
  if (rope && (launch_rope_table(c->rope_lo, 256, 1, g.head_dim, g.rope_theta, 0) != cudaSuccess ||
               launch_rope_table(c->rope_hi, (int)hi, 256, g.head_dim, g.rope_theta, 0) != cudaSuccess))
    return RTVLA_ERR_CUDA;
  return cudaDeviceSynchronize() == cudaSuccess ? RTVLA_OK : RTVLA_ERR_CUDA;
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// the parts of the cache a per-layer call reads
rtvla_status check_kv(const rtvla_pages_ctx *c, int layer, const rtvla_paged_kv *kv) {
  if (!c || !kv || !kv->k || !kv->v || !aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->k_mean, 16) ||
      layer < 0)
    return RTVLA_ERR_INVALID_ARG;
  return layer < c->cfg.n_layers ? RTVLA_OK : RTVLA_ERR_SHAPE;
}

rtvla_status check_requests(const rtvla_pages_ctx *c, const rtvla_paged_kv *kv) {
  if (!kv->table || !kv->lens || !aligned(kv->table, 4) || !aligned(kv->lens, 4) || kv->batch < 1)
    return RTVLA_ERR_INVALID_ARG;
  return kv->batch <= c->cfg.max_batch ? RTVLA_OK : RTVLA_ERR_SHAPE;
}

rtvla_status launched(cudaError_t e) {
  if (e == cudaSuccess) return RTVLA_OK;
  cudaGetLastError();
  return RTVLA_ERR_CUDA;
}

}  // namespace

namespace rtvla {
rtvla_status pages_check_prefix(const rtvla_pages_ctx *c, int device, int n_layers, int n_q_heads, int head_dim,
                                float rope_theta, const int32_t *slots, const int32_t *positions,
                                const rtvla_paged_kv *kv) {
  const rtvla_pages_config &g = c->cfg;
  if (c->device != device || g.dtype != RTVLA_DTYPE_BF16 || g.n_layers != n_layers || g.n_q_heads != n_q_heads ||
      g.n_kv_heads != 1 || g.head_dim != head_dim || g.rope_theta != rope_theta)
    return RTVLA_ERR_UNSUPPORTED;
  const rtvla_status s = check_kv(c, 0, kv);
  if (s != RTVLA_OK) return s;
  if (!aligned(slots, 4) || !aligned(positions, 4)) return RTVLA_ERR_INVALID_ARG;
  return check_requests(c, kv);
}
}  // namespace rtvla

// =======================================================================================
// C ABI

extern "C" {

rtvla_status rtvla_pages_create(const rtvla_pages_config *cfg, rtvla_pages_ctx **out) {
  if (!cfg || !out) return RTVLA_ERR_INVALID_ARG;
  *out = nullptr;
  rtvla_status st = check_cfg(cfg);
  if (st != RTVLA_OK) return st;
  rtvla_pages_ctx *c = new (std::nothrow) rtvla_pages_ctx();
  if (!c) return RTVLA_ERR_OOM;
  c->cfg = *cfg;
  c->g = PageGeom{0, cfg->n_pages, cfg->table_width, cfg->n_kv_heads, cfg->head_dim};
  while ((1 << c->g.shift) < cfg->page_size) ++c->g.shift;
  if (const char *env = std::getenv("RTVLA_CHECKED")) c->checked = std::atoi(env) != 0;
  if (const char *env = std::getenv("RTVLA_DEVICE_MEMORY_CAP")) c->mem_cap = (size_t)std::strtoull(env, nullptr, 10);
  try {
    st = p_create(c);
  } catch (const std::bad_alloc &) {
    st = RTVLA_ERR_OOM;
  }
  if (st != RTVLA_OK) {
    cudaGetLastError();
    p_free(c);
    return st;
  }
  *out = c;
  return RTVLA_OK;
}

rtvla_status rtvla_pages_plan(rtvla_pages_ctx *c, const int32_t *lens, const int32_t *delta, int32_t *free_pages,
                              const int32_t *n_free, const rtvla_paged_kv *kv, int32_t *n_free_out, int32_t *slots,
                              int32_t *positions, int32_t *row_start, int n_rows, void *stream) {
  if (!c || !lens || !delta || !free_pages || !n_free || !kv || !n_free_out || !row_start || n_rows < 0 ||
      (n_rows > 0 && (!slots || !positions)))
    return RTVLA_ERR_INVALID_ARG;
  const void *ints[] = {lens, delta, free_pages, n_free, n_free_out, slots, positions, row_start};
  for (const void *p : ints)
    if (!aligned(p, 4)) return RTVLA_ERR_INVALID_ARG;
  const rtvla_status s = check_requests(c, kv);
  if (s != RTVLA_OK) return s;
  if (n_rows > (1 << 24)) return RTVLA_ERR_SHAPE;
  OnDevice dev(c->device);
  if (!dev.ok) return RTVLA_ERR_CUDA;
  PlanParams p{c->g,     lens,       delta, free_pages, n_free,    kv->table, kv->lens,
               n_free_out, slots, positions, row_start, kv->batch, n_rows, c->done, c->ctl};
  return launched(launch_pages_plan(p, c->sm_count, static_cast<cudaStream_t>(stream)));
}

rtvla_status rtvla_pages_write(rtvla_pages_ctx *c, int layer, const void *qkv, int qkv_dtype, const int32_t *slots,
                               const int32_t *positions, int n_rows, const rtvla_paged_kv *kv, void *q_out,
                               void *stream) {
  const rtvla_status s = check_kv(c, layer, kv);
  if (s != RTVLA_OK) return s;
  if (n_rows < 0 || (qkv_dtype != c->cfg.dtype && qkv_dtype != RTVLA_DTYPE_F32)) return RTVLA_ERR_INVALID_ARG;
  if (n_rows > 0 && (!qkv || !slots || !positions || !q_out || !aligned(qkv, 16) || !aligned(q_out, 16) ||
                     !aligned(slots, 4) || !aligned(positions, 4)))
    return RTVLA_ERR_INVALID_ARG;
  if (n_rows > (1 << 24)) return RTVLA_ERR_SHAPE;
  OnDevice dev(c->device);
  if (!dev.ok) return RTVLA_ERR_CUDA;
  WriteParams p{c->g, layer, c->cfg.n_q_heads, n_rows, qkv,        slots,      positions,
                kv->k, kv->v, kv->k_mean,      q_out,  c->rope_lo, c->rope_hi, c->ctl};
  return launched(launch_pages_write(p, c->cfg.dtype, qkv_dtype, c->sm_count, static_cast<cudaStream_t>(stream)));
}

rtvla_status rtvla_pages_attend(rtvla_pages_ctx *c, int layer, const void *q, const rtvla_paged_kv *kv,
                                const int32_t *sel, int sel_width, void *out, void *stream) {
  rtvla_status s = check_kv(c, layer, kv);
  if (s == RTVLA_OK) s = check_requests(c, kv);
  if (s != RTVLA_OK) return s;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(sel, 4) || (sel && sel_width < 1))
    return RTVLA_ERR_INVALID_ARG;
  if (sel && sel_width > 65536) return RTVLA_ERR_SHAPE;
  OnDevice dev(c->device);
  if (!dev.ok) return RTVLA_ERR_CUDA;
  const float scale = (float)(1.4426950408889634 / std::sqrt((double)c->cfg.head_dim));
  PagedAttnParams p{c->g,     layer,    c->cfg.n_q_heads, kv->batch, q,     kv->k,     kv->v,      kv->table,
                    kv->lens, sel,      sel_width,        out,       scale, c->part_o, c->part_ml, c->ctl};
  return launched(launch_pages_attend(p, c->cfg.dtype, c->sm_count, static_cast<cudaStream_t>(stream)));
}

rtvla_status rtvla_pages_select(rtvla_pages_ctx *c, int layer, const void *q, const rtvla_paged_kv *kv, int budget,
                                int keep_first, int keep_last, int32_t *sel, void *stream) {
  rtvla_status s = check_kv(c, layer, kv);
  if (s == RTVLA_OK) s = check_requests(c, kv);
  if (s != RTVLA_OK) return s;
  if (!q || !kv->k_mean || !sel || !aligned(q, 16) || !aligned(sel, 4) || keep_first < 0 || keep_last < 1 ||
      (long long)keep_first + keep_last > budget)
    return RTVLA_ERR_INVALID_ARG;
  if (budget > 65536) return RTVLA_ERR_SHAPE;
  if (!c->cfg.has_select) return RTVLA_ERR_UNSUPPORTED;
  OnDevice dev(c->device);
  if (!dev.ok) return RTVLA_ERR_CUDA;
  SelectParams p{c->g,     layer,    c->cfg.n_q_heads, kv->batch, q,       kv->k_mean, kv->table,
                 kv->lens, budget, keep_first,       keep_last, sel, c->keys,    c->ctl};
  return launched(launch_pages_select(p, c->cfg.dtype, static_cast<cudaStream_t>(stream)));
}

rtvla_status rtvla_pages_sync_status(rtvla_pages_ctx *c, void *stream) {
  if (!c) return RTVLA_ERR_INVALID_ARG;
  OnDevice dev(c->device);
  if (!dev.ok) return RTVLA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c->checked && launch_check_guards(c->d_guards, (int)c->guards.size(), c->ctl, st) != cudaSuccess) {
    cudaGetLastError();
    return RTVLA_ERR_CUDA;
  }
  if (cudaStreamSynchronize(st) != cudaSuccess) {
    cudaGetLastError();
    return RTVLA_ERR_CUDA;
  }
  DevCtl h;
  if (cudaMemcpy(&h, c->ctl, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return RTVLA_ERR_CUDA;
  if (h.err == 0) return RTVLA_OK;
  const int zero[2] = {0, 0};
  if (cudaMemcpy(c->ctl, zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return RTVLA_ERR_CUDA;
  if (h.err & DEVERR_GUARD) return RTVLA_ERR_GUARD_OVERWRITE;
  if (h.err & DEVERR_BOUNDS) return RTVLA_ERR_DEVICE_BOUNDS;
  return RTVLA_ERR_NO_PAGES;
}

void rtvla_pages_destroy(rtvla_pages_ctx *c) {
  if (!c) return;
  OnDevice dev(c->device);
  cudaDeviceSynchronize();
  p_free(c);
}

}  // extern "C"
