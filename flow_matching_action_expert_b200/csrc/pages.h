// Host-side launchers of the paged KV cache's kernels (internal to librtvla.so).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "pages_index.h"
#include "rtvla.h"

namespace rtvla {

// sites of the device error word
enum : int { PG_AT_PLAN = 801, PG_AT_WRITE = 802, PG_AT_ATTEND = 803, PG_AT_SELECT = 804 };

struct PlanParams {
  PageGeom g;
  const int32_t *lens;
  const int32_t *delta;
  int32_t *free_pages;
  const int32_t *n_free;
  int32_t *table;
  int32_t *lens_out;
  int32_t *n_free_out;
  int32_t *slots;
  int32_t *positions;
  int32_t *row_start;
  int batch;
  int n_rows;
  int *done;  // workspace: CTAs finished, 0 between calls
  DevCtl *ctl;
};
cudaError_t pages_init_attributes(int dtype, int head_dim);
cudaError_t launch_rope_table(float2 *dst, int rows, int step, int head_dim, double theta, cudaStream_t st);
cudaError_t launch_pages_plan(const PlanParams &p, int sm_count, cudaStream_t st);

struct WriteParams {
  PageGeom g;
  int layer, n_q_heads, n_rows;
  const void *qkv;
  const int32_t *slots;
  const int32_t *positions;
  void *k, *v, *k_mean;  // k_mean may be null
  void *q_out;
  const float2 *rope_lo;  // [256][head_dim / 2] (cos, sin) of position 0..255; null: no rotation
  const float2 *rope_hi;  // [positions / 256][head_dim / 2] of position 256 i
  DevCtl *ctl;
};
// dtype: RTVLA_DTYPE_* of the cache and q_out; src_dtype: of the qkv rows
cudaError_t launch_pages_write(const WriteParams &p, int dtype, int src_dtype, int sm_count, cudaStream_t st);

struct PagedAttnParams {
  PageGeom g;
  int layer, n_q_heads, batch;
  const void *q;          // [batch][n_q_heads][head_dim]
  const void *k, *v;
  const int32_t *table;   // [batch][width]
  const int32_t *lens;    // [batch]
  const int32_t *sel;     // [batch][n_kv_heads][sel_width] logical pages, or null
  int sel_width;
  void *out;              // [batch][n_q_heads][head_dim]
  float scale_log2;       // log2(e) / sqrt(head_dim)
  float *part_o;          // workspace [parts][group][head_dim]: unnormalised parts of cut requests
  float2 *part_ml;        // workspace [parts][group]: their maximum (log2 units) and sum
  DevCtl *ctl;
};
int pages_attend_parts(int head_dim, int group, int sm_count);  // parts the workspace holds
cudaError_t pages_attend_init_attributes(int dtype, int head_dim, int group);
cudaError_t launch_pages_attend(const PagedAttnParams &p, int dtype, int sm_count, cudaStream_t st);

struct SelectParams {
  PageGeom g;
  int layer, n_q_heads, batch;
  const void *q;
  const void *k_mean;
  const int32_t *table;
  const int32_t *lens;
  int budget, keep_first, keep_last;
  int32_t *sel;           // [batch][n_kv_heads][budget]
  unsigned long long *keys;  // workspace [batch][n_kv_heads][width]
  DevCtl *ctl;
};
cudaError_t launch_pages_select(const SelectParams &p, int dtype, cudaStream_t st);

// Checks a call that uses a context as the prefix model's cache (defined beside the C ABI).
rtvla_status pages_check_prefix(const rtvla_pages_ctx *c, int device, int n_layers, int n_q_heads, int head_dim,
                                float rope_theta, const int32_t *slots, const int32_t *positions,
                                const rtvla_paged_kv *kv);

}  // namespace rtvla
