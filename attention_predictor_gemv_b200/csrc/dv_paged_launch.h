// Host-side declarations of the paged key-value cache kernels (dv_paged.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dejavu.h"

namespace dv {

constexpr size_t WS_HEADER = 72 * 1024;    // every workspace's fixed header (status word, tickets)
constexpr size_t WS_TICKETS = 1024;        // offset of the attention counters in it
constexpr int PAGED_MAX_ROWS = 4096;       // requests of a call, at most
constexpr int PAGED_MAX_DH = 256;
constexpr int PAGED_UNITS_SPARE = 8192;    // more than the warps of a launch

struct PagedAttnArgs {
  const float* q;             // [B][rows][G][dh]
  const void *K, *V;          // pools
  const int32_t* table;       // [B][W]
  const int32_t* lens;        // [B]
  const int32_t* head_idx;    // nullptr: every key-value head
  const int32_t* head_count;
  float* out;                 // like q
  float* lse;                 // [B][rows][G] or nullptr
  float* part;                // partials: two slots per CTA, and as many for groups of CTAs
  unsigned* tick;             // a counter per slot, zero between calls
  int* status;
  int B, W, rows, G, h_kv, dh, page, page_shift, n_pages, stride_rows, NQ;
  float scale_log2;
  int early;                  // the kernel before on the stream is this call's paged_qkv_kernel
};

// Floats of partial slots the attention needs for heads of dh channels.
size_t paged_attn_part_floats(int dh);
// Whether the pool's sizes are within what the kernels index with; DV_OK or the error.
dv_status paged_kv_check(const dv_paged_kv* kv);
// Whether the attention's work on B requests of up to W pages can be numbered.
bool paged_units_ok(const dv_paged_kv* kv, int B, int W, int rows, int G);
cudaError_t run_paged_attn(const dv_paged_kv* kv, const float* q, int B, int rows, int G, const int32_t* table, int W,
                           const int32_t* lens, float scale, const int32_t* head_idx, const int32_t* head_count,
                           float* out, float* lse, float* part, unsigned* tick, int* status, cudaStream_t st, bool early = false);
// One new token per request: its k, v of every head from the staging rows
// ks, vs [B][h][dh] (the cache's dtype) into slots[b]; heads outside the set
// get zeros unless `all`. Also clears out [B][d] when it is given.
cudaError_t run_paged_token(const dv_paged_kv* kv, const void* ks, const void* vs, const int32_t* slots, int B,
                            const int32_t* head_idx, const int32_t* head_count, int kh_max, int all, float* out, int d,
                            int* status, cudaStream_t st);
// The projections on mma.sync with fp32 operands in three bf16 terms: bf16
// weights, at most 8 requests. q, k, v of the selected heads (k and v into
// their pages, `all`: of every head; else the other heads' places cleared), and
// W^O, which must follow the attention of this call's set on the stream.
bool paged_proj_ok(int B, int d, dv_dtype wdtype, int h, int dh, int kh_max, bool all);
cudaError_t run_paged_qkv(const dv_paged_kv* kv, const void* W, const float* bias, const float* y, int B, int d,
                          const int32_t* slots, const int32_t* head_idx, const int32_t* head_count, int kh_max, int all,
                          float* q, int* status, cudaStream_t st);
cudaError_t run_paged_wo(const void* W, const float* bias, const float* H, int B, int d, int h, int dh,
                         const int32_t* head_idx, const int32_t* head_count, int kh_max, float* out, int accumulate,
                         int* status, cudaStream_t st);

}  // namespace dv
