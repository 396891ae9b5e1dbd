// Paged key-value cache: argument checks, launches and C entry points.
// Declarations and argument contracts: include/dejavu.h.
#include <algorithm>

#include "dv_paged.cuh"
#include "dv_paged_proj.cuh"
#include "dv_launch.cuh"

namespace dv {
namespace {

using bf16 = __nv_bfloat16;

constexpr int PT_SLOTS_IN_ONE = 8192, PT_PAGES_IN_ONE = 16384;  // dv_page_tables: tokens, and table entries, for one CTA
constexpr int CTAS_PER_SM = 2;  // of the attention kernel, at most

bool dtype_ok(int t) { return t == DV_F32 || t == DV_BF16; }
int blocks64(int dh) { return dh <= 64 ? 1 : dh <= 128 ? 2 : 4; }

template <typename KT, int NB, int QR>
cudaError_t launch_attn(PagedAttnArgs a, cudaStream_t st) {
  using Shape = PagedShape<KT, NB, QR>;
  constexpr int per_sm = Shape::CTAS, UNIT = Shape::UNIT;
  static_assert((per_sm == 1 || (NB == 1 && per_sm == CTAS_PER_SM)) && Shape::PARTF <= 16 * (Shape::DH + 2), "partial slots");
  a.NQ = (a.G + Shape::QR - 1) / Shape::QR;
  const size_t smem = (size_t)Shape::WARPS * Shape::WARP_BYTES + 4ull * (a.B + 1);
  cudaError_t e = allow_smem(paged_attn_kernel<KT, NB, QR>, smem);
  if (e != cudaSuccess) return e;
  const long long cap = (long long)a.W * a.page;
  const long long most = a.B * ((cap + UNIT - 1) / UNIT) * (long long)a.rows * a.NQ;  // units, at most
  // a unit for each warp, and a CTA for each item where there are few
  const long long items = std::min((long long)a.B * a.rows * a.NQ, most);
  const long long want = std::max((most + Shape::WARPS - 1) / Shape::WARPS, items), have = (long long)sm_count() * per_sm;
  return launch_main(paged_attn_kernel<KT, NB, QR>, dim3((unsigned)(want < 1 ? 1 : want < have ? want : have)),
                     dim3(32 * Shape::WARPS), smem, st, a);
}

template <typename KT>
cudaError_t launch_attn_kt(const PagedAttnArgs& a, cudaStream_t st) {
  switch (blocks64(a.dh)) {
    case 1: return a.G == 1 ? launch_attn<KT, 1, 1>(a, st) : a.G > 8 ? launch_attn<KT, 1, 16>(a, st) : launch_attn<KT, 1, 8>(a, st);
    case 2: return a.G == 1 ? launch_attn<KT, 2, 1>(a, st) : a.G > 8 ? launch_attn<KT, 2, 16>(a, st) : launch_attn<KT, 2, 8>(a, st);
    default: return a.G == 1 ? launch_attn<KT, 4, 1>(a, st) : launch_attn<KT, 4, 8>(a, st);
  }
}

long long stride_rows(const dv_paged_kv* kv) {
  return kv->page_stride ? kv->page_stride / kv->dh : (long long)kv->h_kv * kv->page;
}

}  // namespace

size_t paged_attn_part_floats(int dh) {
  // two slots per CTA and as many for groups of CTAs; only 64 channels or fewer run two CTAs on an SM
  return (size_t)(dh <= 64 ? CTAS_PER_SM : 1) * sm_count() * 4 * 16 * (64 * blocks64(dh) + 2);
}

dv_status paged_kv_check(const dv_paged_kv* kv) {
  if (!kv || !kv->K || !kv->V || !dtype_ok(kv->kvdtype)) return DV_ERR_ARG;
  if (!aligned16(kv->K) || !aligned16(kv->V)) return DV_ERR_ALIGN;
  if (kv->n_pages < 1 || kv->page < 1 || kv->h_kv < 1 || kv->dh < 8 || kv->dh % 8 != 0 || kv->page_stride < 0)
    return DV_ERR_ARG;
  const long long need = (long long)kv->h_kv * kv->page * kv->dh;
  if (kv->page_stride && (kv->page_stride < need || kv->page_stride % kv->dh != 0)) return DV_ERR_ARG;
  // rows of dh elements and token slots are numbered with 32 bits
  if (kv->dh > PAGED_MAX_DH || stride_rows(kv) > INT32_MAX / kv->n_pages || kv->page > INT32_MAX / kv->n_pages)
    return DV_ERR_UNSUPPORTED;
  return DV_OK;
}

bool paged_units_ok(const dv_paged_kv* kv, int B, int W, int rows, int G) {
  // the units of all requests and heads are numbered with 31 bits, and rounded up to the warps of all CTAs
  return ((long long)W * kv->page + 16) / 16 * B * ((G + 7) / 8) <= (INT32_MAX - PAGED_UNITS_SPARE) / rows;
}

cudaError_t run_paged_attn(const dv_paged_kv* kv, const float* q, int B, int rows, int G, const int32_t* table, int W,
                           const int32_t* lens, float scale, const int32_t* head_idx, const int32_t* head_count,
                           float* out, float* lse, float* part, unsigned* tick, int* status, cudaStream_t st, bool early) {
  PagedAttnArgs a = {};
  a.early = early;
  a.q = q;
  a.K = kv->K;
  a.V = kv->V;
  a.table = table;
  a.lens = lens;
  a.head_idx = head_idx;
  a.head_count = head_count;
  a.out = out;
  a.lse = lse;
  a.part = part;
  a.tick = tick;
  a.status = status;
  a.B = B;
  a.W = W;
  a.rows = rows;
  a.G = G;
  a.h_kv = kv->h_kv;
  a.dh = kv->dh;
  a.page = kv->page;
  a.page_shift = (kv->page & (kv->page - 1)) == 0 ? __builtin_ctz((unsigned)kv->page) : -1;
  a.n_pages = kv->n_pages;
  a.stride_rows = (int)stride_rows(kv);
  a.scale_log2 = scale * 1.4426950408889634f;
  return kv->kvdtype == DV_BF16 ? launch_attn_kt<bf16>(a, st) : launch_attn_kt<float>(a, st);
}

cudaError_t run_paged_token(const dv_paged_kv* kv, const void* ks, const void* vs, const int32_t* slots, int B,
                            const int32_t* head_idx, const int32_t* head_count, int kh_max, int all, float* out, int d,
                            int* status, cudaStream_t st) {
  PagedTokenArgs a = {};
  a.ks = ks;
  a.vs = vs;
  a.slots = slots;
  a.head_idx = head_idx;
  a.head_count = head_count;
  a.K = kv->K;
  a.V = kv->V;
  a.out = out;
  a.status = status;
  a.h = kv->h_kv;
  a.dh8 = kv->dh / 8;
  a.page = kv->page;
  a.stride_rows = (int)stride_rows(kv);
  a.n_slots = kv->n_pages * kv->page;
  a.kh_max = kh_max;
  a.all = all;
  a.d = d;
  const int vecs = a.h * a.dh8 * (kv->kvdtype == DV_BF16 ? 1 : 2);
  const dim3 grid((unsigned)((vecs + PA_THREADS - 1) / PA_THREADS), (unsigned)B);
  return kv->kvdtype == DV_BF16 ? launch(paged_token_kernel<bf16>, grid, dim3(PA_THREADS), 0, st, a)
                                : launch(paged_token_kernel<float>, grid, dim3(PA_THREADS), 0, st, a);
}

bool paged_proj_ok(int B, int d, dv_dtype wdtype, int h, int dh, int kh_max, bool all) {
  // a CTA lists its share of the tiles in shared memory
  const long long per_cta = (qkv_most_tiles(kh_max, h, dh, all) + sm_count() - 1) / sm_count();
  return wdtype == DV_BF16 && B <= PP_MAX_B && d % 8 == 0 && dh % 32 == 0 && per_cta <= PQ_MAX_TILES;
}

cudaError_t run_paged_qkv(const dv_paged_kv* kv, const void* W, const float* bias, const float* y, int B, int d,
                          const int32_t* slots, const int32_t* head_idx, const int32_t* head_count, int kh_max, int all,
                          float* q, int* status, cudaStream_t st) {
  PagedQkvArgs a = {};
  a.W = static_cast<const bf16*>(W);
  a.bias = bias;
  a.y = y;
  a.head_idx = head_idx;
  a.head_count = head_count;
  a.slots = slots;
  a.q = q;
  a.K = static_cast<bf16*>(kv->K);
  a.V = static_cast<bf16*>(kv->V);
  a.status = status;
  a.B = B;
  a.d = d;
  a.h = kv->h_kv;
  a.dh = kv->dh;
  a.kh_max = kh_max;
  a.all = all;
  a.page = kv->page;
  a.stride_rows = (int)stride_rows(kv);
  a.n_slots = kv->n_pages * kv->page;
  const bool one = B == 1 && d <= PT_MAX_D;  // (faster at every width that it takes: see there)
  auto kern = one ? paged_qkv_one_kernel : paged_qkv_kernel;
  const size_t smem = one ? paged_qkv_one_smem() : paged_qkv_smem();
  cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_main(kern, dim3(sm_count()), dim3(PP_THREADS), smem, st, a);
}

namespace {

template <int QR, int NC>
cudaError_t launch_wo(const PagedWoArgs& a, cudaStream_t st) {
  using S = PagedWoShape<NC>;
  const size_t smem = (size_t)PP_WARPS * S::SLOTS * S::SLOT;
  cudaError_t e = allow_smem(paged_wo_kernel<QR, NC>, smem);
  if (e != cudaSuccess) return e;
  const int blocks = (a.d + S::CB - 1) / S::CB;
  return launch_main(paged_wo_kernel<QR, NC>, dim3(blocks < sm_count() ? blocks : sm_count()), dim3(PP_THREADS), smem, st, a);
}

// Columns per CTA: the fewest (32-byte sectors whole) that give no more CTAs than SMs
template <int QR>
cudaError_t launch_wo_qr(const PagedWoArgs& a, cudaStream_t st) {
  const int nc = ((a.d + sm_count() - 1) / sm_count() + 7) / 8;
  if (nc <= 2) return launch_wo<QR, 2>(a, st);
  if (nc <= 4) return launch_wo<QR, 4>(a, st);
  if (nc <= 6) return launch_wo<QR, 6>(a, st);
  if (nc <= 8) return launch_wo<QR, 8>(a, st);
  if (nc <= 10) return launch_wo<QR, 10>(a, st);
  return launch_wo<QR, 12>(a, st);
}

}  // namespace

cudaError_t run_paged_wo(const void* W, const float* bias, const float* H, int B, int d, int h, int dh,
                         const int32_t* head_idx, const int32_t* head_count, int kh_max, float* out, int accumulate,
                         int* status, cudaStream_t st) {
  PagedWoArgs a = {static_cast<const bf16*>(W), bias, H, head_idx, head_count, out, status, B, d, h, dh, kh_max, accumulate};
  return B == 1 ? launch_wo_qr<1>(a, st) : launch_wo_qr<8>(a, st);
}

}  // namespace dv

using namespace dv;

namespace {

dv_status ws_check(void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return DV_ERR_ARG;
  if (!aligned16(ws)) return DV_ERR_ALIGN;
  return ws_bytes < need ? DV_ERR_WORKSPACE : DV_OK;
}

dv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DV_OK : DV_ERR_CUDA; }

}  // namespace

extern "C" {

dv_status dv_page_tables(const int32_t* want, int R, int page, int n_pages, int W, const int32_t* lens,
                         int32_t* lens_out, int32_t* table, int32_t* free_list, const int32_t* free_count,
                         int32_t* free_count_out, int max_tokens, int32_t* slots, int32_t* offsets, int32_t* granted,
                         void* ws, size_t ws_bytes, dv_stream_t stream) {
  if (!want || !lens || !lens_out || !table || !free_list || !free_count || !free_count_out || !offsets || !granted)
    return DV_ERR_ARG;
  if (R < 1 || page < 1 || n_pages < 1 || W < 1 || max_tokens < 0 || (max_tokens > 0 && !slots)) return DV_ERR_ARG;
  for (const void* p : {(const void*)want, (const void*)lens, (const void*)lens_out, (const void*)table,
                        (const void*)free_list, (const void*)free_count, (const void*)free_count_out,
                        (const void*)slots, (const void*)offsets, (const void*)granted})
    if (!ok_opt(p)) return DV_ERR_ALIGN;
  // tokens, slots and pages of all requests are counted with 31 bits
  if (R > PAGED_MAX_ROWS || page > INT32_MAX / n_pages || page > INT32_MAX / 2 / R / W || max_tokens > INT32_MAX - 4)
    return DV_ERR_UNSUPPORTED;
  const dv_status s = ws_check(ws, ws_bytes, WS_HEADER);
  if (s != DV_OK) return s;
  PageTablesArgs a = {want, lens, lens_out, table, free_list, free_count, free_count_out, slots, offsets, granted,
                      static_cast<int*>(ws), R, W, page, n_pages, max_tokens};
  const size_t smem = 16ull * (R + 1);
  cudaError_t e = allow_smem(page_tables_kernel, smem);
  if (e != cudaSuccess) return DV_ERR_CUDA;
  // One CTA for little: eight are a barrier across SMs more. Many slots: a kernel over all SMs, against 20.4 us in one of
  // 124,000 tokens for 1024 requests.
  const bool many = max_tokens > PT_SLOTS_IN_ONE;
  const int cs = R > 1024 || many || (long long)R * W > PT_PAGES_IN_ONE ? 8 : 1;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (many) a.slots = nullptr;
  e = launch_cluster(page_tables_kernel, dim3(cs), dim3(PT_THREADS), smem, st, cs, a);
  if (e != cudaSuccess || !many) return cuda_status(e);
  const int grid = ((max_tokens + 3) / 4 + PS_THREADS - 1) / PS_THREADS;
  return cuda_status(launch(page_slots_kernel, dim3(grid < 2 * sm_count() ? grid : 2 * sm_count()), dim3(PS_THREADS), 4ull * (R + 1), st,
                            (const int32_t*)lens_out, (const int32_t*)table, (const int32_t*)offsets, slots, R, W, page, max_tokens));
}

dv_status dv_paged_append(const dv_paged_kv* kv, const float* k, const float* v, int T, const int32_t* slots, void* ws,
                          size_t ws_bytes, dv_stream_t stream) {
  dv_status s = paged_kv_check(kv);
  if (s != DV_OK) return s;
  if (T < 0 || !k || !v || !slots) return DV_ERR_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(slots)) return DV_ERR_ALIGN;
  s = ws_check(ws, ws_bytes, WS_HEADER);
  if (s != DV_OK) return s;
  if (T == 0) return DV_OK;
  PagedAppendArgs a = {};
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.K = kv->K;
  a.V = kv->V;
  a.status = static_cast<int*>(ws);
  a.h = kv->h_kv;
  a.dh8 = kv->dh / 8;
  const long long chunks = (long long)T * a.h * a.dh8;
  if (chunks > INT32_MAX - PA_THREADS) return DV_ERR_UNSUPPORTED;
  a.chunks = (int)chunks;
  a.page = kv->page;
  a.stride_rows = (int)stride_rows(kv);
  a.n_slots = kv->n_pages * kv->page;
  const int grid = (a.chunks + PA_THREADS - 1) / PA_THREADS;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(kv->kvdtype == DV_BF16
                         ? launch(paged_append_kernel<bf16>, dim3((unsigned)grid), dim3(PA_THREADS), 0, st, a)
                         : launch(paged_append_kernel<float>, dim3((unsigned)grid), dim3(PA_THREADS), 0, st, a));
}

dv_status dv_paged_attn(const dv_paged_kv* kv, const float* q, int B, int h_q, const int32_t* table, int W,
                        const int32_t* lens, float scale, const int32_t* head_idx, const int32_t* head_count,
                        int kh_max, float* out, float* lse, void* ws, size_t ws_bytes, dv_stream_t stream) {
  dv_status s = paged_kv_check(kv);
  if (s != DV_OK) return s;
  if (!q || !table || !lens || !out || B < 1 || W < 1 || h_q < 1 || h_q % kv->h_kv != 0) return DV_ERR_ARG;
  if ((head_idx != nullptr) != (head_count != nullptr)) return DV_ERR_ARG;
  if (head_idx && (kh_max < 0 || kh_max > kv->h_kv)) return DV_ERR_ARG;
  for (const void* p : {(const void*)q, (const void*)table, (const void*)lens, (const void*)head_idx,
                        (const void*)head_count, (const void*)out, (const void*)lse})
    if (!ok_opt(p)) return DV_ERR_ALIGN;
  if (B > PAGED_MAX_ROWS || kv->page > (INT32_MAX - 32) / W || h_q > INT32_MAX / kv->dh) return DV_ERR_UNSUPPORTED;
  const int rows = head_idx ? kh_max : kv->h_kv, G = h_q / kv->h_kv;
  if (!paged_units_ok(kv, B, W, rows > 0 ? rows : 1, G)) return DV_ERR_UNSUPPORTED;
  s = ws_check(ws, ws_bytes, WS_HEADER + 4 * paged_attn_part_floats(kv->dh));
  if (s != DV_OK) return s;
  if (head_idx && kh_max == 0) return DV_OK;
  char* w = static_cast<char*>(ws);
  return cuda_status(run_paged_attn(kv, q, B, rows, G, table, W, lens, scale,
                                    head_idx, head_count, out, lse, reinterpret_cast<float*>(w + WS_HEADER),
                                    reinterpret_cast<unsigned*>(w + WS_TICKETS), reinterpret_cast<int*>(w),
                                    reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
