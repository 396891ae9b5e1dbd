// Paged key-value cache: block tables and slot maps from request lengths, the
// append of new tokens, and the attention of one new token per request.
//
// A pool holds pages of `page` tokens; page p, head i, token s, channel c of K
// (and of V) is element ((p * stride_rows) + i * page + s) * dh + c, so one
// head's rows of a page are contiguous. Rows of dh elements are numbered with
// 32 bits, elements with 64.
#pragma once

#include "dv_common.cuh"
#include "dv_paged_launch.h"

namespace dv {

enum : int { ST_CLAMPED = 1, ST_RANGE = 2, ST_REFUSED = 16 };  // DV_DEV_* bits the kernels below set

// Number of entries of the ascending prefix sums pre[0..n] that are <= x,
// minus one: the row whose range [pre[r], pre[r + 1]) holds x (rows of no
// extent are passed over). pre[0] = 0 <= x < pre[n].
__device__ __forceinline__ int row_of(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// ----------------------------------------------------------------------------
// Block tables. Request r holds ceil(len / page) pages and wants
// ceil(goal / page). Pages of shrunk requests go on the free stack in (row,
// column) order; then requests that grow take pages from its top in row
// order, the a-th page taken being stack[avail - 1 - a]. A request is granted
// when the running sums of pages and of tokens up to it are covered, so the
// decision is three prefix sums over the rows.
//
// One cluster does that: every CTA forms the prefix sums of all rows for itself
// (at most 4096 rows, 8 bytes each from L2; one scan of all three sums, a second
// only where a request is refused), so the only exchange is one cluster barrier
// between the pushes onto the stack and the takes from it. Many tokens' slots
// are written by a second kernel over all SMs (page_slots_kernel). Bound by
// latency: launch, scan, three dependent loads.
// ----------------------------------------------------------------------------
constexpr int PT_THREADS = 1024;

struct PageTablesArgs {
  const int32_t* want;
  const int32_t* lens;
  int32_t* lens_out;
  int32_t* table;
  int32_t* free_list;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* slots;
  int32_t* offsets;
  int32_t* granted;
  int* status;
  int R, W, page, n_pages, T;
};

struct PtSums {
  unsigned gone, need, add;  // pages given back, pages wanted, tokens added
};

// Exclusive prefix sums of three values over the block, and their totals
__device__ __forceinline__ PtSums pt_scan(PtSums v, PtSums (&sc)[33], PtSums& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  auto warp_scan = [&](PtSums x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned a = __shfl_up_sync(0xffffffffu, x.gone, o), b = __shfl_up_sync(0xffffffffu, x.need, o),
                     c = __shfl_up_sync(0xffffffffu, x.add, o);
      if (lane >= o) x.gone += a, x.need += b, x.add += c;
    }
    return x;
  };
  const PtSums in = warp_scan(v);
  if (lane == 31) sc[w] = in;
  __syncthreads();
  if (w == 0) {
    const PtSums x = sc[lane], y = warp_scan(x);
    sc[lane] = {y.gone - x.gone, y.need - x.need, y.add - x.add};
    if (lane == 31) sc[32] = y;
  }
  __syncthreads();
  total = sc[32];
  const PtSums b = sc[w];
  __syncthreads();
  return {b.gone + in.gone - v.gone, b.need + in.need - v.need, b.add + in.add - v.add};
}

__global__ void __launch_bounds__(PT_THREADS) page_tables_kernel(PageTablesArgs a) {
  extern __shared__ int sm[];
  __shared__ PtSums sc[33];
  static_assert(PT_THREADS == 1024, "a warp scans the warps' sums");
  const int R = a.R, tid = threadIdx.x;
  int* s_len = sm;               // current lengths
  int* s_free = s_len + R + 1;   // prefix of pages given back
  int* s_need = s_free + R + 1;  // prefix of pages taken
  int* s_tok = s_need + R + 1;   // prefix of tokens added
  griddep_wait();
  griddep_launch();  // (after the wait: the slots' kernel starts early)
  const int cap = a.W * a.page;
  int bad = 0;
  int fc = *a.free_count;
  if (fc < 0 || fc > a.n_pages) {
    fc = fc < 0 ? 0 : a.n_pages;
    bad |= ST_RANGE;
  }
  auto pages = [&](int n) { return (n + a.page - 1) / a.page; };
  // a row's wishes; whether its lengths are within its table
  auto wishes = [&](int len, int want, bool& fits) {
    PtSums v = {0u, 0u, 0u};
    fits = len >= 0 && len <= cap && want <= cap;
    if (fits && want >= 0) {
      if (want < len) v.gone = pages(len) - pages(want);
      else v.need = pages(want) - pages(len), v.add = want - len;
    }
    return v;
  };
  PtSums sum = {0u, 0u, 0u};
  bool all_fit = true;
  for (int r0 = 0; r0 < R; r0 += PT_THREADS) {
    const int r = r0 + tid;
    PtSums v = {0u, 0u, 0u}, tot;
    bool fits = true;
    if (r < R) {
      const int len = a.lens[r];
      s_len[r] = len;
      if (len < 0 || len > cap) bad |= ST_RANGE;
      v = wishes(len, a.want[r], fits);
    }
    all_fit &= fits;
    const PtSums ex = pt_scan(v, sc, tot);
    if (r < R) {
      s_free[r] = sum.gone + ex.gone;
      s_need[r] = sum.need + ex.need;
      s_tok[r] = sum.add + ex.add;
    }
    sum = {sum.gone + tot.gone, sum.need + tot.need, sum.add + tot.add};
  }
  const int F = (int)sum.gone;
  // (a free count that does not go with the lengths: the sum is above n_pages, and may pass 31 bits)
  const int avail = (int)min((unsigned)fc + (unsigned)F, (unsigned)a.n_pages);
  if (F > a.n_pages - fc) bad |= ST_RANGE;
  unsigned need_ok = sum.need, tok_ok = sum.add;
  if (__syncthreads_and(all_fit) && sum.need <= (unsigned)avail && sum.add <= (unsigned)a.T) {
    if (cluster_rank() == 0)
      for (int r = tid; r < R; r += PT_THREADS) a.granted[r] = 1;
  } else {  // some request is refused: the prefix sums again, of those granted
    need_ok = tok_ok = 0;
    for (int r0 = 0; r0 < R; r0 += PT_THREADS) {
      const int r = r0 + tid;
      PtSums v = {0u, 0u, 0u}, tot;
      bool ok = true;
      if (r < R) {
        v = wishes(s_len[r], a.want[r], ok);
        v.gone = 0;
        ok = ok && (v.need == 0 || s_need[r] + v.need <= (unsigned)avail) && (v.add == 0 || s_tok[r] + v.add <= (unsigned)a.T);
        if (!ok) {
          v.need = v.add = 0;
          bad |= ST_REFUSED;
        }
        if (cluster_rank() == 0) a.granted[r] = ok;
      }
      const PtSums ex = pt_scan(v, sc, tot);
      if (r < R) {
        s_need[r] = need_ok + ex.need;
        s_tok[r] = tok_ok + ex.add;
      }
      need_ok += tot.need;
      tok_ok += tot.add;
    }
  }
  if (tid == 0) {
    s_free[R] = F;
    s_need[R] = need_ok;
    s_tok[R] = tok_ok;
  }
  __syncthreads();
  const int gt = cluster_rank() * PT_THREADS + tid, GT = cluster_size() * PT_THREADS;
  // pushes
  for (int i = gt; i < F; i += GT) {
    const int r = row_of(s_free, R, i);
    const int oldp = (s_len[r] + a.page - 1) / a.page;
    const int newp = oldp - (s_free[r + 1] - s_free[r]);
    if (i < a.n_pages - fc) a.free_list[fc + i] = a.table[(size_t)r * a.W + newp + (i - s_free[r])];
  }
  cluster_barrier();  // every CTA has read lens and want; the pushes are visible
  for (int i = gt; i < (int)need_ok; i += GT) {
    const int r = row_of(s_need, R, i);
    const int oldp = (s_len[r] + a.page - 1) / a.page;
    a.table[(size_t)r * a.W + oldp + (i - s_need[r])] = __ldcg(a.free_list + avail - 1 - i);
  }
  for (int r = gt; r <= R; r += GT) {
    a.offsets[r] = s_tok[r];
    if (r == R) break;
    const int len = s_len[r], want = a.want[r];
    a.lens_out[r] = len >= 0 && len <= cap && want >= 0 && want < len ? want : len + (s_tok[r + 1] - s_tok[r]);
  }
  if (gt == 0) *a.free_count_out = avail - (int)need_ok;
  if (bad) raise_status(a.status, bad);
  if (!a.slots) return;  // (page_slots_kernel's)
  // slots: four consecutive tokens a thread; a token's page is one just taken
  // (from the stack, not from the table another CTA writes) or an old one
  const int Tq = (a.T + 3) >> 2;
  for (int i = gt; i < Tq; i += GT) {
    int s[4];
    int r = -1, end = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 4 * i + e;
      s[e] = -1;
      if (t >= (int)tok_ok) continue;
      if (t >= end) {
        r = row_of(s_tok, R, t);
        end = s_tok[r + 1];
      }
      const int pos = s_len[r] + (t - s_tok[r]);
      const int pi = pos / a.page, oldp = (s_len[r] + a.page - 1) / a.page;
      const int p = pi >= oldp ? __ldcg(a.free_list + avail - 1 - (s_need[r] + pi - oldp))
                               : __ldcg(a.table + (size_t)r * a.W + pi);
      s[e] = p * a.page + (pos - pi * a.page);
    }
    if (4 * i + 3 < a.T) {
      *reinterpret_cast<int4*>(a.slots + 4 * i) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
      for (int e = 0; e < 4; ++e)
        if (4 * i + e < a.T) a.slots[4 * i + e] = s[e];
    }
  }
}

// The slots of many tokens, from the block tables and lengths just written:
// four consecutive tokens a thread, their row found in the offsets.
constexpr int PS_THREADS = 256;

__global__ void __launch_bounds__(PS_THREADS)
    page_slots_kernel(const int32_t* __restrict__ lens_out, const int32_t* __restrict__ table, const int32_t* __restrict__ offsets,
                      int32_t* __restrict__ slots, int R, int W, int page, int T) {
  extern __shared__ int s_tok[];
  griddep_launch();
  griddep_wait();
  for (int r = threadIdx.x; r <= R; r += PS_THREADS) s_tok[r] = __ldcg(offsets + r);
  __syncthreads();
  const int tokens = s_tok[R];
  for (int i = blockIdx.x * PS_THREADS + threadIdx.x; i < (T + 3) >> 2; i += gridDim.x * PS_THREADS) {
    int s[4], r = -1, end = -1, old = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 4 * i + e;
      s[e] = -1;
      if (t >= tokens) continue;
      if (t >= end) {
        r = row_of(s_tok, R, t);
        end = s_tok[r + 1];
        old = __ldcg(lens_out + r) - end;  // the length after its last token, so a token's place is old + t
      }
      const int pos = old + t, pi = pos / page;
      s[e] = __ldcg(table + (size_t)r * W + pi) * page + (pos - pi * page);
    }
    if (4 * i + 3 < T) {
      *reinterpret_cast<int4*>(slots + 4 * i) = make_int4(s[0], s[1], s[2], s[3]);
    } else {
      for (int e = 0; e < 4; ++e)
        if (4 * i + e < T) slots[4 * i + e] = s[e];
    }
  }
}

// ----------------------------------------------------------------------------
// Append: k, v [T][h][dh] fp32 into slot slots[t] of the pools, rounded once to
// the cache's dtype. A copy: bound by reading 4 bytes and writing 2 or 4 an
// element. A thread moves eight channels of K and of V; 16384 tokens of 32 heads
// of 128 channels into bf16 pages take 137 us, 0.89 of the copy bandwidth. Two
// or four such pieces a thread were slower (155, 146 us), evict-first loads too
// (150 us), and loads past the L1 cache (169 us: a warp's two 16-byte loads of k
// share their sectors). The loads are coherent, since the kernel before may
// still be writing k and v when this one becomes resident; read-only ones took
// the same time.
// ----------------------------------------------------------------------------
constexpr int PA_THREADS = 256;

struct PagedAppendArgs {
  const float *k, *v;
  const int32_t* slots;
  void *K, *V;
  int* status;
  int chunks;  // T * h * dh / 8
  int h, dh8, page, stride_rows;
  int n_slots;       // n_pages * page
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

template <typename KT>
__device__ __forceinline__ void store8(KT* dst, const float4& x, const float4& y) {
  if constexpr (sizeof(KT) == 2) {
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(bf16_pair(x.x, x.y), bf16_pair(x.z, x.w), bf16_pair(y.x, y.y), bf16_pair(y.z, y.w));
  } else {
    reinterpret_cast<float4*>(dst)[0] = x;
    reinterpret_cast<float4*>(dst)[1] = y;
  }
}

template <typename KT>
__global__ void __launch_bounds__(PA_THREADS) paged_append_kernel(PagedAppendArgs a) {
  griddep_launch();
  griddep_wait();
  const int i = blockIdx.x * PA_THREADS + threadIdx.x;
  if (i >= a.chunks) return;
  const int per = a.h * a.dh8;
  const int t = i / per, rem = i - t * per;
  const int head = rem / a.dh8, c = rem - head * a.dh8;
  const int slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    raise_status(a.status, ST_RANGE);
    return;
  }
  const float4* ks = reinterpret_cast<const float4*>(a.k) + 2ll * i;
  const float4* vs = reinterpret_cast<const float4*>(a.v) + 2ll * i;
  const float4 k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
  const int p = slot / a.page;
  const long long row = (long long)p * a.stride_rows + head * a.page + (slot - p * a.page);
  store8<KT>(static_cast<KT*>(a.K) + (row * a.dh8 + c) * 8, k0, k1);
  store8<KT>(static_cast<KT*>(a.V) + (row * a.dh8 + c) * 8, v0, v1);
}

// One new token per request from staging rows already in the cache's dtype.
// Heads outside the set store zeros: a recycled page still holds another
// request's keys and values, which must not be attended to later.
struct PagedTokenArgs {
  const void *ks, *vs;  // [B][h][dh]
  const int32_t* slots;
  const int32_t *head_idx, *head_count;
  void *K, *V;
  float* out;  // [B][d] cleared, or nullptr
  int* status;
  int h, dh8, page, stride_rows, n_slots, kh_max, all, d;
};
constexpr int PTK_MAX_H = 1024;

template <typename KT>
__global__ void __launch_bounds__(PA_THREADS) paged_token_kernel(PagedTokenArgs a) {
  __shared__ unsigned char s_sel[PTK_MAX_H];
  griddep_launch();
  griddep_wait();
  const int b = blockIdx.y;
  const int slot = a.slots[b];
  int hc = *a.head_count;
  hc = hc < 0 ? 0 : hc > a.kh_max ? a.kh_max : hc;
  for (int i = threadIdx.x; i < a.h; i += PA_THREADS) s_sel[i] = a.all != 0;
  __syncthreads();
  for (int j = threadIdx.x; j < hc; j += PA_THREADS) {
    const int head = a.head_idx[j];
    if (head >= 0 && head < a.h) s_sel[head] = 1;
  }
  __syncthreads();
  if (a.out)
    for (int i = blockIdx.x * PA_THREADS + threadIdx.x; i < a.d; i += gridDim.x * PA_THREADS) a.out[(size_t)b * a.d + i] = 0.f;
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    if (threadIdx.x == 0) raise_status(a.status, ST_RANGE);
    return;
  }
  const int p = slot / a.page, off = slot - p * a.page;
  constexpr int V = sizeof(KT) == 2 ? 1 : 2;  // 16-byte vectors of eight channels
  const int per = a.h * a.dh8 * V;
  const uint4* ks = static_cast<const uint4*>(a.ks) + (size_t)b * per;
  const uint4* vs = static_cast<const uint4*>(a.vs) + (size_t)b * per;
  for (int i = blockIdx.x * PA_THREADS + threadIdx.x; i < per; i += gridDim.x * PA_THREADS) {
    const int head = i / (a.dh8 * V), c = i - head * a.dh8 * V;
    const bool on = s_sel[head];
    const uint4 z = make_uint4(0, 0, 0, 0);
    const uint4 k = on ? ks[i] : z, v = on ? vs[i] : z;
    const long long at = ((long long)p * a.stride_rows + head * a.page + off) * (a.dh8 * V) + c;
    static_cast<uint4*>(a.K)[at] = k;
    static_cast<uint4*>(a.V)[at] = v;
  }
}

// ----------------------------------------------------------------------------
// Attention of one new token per request over its pages:
//   out = sum_s p_s V_s / sum_s p_s,  p_s = exp(scale q . K_s),
// one pass over K and V with a running maximum and sum (base 2).
//
// Work: the keys of an item (request, key-value head, up to 16 query heads) are
// cut into units of 16 or 32 keys, all units form one line, and every warp
// takes an equal stretch of it, so ragged lengths, few requests and few heads
// balance alike. An item inside one stretch is finished there; what crosses
// warps is joined through shared memory, what crosses CTAs through partials in
// the workspace, by the last CTA of the item to arrive, in CTA order: results
// do not depend on timing.
//
// Arithmetic: mma.sync m16n8k16 (bf16 in, fp32 out) with the queries as rows,
// the keys (then V's channels) as columns. q and p are fp32: they enter as
// three bf16 terms whose sum is the fp32 value to 2^-25, in rows of one
// fragment where 16 rows have room for them, so of bf16 caches nothing is
// rounded; fp32 caches are split the same way and the products down to 2^-24
// are kept. The tensor core truncates its sums, so chains are kept to one unit
// and added in fp32 outside. The scores' fragment is the second product's
// operand as it stands. tcgen05 would need 128 rows of A for at most 16 queries.
//
// Data: K and V rows come by 16-byte asynchronous copies, whole rows side by
// side, into the warp's own two slots (pitch one piece over the row, so the
// fragments' 16-byte reads have no bank conflicts); K of the next unit is
// requested once the scores of this one are formed, its V once this one's is
// used, the next item's q with it. No barrier in the loop. Any page size and
// alignment of pages costs the same (55 us with pages of 16 and of 8).
// Measured on the way: fragments loaded from global memory directly 71 us
// (8 rows of 64 bytes a load hold the L1 path at 4.8 TB/s), row-wise bulk copies
// 4.3 TB/s in a copy test that ran 6.3 TB/s with these; 4 warps in two CTAs the
// same; three CTAs' worth of shorter stretches per SM slower (66 us).
//
// Bound by HBM for long contexts: 16 requests of 32 heads, 0 to 2176 keys,
// 55 us on the device (5.2 TB/s, 0.79 of the copy bandwidth); 64 requests of 64
// heads over 8, 0 to 8192 keys, 193 us (5.6 TB/s, 0.85); one of 131071 keys
// 98 us (0.84). About 8 us of each are launch, schedule, the first rows' latency
// and the joins; the last SM's loop ends 18 % after the median one's. One
// request of 65 keys: 6.5 us.
// ----------------------------------------------------------------------------
constexpr int PGA_JOIN = 16;  // CTAs' partials that one CTA adds, at most (of more, groups first)

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// 2^x; what underflows fp32's normal range is 0, nothing next to a weight of 1
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x, y as three bf16 pairs (x in the low half): x = h.x + m.x + l.x to 2^-25 |x|.
__device__ __forceinline__ void split3(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = bf16_pair(x, y);
  const float x1 = x - __uint_as_float(h << 16), y1 = y - __uint_as_float(h & 0xffff0000u);
  m = bf16_pair(x1, y1);
  l = bf16_pair(x1 - __uint_as_float(m << 16), y1 - __uint_as_float(m & 0xffff0000u));
}

__device__ __forceinline__ uint32_t word_of(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t to, const void* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest group have landed, the whole warp's
__device__ __forceinline__ void copies_wait_all_but_one() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  __syncwarp();
}

// A stretch's place: row b of `len` keys, item it within the row, unit t of nt.
struct PagedAt {
  int b, it, t, nt, len;
};

// Shape of a kernel for NB blocks of 64 channels and up to QR query heads of a
// key-value head: 1 (its bf16 terms in three rows of the 16), 8 (high terms
// above middle ones) or 16 (each term a fragment of its own): warps of a CTA,
// 16-key tiles in a unit, CTAs per SM, floats of a partial ([QR][DH] sums, then
// QR maxima and QR weight sums), and shared memory per warp: K and V rows of a
// unit, a partial, the next item's q.
template <typename KT, int NB, int QR_>
struct PagedShape {
  static constexpr int DH = 64 * NB;
  static constexpr int ROW = DH * sizeof(KT);  // bytes
  static constexpr int PITCH = ROW + 16;       // of rows in shared memory: 16-byte pieces of neighbours in other banks
  static constexpr int WARPS = ROW <= 512 ? 8 : 4;
  static constexpr int QR = QR_;
  static constexpr int MT = ROW <= 128 || (ROW <= 256 && QR <= 8) ? 2 : 1;
  static constexpr int UNIT = 16 * MT;
  static constexpr int CTAS = ROW == 128 && QR <= 8 ? 2 : 1;
  static constexpr int PARTF = (QR * (DH + 2) + 3) & ~3;
  static constexpr bool STAGE = QR == 1 || (QR == 8 && NB <= 2);  // the next item's q is copied ahead
  static constexpr int RAWF = STAGE ? QR * DH : 0;
  static constexpr int SLOT = UNIT * PITCH;
  static constexpr int WARP_BYTES = 2 * SLOT + 4 * (PARTF + RAWF);
  static_assert(2 * SLOT >= 4 * PARTF, "an item left open at the end of a stretch takes the place of K and V");
  static_assert(WARPS * WARP_BYTES + 4 * (PAGED_MAX_ROWS + 1) + 1024 <= 227 * 1024, "shared memory");
};

template <typename KT, int NB, int QR>
__global__ void __launch_bounds__(32 * PagedShape<KT, NB, QR>::WARPS, PagedShape<KT, NB, QR>::CTAS)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  using Shape = PagedShape<KT, NB, QR>;
  constexpr bool F32 = sizeof(KT) == 4, ONE = QR == 1, WIDE = QR == 16;
  constexpr int MT = Shape::MT, UNIT = Shape::UNIT, DH = Shape::DH, PARTF = Shape::PARTF;
  constexpr int WARPS = Shape::WARPS, THREADS = 32 * WARPS, ROW = Shape::ROW, PITCH = Shape::PITCH;
  constexpr int SPL = F32 ? 3 : 1;  // bf16 terms of a cache element
  constexpr int AF = ONE ? 1 : WIDE ? 3 : 2;  // A fragments that hold the terms of q, and of p
  constexpr int QH = WIDE ? 2 : 1;  // query rows of a lane: g, and g + 8
  constexpr int NK = 4 * NB;        // MMA steps over the channels
  constexpr int EN = F32 || NB * QR >= 32 ? 2 : 4;  // channel tiles whose products run side by side
  extern __shared__ __align__(16) char smem_raw[];
  __shared__ unsigned sc[WARPS + 1];
  // items that cross warps or CTAs: first unit (-1: none), unit behind the last, row, item. 0..7: left open by that
  // warp, which began it; 8: begun by an earlier CTA
  __shared__ int s_item[9][4];
  __shared__ int s_last[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  int* s_pre = reinterpret_cast<int*>(smem_raw + WARPS * Shape::WARP_BYTES);  // [B + 1]
  // per warp: K rows, V rows (at the end of the stretch an item left open), what it adds to an item begun before it, q
  char* mine = smem_raw + warp * Shape::WARP_BYTES;
  auto part_of = [&](int w) { return reinterpret_cast<float*>(smem_raw + w * Shape::WARP_BYTES + 2 * Shape::SLOT); };
  auto open_of = [&](int w) { return reinterpret_cast<float*>(smem_raw + w * Shape::WARP_BYTES); };
  if (tid < 9) s_item[tid][0] = -1;
  __syncthreads();
  // `early`: what this call reads before its q was written before the kernel that writes q began (that one lets this
  // start only after its own wait), so only q and the new tokens' rows are waited for, further down
  if (!a.early) griddep_wait();
  griddep_launch();

  // units of every row, and their prefix sums
  const int cap = a.W * a.page;
  int nh = a.rows;
  if (a.head_idx) {
    const int hc = *a.head_count;
    nh = hc < 0 ? 0 : min(hc, a.rows);
    if (hc != nh && blockIdx.x == 0 && tid == 0) raise_status(a.status, ST_CLAMPED);
  }
  const int HR = a.rows * a.G;  // query rows of a request
  int units = 0, same = 0;  // units of all rows; of each where they are equal
  // Up to 32 rows: every warp for itself, the same values, no barrier, and rows of one length are seen at once. More go by
  // the even share, whose items may cross CTAs: 33 rows of 65 keys of 32 heads 17.1 us, 32 rows 15.3 us; 55.4 and 53.8 us
  // with 520 keys, and no difference a row with 2048.
  if (a.B <= 32) {
    const int len = lane < a.B ? a.lens[lane] : 0;
    if (len > cap && blockIdx.x == 0 && warp == 0) raise_status(a.status, ST_CLAMPED);
    units = len > 0 ? (min(len, cap) + UNIT - 1) / UNIT : 0;
    same = __shfl_sync(0xffffffffu, units, 0);
    if (!__all_sync(0xffffffffu, lane >= a.B || units == same)) same = 0;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, units, x);
      if (lane >= x) units += y;
    }
    if (lane < a.B) s_pre[lane + 1] = units;
    if (lane == 0) s_pre[0] = 0;
    units = __shfl_sync(0xffffffffu, units, 31);
    __syncwarp();
  } else {
    for (int r0 = 0; r0 < a.B; r0 += THREADS) {
      const int r = r0 + tid;
      const int len = r < a.B ? a.lens[r] : 0;
      if (len > cap && blockIdx.x == 0) raise_status(a.status, ST_CLAMPED);
      unsigned tot;
      const unsigned ex = block_exclusive_scan<THREADS>(len > 0 ? (unsigned)((min(len, cap) + UNIT - 1) / UNIT) : 0u, sc, &tot);
      if (r < a.B) s_pre[r] = units + ex;
      units += tot;
    }
    if (tid == 0) s_pre[a.B] = units;
    __syncthreads();
  }
  const int IR = nh * a.NQ;     // items of a row
  const int U = units * IR;     // (below 2^31: checked on the host for the largest lengths)
  // CTA c takes the units from cta_first(c) on, its warps equal stretches of them. Rows of one length: each CTA has whole
  // items, or each item has whole CTAs, where that takes (nearly) as few units a warp; else CTAs share evenly.
  int CE = min((int)gridDim.x, (U + WARPS - 1) / WARPS);  // CTAs with work
  int group = U, ctas = CE;                               // `ctas` CTAs share each `group` units
  if (same > 0 && U > 0) {
    const int items = a.B * IR;
    if (same <= WARPS) {
      const int per = WARPS / same, need = (items + per - 1) / per;
      if (need <= (int)gridDim.x) group = per * same, ctas = 1, CE = need;
    } else {
      const int per = min((int)gridDim.x / max(items, 1), (same + WARPS - 1) / WARPS);
      const int even = (U + WARPS * CE - 1) / (WARPS * CE);
      if (per > 0 && (same + WARPS * per - 1) / (WARPS * per) * 16 <= even * 17) group = same, ctas = per, CE = items * per;
    }
  }
  // rows without keys: zeros (and minus infinity)
  auto empty_rows = [&]() {
    for (int r = blockIdx.x; r < a.B; r += gridDim.x) {
      if (s_pre[r + 1] > s_pre[r]) continue;
      for (int i = tid; i < nh * a.G * a.dh; i += THREADS) a.out[(size_t)r * HR * a.dh + i] = 0.f;
      if (a.lse)
        for (int i = tid; i < nh * a.G; i += THREADS) a.lse[(size_t)r * HR + i] = -INFINITY;
    }
  };
  if ((int)blockIdx.x >= CE) {
    if (a.early) griddep_wait();
    empty_rows();
    return;
  }
  const int each = group / ctas, extra = group - each * ctas;
  auto cta_first = [&](int c) {
    const int gr = c / ctas, p = c - gr * ctas;
    return min(U, gr * group + p * each + min(p, extra));
  };
  auto cta_of = [&](int u) {
    const int gr = u / group, r = u - gr * group, big = extra * (each + 1);
    return gr * ctas + (r < big ? r / (each + 1) : extra + (r - big) / each);  // (r >= big only if each > 0)
  };
  const int clo = cta_first(blockIdx.x), chi = cta_first(blockIdx.x + 1);
  auto warp_first = [&](int w) { return clo + w * ((chi - clo) / WARPS) + min(w, (chi - clo) % WARPS); };
  const int wlo = warp_first(warp), whi = warp_first(warp + 1);
  const int row_bytes = a.dh * (int)sizeof(KT);

  auto locate = [&](int u) {
    PagedAt p;
    p.b = row_of(s_pre, a.B, u / IR);
    p.nt = s_pre[p.b + 1] - s_pre[p.b];
    p.len = min(a.lens[p.b], cap);
    const int rem = u - s_pre[p.b] * IR;
    p.it = rem / p.nt;
    p.t = rem - p.it * p.nt;
    return p;
  };
  auto advance = [&](PagedAt& p) {  // (never past the last unit)
    if (++p.t < p.nt) return;
    p.t = 0;
    if (++p.it < IR) return;
    p.it = 0;
    do { ++p.b; } while ((p.nt = s_pre[p.b + 1] - s_pre[p.b]) == 0);
    p.len = min(a.lens[p.b], cap);
  };
  // The pool row of key `lane` of a unit (of 16: both halves of the warp alike), -1 where masked
  auto pool_row = [&](const PagedAt& p) {
    const int key = p.t * UNIT + (lane & (UNIT - 1));
    if (key >= p.len) return -1;
    const int j = a.NQ == 1 ? p.it : p.it / a.NQ;
    const int head = a.head_idx ? a.head_idx[j] : j;
    const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page;
    const int pg = a.table[(size_t)p.b * a.W + pi];
    if ((unsigned)pg >= (unsigned)a.n_pages || (unsigned)head >= (unsigned)a.h_kv) {
      raise_status(a.status, ST_RANGE);
      return -1;
    }
    return pg * a.stride_rows + head * a.page + (key - pi * a.page);
  };

  // A unit's rows of K or V on their way to the warp's slot, 16 bytes a lane, whole rows side by side. Where pages
  // hold whole 16-key tiles and rows have no padding, a tile's rows are consecutive: one pointer and constant
  // offsets. Masked rows and channels past dh become zeros.
  constexpr int CPR = ROW / 16 < 32 ? ROW / 16 : 32, RPI = 32 / CPR;  // lanes on a row, rows of one request
  const uint32_t slot_at = (uint32_t)__cvta_generic_to_shared(mine) + (lane / CPR) * PITCH + (lane % CPR) * 16;
  const bool tiled = a.dh == DH && (a.page & 15) == 0;
  auto request = [&](const void* pool, uint32_t slot, int row, unsigned in) {
    if (tiled && in == ~0u) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const char* p = static_cast<const char*>(pool) +
                        (long long)(__shfl_sync(0xffffffffu, row, 16 * mt) + lane / CPR) * ROW + (lane % CPR) * 16;
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i)
#pragma unroll
          for (int c = 0; c < ROW; c += CPR * 16)
            copy16(slot + (16 * mt + i * RPI) * PITCH + c, p + i * RPI * ROW + c);
      }
    } else {
#pragma unroll
      for (int i = 0; i < UNIT / RPI; ++i) {
        const int r = __shfl_sync(0xffffffffu, row, i * RPI + lane / CPR);
#pragma unroll
        for (int c = 0; c < ROW; c += CPR * 16) {
          const int at = (lane % CPR) * 16 + c;
          const bool on = r >= 0 && at < row_bytes;
          copy16_or_zero(slot + i * RPI * PITCH + c, static_cast<const char*>(pool) + (on ? (long long)r * row_bytes + at : 0), on);
        }
      }
    }
  };

  const uint32_t row0 = g == 0 ? ~0u : 0u, row1 = g == 1 ? ~0u : 0u;  // (masks: choices by row became branches)
  float o[NB][8][QH][2], m[QH], l[QH];  // (l: this lane's keys)
  uint32_t qa[NK][4], ql[ONE ? 1 : NK][2], qw[WIDE ? NK : 1][4];  // (WIDE: high in qa, middle in qw, low in ql and qx)
  uint32_t qx[WIDE ? NK : 1][2];
  float* raw_mine = part_of(warp) + PARTF;
  // q of an item on its way to shared memory
  auto stage_q = [&](const PagedAt& p) {
    if constexpr (Shape::STAGE) {
      const int j = p.it / a.NQ, z = p.it - j * a.NQ;
      const float* qr = a.q + (((size_t)p.b * a.rows + j) * a.G + z * QR) * a.dh;
      const int rows = min(QR, a.G - z * QR), d4 = a.dh >> 2;
      for (int r = 0; r < rows; ++r)
        for (int c = lane; c < d4; c += 32)
          copy16((uint32_t)__cvta_generic_to_shared(raw_mine + r * DH + 4 * c), qr + r * a.dh + 4 * c);
    }
  };
  // q of an item as A fragments: rows 0-7 its high terms, rows 8-15 the middle ones, and the low ones in rows 8-15 of
  // another; of one query row 0 is high, row 8 middle, row 1 low; of 16 queries each term has its fragment. An MMA step takes from lane t four channels that K's
  // fragments have there: half of the 16 bytes (bf16) or the 16 bytes (fp32) that it reads, pieces 2 t and 2 t + 1 of
  // every 128 bytes of the row.
  auto begin_item = [&](const PagedAt& p) {
    const int j = p.it / a.NQ, z = p.it - j * a.NQ;
#pragma unroll
    for (int h = 0; h < QH; ++h) {
      const int r = ONE ? 0 : g + 8 * h, n = z * QR + r;
      const float* qr = Shape::STAGE ? raw_mine + r * DH : a.q + (((size_t)p.b * a.rows + j) * a.G + n) * a.dh;
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        const int c = F32 ? 32 * (s >> 1) + 8 * t4 + 4 * (s & 1) : 64 * (s >> 2) + 16 * t4 + 4 * (s & 3);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n < a.G && c < a.dh) x = *reinterpret_cast<const float4*>(qr + c);
        uint2 hi, mm, ll;
        split3(x.x, x.y, hi.x, mm.x, ll.x);
        split3(x.z, x.w, hi.y, mm.y, ll.y);
        if constexpr (ONE) {
          qa[s][0] = (hi.x & row0) | (ll.x & row1);
          qa[s][1] = mm.x & row0;
          qa[s][2] = (hi.y & row0) | (ll.y & row1);
          qa[s][3] = mm.y & row0;
        } else if constexpr (WIDE) {
          qa[s][h] = hi.x;
          qa[s][2 + h] = hi.y;
          qw[s][h] = mm.x;
          qw[s][2 + h] = mm.y;
          (h ? qx : ql)[s][0] = ll.x;
          (h ? qx : ql)[s][1] = ll.y;
        } else {
          qa[s][0] = hi.x;
          qa[s][1] = mm.x;
          qa[s][2] = hi.y;
          qa[s][3] = mm.y;
          ql[s][0] = ll.x;
          ql[s][1] = ll.y;
        }
      }
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[nb][e][h][0] = o[nb][e][h][1] = 0.f;
    }
    __syncwarp();
  };
  // The warp's sums complete: l over the lanes of a query, one query's low terms (row 1) added to row 0
  auto finish = [&]() {
#pragma unroll
    for (int h = 0; h < QH; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if constexpr (ONE) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i) o[nb][e][0][i] += __shfl_xor_sync(0xffffffffu, o[nb][e][0][i], 4);
    }
  };
  // A lane's row h times f, `dh` channels, to d. Tile e of block nb holds channels 64 nb + 8 (2 t + i) + e (bf16) or
  // 64 nb + 32 (e / 4) + 4 (2 t + i) + e % 4 (fp32: a lane's 16 bytes of a V row are four channels).
  auto store_row = [&](int h, float* d, int dh, float f) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const int c = 64 * nb + (F32 ? 8 * e + 8 * t4 + 4 * i : 16 * t4 + 8 * i + e);
          if (c < dh)
            *reinterpret_cast<float4*>(d + c) =
                make_float4(o[nb][e][h][i] * f, o[nb][e + 1][h][i] * f, o[nb][e + 2][h][i] * f, o[nb][e + 3][h][i] * f);
        }
  };
  auto put_part = [&](float* d) {
    if (ONE && g > 0) return;
#pragma unroll
    for (int h = 0; h < QH; ++h) {
      const int n = ONE ? 0 : g + 8 * h;
      if (t4 == 0) {
        d[QR * DH + n] = m[h];
        d[QR * DH + QR + n] = l[h];
      }
      store_row(h, d + n * DH, DH, 1.f);
    }
  };
  const auto inverse = [](float sum) { return sum > 0.f || sum != sum ? 1.f / sum : 0.f; };  // (NaN stays)
  const auto log_sum = [](float top, float sum) { return sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f; };
  auto output = [&](const PagedAt& p) {
    const int j = p.it / a.NQ, z = p.it - j * a.NQ;
#pragma unroll
    for (int h = 0; h < QH; ++h) {
      const int n = z * QR + (ONE ? 0 : g + 8 * h);
      if (ONE ? g > 0 : n >= a.G) continue;
      const size_t row = ((size_t)p.b * a.rows + j) * a.G + n;
      store_row(h, a.out + row * a.dh, a.dh, inverse(l[h]));
      if (a.lse && t4 == 0) a.lse[row] = log_sum(m[h], l[h]);
    }
  };
  // n partials, the first at p0 and the others from p1 on, `step` floats apart, added in that order by all warps (one
  // query: by this warp): into a partial `dst`, or divided into the outputs of item (b, it). Eight at a time, so that their loads overlap.
  auto combine = [&](const float* p0, const float* p1, int step, int n, int b, int it, float* dst) {
    const int j = it / a.NQ, z = it - j * a.NQ;
    const int gq = min(QR, a.G - z * QR);
    const size_t row = ((size_t)b * a.rows + j) * a.G + z * QR;
#pragma unroll 1
    for (int x = ONE ? lane : tid; x < gq * (DH / 4); x += ONE ? 32 : THREADS) {
      const int qn = x / (DH / 4), c = (x % (DH / 4)) * 4;
      float top = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int s0 = 0; s0 < n; s0 += 8) {
        float pm[8], pl[8];
        float4 pv[8];
        float mn = top;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int s = s0 + i;
          const float* p = s == 0 ? p0 : p1 + (size_t)(s - 1) * step;
          pm[i] = -INFINITY;
          pl[i] = 0.f;
          pv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (s < n) {
            pm[i] = p[QR * DH + qn];
            pl[i] = p[QR * DH + QR + qn];
            pv[i] = *reinterpret_cast<const float4*>(p + qn * DH + c);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mn = fmaxf(mn, pm[i]);
        const float mu = mn == -INFINITY ? 0.f : mn;
        float f = exp2_ftz(top - mu);
        sum *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
        top = mn;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f = exp2_ftz(pm[i] - mu);
          sum = fmaf(f, pl[i], sum);
          acc.x = fmaf(f, pv[i].x, acc.x);
          acc.y = fmaf(f, pv[i].y, acc.y);
          acc.z = fmaf(f, pv[i].z, acc.z);
          acc.w = fmaf(f, pv[i].w, acc.w);
        }
      }
      if (dst) {
        *reinterpret_cast<float4*>(dst + qn * DH + c) = acc;
        if (c == 0) {
          dst[QR * DH + qn] = top;
          dst[QR * DH + QR + qn] = sum;
        }
      } else {
        const float f = inverse(sum);
        if (c < a.dh)
          *reinterpret_cast<float4*>(a.out + (row + qn) * a.dh + c) = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
        if (a.lse && c == 0) a.lse[row + qn] = log_sum(top, sum);
      }
    }
  };

  if (wlo >= whi && a.early) griddep_wait();
  if (wlo < whi) {
    PagedAt cur = locate(wlo);
    if (warp == 0 && lane == 0 && cur.t > 0) {
      s_item[8][0] = wlo - cur.t;
      s_item[8][1] = wlo - cur.t + cur.nt;
      s_item[8][2] = cur.b;
      s_item[8][3] = cur.it;
    }
    PagedAt nxt = cur;
    const int count = whi - wlo;
    int row = pool_row(cur);
    unsigned in = __ballot_sync(0xffffffffu, row >= 0);
    if (a.early) griddep_wait();
    stage_q(cur);
    request(a.K, slot_at, row, in);
    copies_commit();
    request(a.V, slot_at + Shape::SLOT, row, in);
    copies_commit();
    if (count > 1) {
      advance(nxt);
      row = pool_row(nxt);
    }
    bool started = cur.t == 0, fresh = true;
#pragma unroll 1
    for (int n = 0; n < count; ++n) {
      const bool more = n + 1 < count;
      copies_wait_all_but_one();  // this unit's K, and q
      if (fresh) begin_item(cur);
      if (more && nxt.t == 0) stage_q(nxt);  // (lands with the next unit's K)
      // scores of UNIT keys by QR queries
      float s[QH][2 * MT][2];  // scores, then weights, of keys 8 j + 2 t and + 1
      {
        // two sums where few would leave the tensor cores waiting for one another
        constexpr int CN = !ONE && MT == 1 ? 2 : 1;
        float c[CN][2 * MT][4];
#pragma unroll
        for (int k = 0; k < NK; k += F32 ? 1 : 2) {
          // 16 bytes of a K row: eight channels (two steps), fp32 four (one)
          uint32_t b0[2 * MT][F32 ? SPL : 2], b1[2 * MT][F32 ? SPL : 2];
#pragma unroll
          for (int j = 0; j < 2 * MT; ++j) {
            const int piece = F32 ? k : k >> 1;
            const uint4 x = *reinterpret_cast<const uint4*>(mine + (8 * j + g) * PITCH + (piece >> 1) * 128 + t4 * 32 + (piece & 1) * 16);
            if constexpr (!F32) {
              b0[j][0] = x.x;
              b1[j][0] = x.y;
              b0[j][1] = x.z;
              b1[j][1] = x.w;
            } else {
              split3(__uint_as_float(x.x), __uint_as_float(x.y), b0[j][0], b0[j][1], b0[j][2]);
              split3(__uint_as_float(x.z), __uint_as_float(x.w), b1[j][0], b1[j][1], b1[j][2]);
            }
          }
#pragma unroll
          for (int h = 0; h < (F32 ? 1 : 2); ++h) {
            // products from the smallest on, those of one score apart
#pragma unroll
            for (int t = SPL - 1; t >= 0; --t) {
#pragma unroll
              for (int j = 0; j < 2 * MT; ++j) {
                if (k + h == 0 && t == SPL - 1) mma_bf16_first(c[0][j], qa[k + h], b0[j][F32 ? t : h], b1[j][F32 ? t : h]);
                else mma_bf16(c[0][j], qa[k + h], b0[j][F32 ? t : h], b1[j][F32 ? t : h]);
              }
              if constexpr (WIDE) {
                if (t < 2) {
#pragma unroll
                  for (int j = 0; j < 2 * MT; ++j) {
                    if (CN > 1 && k + h == 0 && t == (SPL > 1 ? 1 : 0)) mma_bf16_first(c[CN - 1][j], qw[k + h], b0[j][F32 ? t : h], b1[j][F32 ? t : h]);
                    else mma_bf16(c[CN - 1][j], qw[k + h], b0[j][F32 ? t : h], b1[j][F32 ? t : h]);
                  }
                }
              }
            }
            if constexpr (!ONE) {
              const uint32_t low[4] = {WIDE ? ql[k + h][0] : 0u, WIDE ? qx[WIDE ? k + h : 0][0] : ql[k + h][0],
                                       WIDE ? ql[k + h][1] : 0u, WIDE ? qx[WIDE ? k + h : 0][1] : ql[k + h][1]};
#pragma unroll
              for (int j = 0; j < 2 * MT; ++j) {
                if (CN > 1 && !WIDE && k + h == 0) mma_bf16_first(c[CN - 1][j], low, b0[j][F32 ? 0 : h], b1[j][F32 ? 0 : h]);
                else mma_bf16(c[CN - 1][j], low, b0[j][F32 ? 0 : h], b1[j][F32 ? 0 : h]);
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v[2] = {c[0][j][i], c[0][j][2 + i]};
            if constexpr (CN > 1) {
              v[0] += c[1][j][i];
              v[1] += c[1][j][2 + i];
            }
            if constexpr (!WIDE) v[0] += v[1];
            if constexpr (ONE) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 4);  // row 1's: rows 0 and 1 get the score
#pragma unroll
            for (int h = 0; h < QH; ++h) s[h][j][i] = v[h] * a.scale_log2;
          }
        if (in != ~0u) {
#pragma unroll
          for (int h = 0; h < QH; ++h)
#pragma unroll
            for (int j = 0; j < 2 * MT; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (!((in >> (8 * j + 2 * t4 + i)) & 1)) s[h][j][i] = -INFINITY;
        }
      }
      __syncwarp();  // K's slot is free
      if (more) {
        in = __ballot_sync(0xffffffffu, row >= 0);
        request(a.K, slot_at, row, in);
      }
      copies_commit();
      // running maximum and sum; p in bf16 terms: the scores' places are the A fragments' of the second product
      uint32_t pf[MT][AF][4];
      float corr[QH];
#pragma unroll
      for (int h = 0; h < QH; ++h) {
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j) mx = fmaxf(mx, fmaxf(s[h][j][0], s[h][j][1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[h], mx), mu = mn == -INFINITY ? 0.f : mn;
        corr[h] = exp2_ftz(m[h] - mu);
        m[h] = mn;
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j) {
          const float x = exp2_ftz(s[h][j][0] - mu), y = exp2_ftz(s[h][j][1] - mu);
          sum += x + y;
          uint32_t hi, mm, ll;
          split3(x, y, hi, mm, ll);
          uint32_t(&f)[AF][4] = pf[j >> 1];
          const int at = (j & 1) * 2;
          if constexpr (ONE) {
            f[0][at] = (hi & row0) | (ll & row1);
            f[0][at + 1] = mm & row0;
          } else if constexpr (WIDE) {
            f[0][at + h] = hi;
            f[AF - 2][at + h] = mm;
            f[AF - 1][at + h] = ll;
          } else {
            f[0][at] = hi;
            f[0][at + 1] = mm;
            f[AF - 1][at] = 0u;
            f[AF - 1][at + 1] = ll;
          }
        }
        l[h] = l[h] * corr[h] + sum;
      }
      copies_wait_all_but_one();  // this unit's V
      // o = o corr + p V
      const char* vp = mine + Shape::SLOT + 2 * t4 * PITCH + 16 * g;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int hv = 0; hv < (F32 ? 2 : 1); ++hv) {  // 16 bytes of V rows 2 t, + 1, + 8, + 9: eight channels, fp32 four
          uint4 v[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[mt][i] = *reinterpret_cast<const uint4*>(vp + (16 * mt + (i & 1) + (i >> 1) * 8) * PITCH + 128 * (F32 ? 2 * nb + hv : nb));
#pragma unroll
          for (int e0 = 0; e0 < (F32 ? 4 : 8); e0 += EN) {
            float c[EN][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t b0[EN][SPL], b1[EN][SPL];
#pragma unroll
              for (int i = 0; i < EN; ++i) {
                const int e = e0 + i;
                if constexpr (!F32) {
                  const uint32_t sel = (e & 1) ? 0x7632u : 0x5410u;
                  b0[i][0] = __byte_perm(word_of(v[mt][0], e >> 1), word_of(v[mt][1], e >> 1), sel);
                  b1[i][0] = __byte_perm(word_of(v[mt][2], e >> 1), word_of(v[mt][3], e >> 1), sel);
                } else {
                  split3(__uint_as_float(word_of(v[mt][0], e)), __uint_as_float(word_of(v[mt][1], e)), b0[i][0], b0[i][1], b0[i][2]);
                  split3(__uint_as_float(word_of(v[mt][2], e)), __uint_as_float(word_of(v[mt][3], e)), b1[i][0], b1[i][1], b1[i][2]);
                }
              }
              const uint32_t(&f)[AF][4] = pf[mt];
#pragma unroll
              for (int t = SPL - 1; t >= 0; --t) {
#pragma unroll
                for (int i = 0; i < EN; ++i) {
                  if (mt == 0 && t == SPL - 1) mma_bf16_first(c[i], f[0], b0[i][t], b1[i][t]);
                  else mma_bf16(c[i], f[0], b0[i][t], b1[i][t]);
                }
                if constexpr (WIDE) {
                  if (t < 2) {
#pragma unroll
                    for (int i = 0; i < EN; ++i) mma_bf16(c[i], f[AF - 2], b0[i][t], b1[i][t]);
                  }
                }
              }
              if constexpr (!ONE) {
#pragma unroll
                for (int i = 0; i < EN; ++i) mma_bf16(c[i], f[AF - 1], b0[i][0], b1[i][0]);
              }
            }
#pragma unroll
            for (int i = 0; i < EN; ++i) {
              float(&d)[QH][2] = o[nb][4 * hv + e0 + i];
              if constexpr (WIDE) {
                d[0][0] = fmaf(d[0][0], corr[0], c[i][0]);
                d[0][1] = fmaf(d[0][1], corr[0], c[i][1]);
                d[QH - 1][0] = fmaf(d[QH - 1][0], corr[QH - 1], c[i][2]);
                d[QH - 1][1] = fmaf(d[QH - 1][1], corr[QH - 1], c[i][3]);
              } else {
                d[0][0] = fmaf(d[0][0], corr[0], c[i][0] + c[i][2]);
                d[0][1] = fmaf(d[0][1], corr[0], c[i][1] + c[i][3]);
              }
            }
          }
        }
      }
      __syncwarp();  // V's slot is free
      if (more) request(a.V, slot_at + Shape::SLOT, row, in);
      copies_commit();
      const bool ends = cur.t + 1 == cur.nt;
      if (ends || !more) {
        finish();
        if (started && ends) {
          output(cur);
        } else if (!started) {
          put_part(part_of(warp));
        } else {
          put_part(open_of(warp));
          if (lane == 0) {
            s_item[warp][0] = whi - 1 - cur.t;
            s_item[warp][1] = whi - 1 - cur.t + cur.nt;
            s_item[warp][2] = cur.b;
            s_item[warp][3] = cur.it;
          }
        }
      }
      if (more) {
        cur = nxt;
        if (n + 2 < count) {
          advance(nxt);
          row = pool_row(nxt);
        }
        if (ends) started = true;
        fresh = ends;
      }
    }
  }
  empty_rows();
  __syncthreads();

  // What crosses warps: item by item, its partials in the order of their warps; by all warps, items of one query by a
  // warp each. What crosses CTAs too goes to the workspace, and the last CTA to arrive adds the CTAs' partials in order.
  auto sync = [&]() {
    if constexpr (ONE) __syncwarp();
    else __syncthreads();
  };
  const bool first = ONE ? lane == 0 : tid == 0;
#pragma unroll 1
  for (int i = ONE ? warp : 0; i < 9; i += ONE ? WARPS : 1) {
    const int begin = s_item[i][0], end = s_item[i][1], b = s_item[i][2], it = s_item[i][3];
    if (begin < 0) continue;
    const int w = i & 7;  // (item 8 starts with warp 0)
    const float *p0 = i < 8 ? open_of(w) : part_of(0), *p1 = part_of(w + 1);
    int n = 1, step = Shape::WARP_BYTES / 4;
    while (w + n < WARPS && warp_first(w + n) < min(end, chi)) ++n;
    const bool shared = i == 8 || end > chi;
    const int C = gridDim.x, mine = 2 * blockIdx.x + (i == 8 ? 0 : 1);
    auto slot = [&](int s) { return a.part + (size_t)s * PARTF; };
    float* dst = shared ? slot(mine) : nullptr;
    const int c0 = shared ? cta_of(begin) : 0, ctas_of = shared ? cta_of(end - 1) - c0 + 1 : 1;
    const bool two = ctas_of > PGA_JOIN;  // many CTAs: groups of PGA_JOIN join first, side by side
#pragma unroll 1
    for (int level = two ? 0 : 1; ; ++level) {
      combine(p0, p1, step, n, b, it, dst);
      if (!dst) break;
      // the partial's group (all of the item's; of many, PGA_JOIN neighbours) and its counter
      const int gr = two && level == 0 ? ((int)blockIdx.x - c0) / PGA_JOIN : 0;
      const int head = 2 * (c0 + gr * PGA_JOIN) + (gr == 0 ? 1 : 0);  // the slot of the group's first: begun in c0, or not
      n = !two ? ctas_of : level == 0 ? min(PGA_JOIN, ctas_of - gr * PGA_JOIN) : (ctas_of + PGA_JOIN - 1) / PGA_JOIN;
      __threadfence();
      sync();
      if (first) {
        unsigned* t = a.tick + (two && level == 1 ? 2 * C : 0) + head;
        const bool last = atomicAdd(t, 1u) == (unsigned)(n - 1);
        if (last) *t = 0;
        __threadfence();
        s_last[ONE ? warp : 0] = last;
      }
      sync();
      const bool last = s_last[ONE ? warp : 0];
      sync();
      if (!last) break;
      if (two && level == 1) {  // the groups' sums, kept behind the CTAs' slots
        p0 = slot(2 * C + head);
        p1 = slot(2 * C + 2 * (c0 + PGA_JOIN));
        step = 2 * PGA_JOIN * PARTF;
        dst = nullptr;
      } else {
        p0 = slot(head);
        p1 = slot((head & ~1) + 2);
        step = 2 * PARTF;
        dst = two ? slot(2 * C + head) : nullptr;
      }
    }
  }
}

}  // namespace dv
