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
// One cluster does a call: every CTA forms the prefix sums of all rows for
// itself (at most 4096 rows, 8 bytes each from L2), so the only exchange is one
// cluster barrier between the pushes onto the stack and the takes from it.
// Bound by latency: launch, the scans, three dependent loads.
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

__global__ void __launch_bounds__(PT_THREADS) page_tables_kernel(PageTablesArgs a) {
  extern __shared__ int sm[];
  __shared__ unsigned sc[PT_THREADS / 32 + 1];
  const int R = a.R, tid = threadIdx.x;
  int* s_len = sm;               // current lengths
  int* s_free = s_len + R + 1;   // prefix of pages given back
  int* s_need = s_free + R + 1;  // prefix of pages taken
  int* s_tok = s_need + R + 1;   // prefix of tokens added
  griddep_launch();
  griddep_wait();
  const int cap = a.W * a.page;
  int bad = 0;
  int fc = *a.free_count;
  if (fc < 0 || fc > a.n_pages) {
    fc = fc < 0 ? 0 : a.n_pages;
    bad |= ST_RANGE;
  }
  unsigned base = 0;
  for (int r0 = 0; r0 < R; r0 += PT_THREADS) {
    const int r = r0 + tid;
    unsigned gone = 0;
    if (r < R) {
      const int len = a.lens[r], want = a.want[r];
      s_len[r] = len;
      if (len < 0 || len > cap) bad |= ST_RANGE;
      else if (want >= 0 && want < len) gone = (len + a.page - 1) / a.page - (want + a.page - 1) / a.page;
    }
    unsigned tot;
    const unsigned ex = block_exclusive_scan<PT_THREADS>(gone, sc, &tot);
    if (r < R) s_free[r] = base + ex;
    base += tot;
  }
  if (tid == 0) s_free[R] = base;
  const int F = (int)base;
  const int avail = min(fc + F, a.n_pages);
  if (fc + F > a.n_pages) bad |= ST_RANGE;
  unsigned need_all = 0, tok_all = 0, need_ok = 0, tok_ok = 0;
  for (int r0 = 0; r0 < R; r0 += PT_THREADS) {
    const int r = r0 + tid;
    unsigned need = 0, add = 0;
    bool fits = true;
    if (r < R) {
      const int len = s_len[r], want = a.want[r];
      fits = len >= 0 && len <= cap && want <= cap;
      if (fits && want > len) {
        need = (want + a.page - 1) / a.page - (len + a.page - 1) / a.page;
        add = want - len;
      }
    }
    unsigned nt, tt, n2, t2;
    const unsigned ne = block_exclusive_scan<PT_THREADS>(need, sc, &nt);
    const unsigned te = block_exclusive_scan<PT_THREADS>(add, sc, &tt);
    const bool ok = fits && (need == 0 || need_all + ne + need <= (unsigned)avail) &&
                    (add == 0 || tok_all + te + add <= (unsigned)a.T);
    const unsigned ge = block_exclusive_scan<PT_THREADS>(ok ? need : 0u, sc, &n2);
    const unsigned he = block_exclusive_scan<PT_THREADS>(ok ? add : 0u, sc, &t2);
    if (r < R) {
      s_need[r] = need_ok + ge;
      s_tok[r] = tok_ok + he;
      if (!ok) bad |= ST_REFUSED;
      if (cluster_rank() == 0) a.granted[r] = ok;
    }
    need_all += nt;
    tok_all += tt;
    need_ok += n2;
    tok_ok += t2;
  }
  if (tid == 0) {
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
    if (fc + i < a.n_pages) a.free_list[fc + i] = a.table[(size_t)r * a.W + newp + (i - s_free[r])];
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
  if (gt == 0) *a.free_count_out = avail - (int)need_ok;
  if (bad) raise_status(a.status, bad);
}

// ----------------------------------------------------------------------------
// Append: k, v [T][h][dh] fp32 into slot slots[t] of the pools, rounded once to
// the cache's dtype. A copy: bound by reading 4 bytes and writing 2 or 4 an
// element. A thread moves eight channels of K and of V.
// ----------------------------------------------------------------------------
constexpr int PA_THREADS = 256;

struct PagedAppendArgs {
  const float *k, *v;
  const int32_t* slots;
  void *K, *V;
  int* status;
  long long chunks;  // T * h * dh / 8
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
  const long long i = (long long)blockIdx.x * PA_THREADS + threadIdx.x;
  if (i >= a.chunks) return;
  const int per = a.h * a.dh8;
  const int t = (int)(i / per), rem = (int)(i - (long long)t * per);
  const int head = rem / a.dh8, c = rem - head * a.dh8;
  const int slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    raise_status(a.status, ST_RANGE);
    return;
  }
  const float4* ks = reinterpret_cast<const float4*>(a.k) + 2 * i;
  const float4* vs = reinterpret_cast<const float4*>(a.v) + 2 * i;
  const float4 k0 = __ldcs(ks), k1 = __ldcs(ks + 1), v0 = __ldcs(vs), v1 = __ldcs(vs + 1);
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
// Work: the keys of a (request, head, group of 8 NT query heads) are cut into
// units of 16 keys, all units form one line, and every warp takes an equal
// stretch of it, so ragged lengths, few requests and few heads balance alike.
// A stretch's items that lie inside one warp are finished there; what crosses
// warps is joined through shared memory, what crosses CTAs through partials in
// the workspace, by the last CTA of the item to arrive, in CTA order.
//
// Arithmetic: the products run on mma.sync m16n8k16 (bf16 in, fp32 out) with
// the keys (then V's channels) as the 16 rows and 8 query heads as the columns.
// q and p are fp32: they enter as three bf16 terms whose sum is the fp32 value
// to 2^-25, so only K and V (bf16 by storage) are ever rounded; fp32 caches are
// split the same way and the six products down to 2^-24 are kept. The tensor
// core truncates its sums, so chains are kept short and added in fp32 outside.
// tcgen05 would need 128 rows of A for at most 16 queries and the operands in
// shared memory; the kernel is bound by HBM either way.
//
// K and V go straight from global memory into the fragments: a lane's 16-byte
// load of a K row is the k-slots (2t, 2t+1, 2t+8, 2t+9) of two MMAs, with the
// query's channels permuted alike, and V's channels are spread over the MMA's
// rows so that one byte permute pairs two keys. So there is no shared-memory
// staging and no barrier in the loop; the next unit's K is requested once the
// scores of this one are formed, its V once this one's is used.
// ----------------------------------------------------------------------------
constexpr int PGA_WARPS = 8;
constexpr int PGA_THREADS = PGA_WARPS * 32;

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// x, y as three bf16 pairs (x in the low half): x = h.x + m.x + l.x to 2^-25 |x|.
__device__ __forceinline__ void split3(float x, float y, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = bf16_pair(x, y);
  const float x1 = x - __uint_as_float(h << 16), y1 = y - __uint_as_float(h & 0xffff0000u);
  m = bf16_pair(x1, y1);
  l = bf16_pair(x1 - __uint_as_float(m << 16), y1 - __uint_as_float(m & 0xffff0000u));
}

// A stretch's place: row b, item it within the row, unit t of nt.
struct PagedAt {
  int b, it, t, nt;
};

// Eight channels of a cache row in registers.
template <typename KT>
struct Chunk {
  static constexpr int N = sizeof(KT) / 2;
  uint4 v[N];
  __device__ __forceinline__ void load(const KT* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = ld_stream(reinterpret_cast<const uint4*>(p) + i);
  }
  // zeros where the row is masked or the channels lie past dh
  __device__ __forceinline__ void load(const KT* pool, int row, int dh8, int c) {
    const uint4* p = reinterpret_cast<const uint4*>(pool) + ((long long)row * dh8 + c) * N;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row >= 0 && c < dh8 ? ld_stream(p + i) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int i) const {  // i-th 32-bit word
    const uint4& u = v[i >> 2];
    return (i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w;
  }
};

// Shape of a kernel for NB blocks of 64 channels and NT tiles of 8 query heads:
// 16-key tiles in a unit, CTAs per SM.
template <typename KT, int NB, int NT>
struct PagedShape {
  static constexpr int BYTES = sizeof(KT) * NB;  // a tile's K row bytes / 64
  static constexpr int MT = BYTES <= 4 && NT == 1 ? 2 : 1;
  static constexpr int CTAS = BYTES == 2 && NT == 1 ? 2 : 1;
  static constexpr int UNIT = 16 * MT;
};

template <typename KT, int NB, int NT>
__global__ void __launch_bounds__(PGA_THREADS, PagedShape<KT, NB, NT>::CTAS)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr bool F32 = sizeof(KT) == 4;
  constexpr int MT = PagedShape<KT, NB, NT>::MT, UNIT = 16 * MT;
  constexpr int DH = 64 * NB;                // channels, padded
  constexpr int SPL = F32 ? 3 : 1;           // bf16 terms of a cache element
  constexpr int NC = 2 * NB;                 // K chunks a lane holds per row
  constexpr int NK = 4 * NB;                 // MMA steps over the channels
  constexpr bool PRE = !(F32 && NB == 4);    // the next unit's rows fit in registers
  constexpr int PARTF = NT * (NB * 4 + 1) * 128;  // floats of a partial
  extern __shared__ __align__(16) char smem_raw[];
  __shared__ unsigned sc[PGA_WARPS + 1];
  __shared__ long long s_join[2][2];  // units [first, last] of the items this CTA shares with others; -1: none
  __shared__ int s_joinat[2][2];      // their row and item
  __shared__ int s_last;
  float* s_part = reinterpret_cast<float*>(smem_raw);                    // [warps][PARTF]
  uint2* s_q = reinterpret_cast<uint2*>(s_part + PGA_WARPS * PARTF);     // [warps][NT][NK][3][32]
  int* s_pre = reinterpret_cast<int*>(s_q + PGA_WARPS * NT * NK * 3 * 32);  // [B + 1]
  int* s_len = s_pre + a.B + 1;                                          // [B]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  griddep_launch();
  griddep_wait();

  // units of every row, and their prefix sums
  const int cap = a.W * a.page;
  int nh = a.rows;
  if (a.head_idx) {
    const int hc = *a.head_count;
    nh = hc < 0 ? 0 : min(hc, a.rows);
    if (hc != nh && blockIdx.x == 0 && tid == 0) raise_status(a.status, ST_CLAMPED);
  }
  unsigned base = 0;
  for (int r0 = 0; r0 < a.B; r0 += PGA_THREADS) {
    const int r = r0 + tid;
    int len = r < a.B ? a.lens[r] : 0;
    if (len > cap) {
      len = cap;
      if (blockIdx.x == 0) raise_status(a.status, ST_CLAMPED);
    }
    unsigned tot;
    const unsigned ex = block_exclusive_scan<PGA_THREADS>(len > 0 ? (unsigned)((len + UNIT - 1) / UNIT) : 0u, sc, &tot);
    if (r < a.B) {
      s_pre[r] = base + ex;
      s_len[r] = len;
    }
    base += tot;
  }
  if (tid == 0) s_pre[a.B] = base;
  if (tid < 2) s_join[tid][0] = -1;
  __syncthreads();
  const int IR = nh * a.NQ;  // items of a row
  const int HR = a.rows * a.G;  // query rows of a request
  // rows without keys: zeros (and minus infinity)
  for (int r = blockIdx.x; r < a.B; r += gridDim.x) {
    if (s_len[r] > 0) continue;
    for (int i = tid; i < nh * a.G * a.dh; i += PGA_THREADS) a.out[(size_t)r * HR * a.dh + i] = 0.f;
    if (a.lse)
      for (int i = tid; i < nh * a.G; i += PGA_THREADS) a.lse[(size_t)r * HR + i] = -INFINITY;
  }
  const long long U = (long long)base * IR;
  const int CE = (int)min((long long)gridDim.x, (U + PGA_WARPS - 1) / PGA_WARPS);  // CTAs with work
  if ((int)blockIdx.x >= CE) return;
  const int NW = CE * PGA_WARPS, wid = blockIdx.x * PGA_WARPS + warp;
  const long long wlo = U * wid / NW, whi = U * (wid + 1) / NW;
  const bool lead = wlo == U * ((long long)blockIdx.x * PGA_WARPS) / NW;  // the CTA's first units are this warp's
  const int dh8 = a.dh >> 3;
  const KT* Kp = static_cast<const KT*>(a.K);
  const KT* Vp = static_cast<const KT*>(a.V);

  auto locate = [&](long long u) {
    PagedAt p;
    p.b = row_of(s_pre, a.B, (int)(u / IR));
    p.nt = s_pre[p.b + 1] - s_pre[p.b];
    const long long rem = u - (long long)s_pre[p.b] * IR;
    p.it = (int)(rem / p.nt);
    p.t = (int)(rem - (long long)p.it * p.nt);
    return p;
  };
  auto advance = [&](PagedAt& p) {  // (never past the last unit)
    if (++p.t < p.nt) return;
    p.t = 0;
    if (++p.it < IR) return;
    p.it = 0;
    do { ++p.b; } while ((p.nt = s_pre[p.b + 1] - s_pre[p.b]) == 0);
  };
  // The pool row of key `lane` of a unit (of 16: both halves of the warp alike), -1 where masked
  auto pool_row = [&](const PagedAt& p) {
    const int key = p.t * UNIT + (lane & (UNIT - 1));
    if (key >= s_len[p.b]) return -1;
    const int j = p.it / a.NQ;
    const int head = a.head_idx ? a.head_idx[j] : j;
    const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page;
    const int pg = a.table[(size_t)p.b * a.W + pi];
    if ((unsigned)pg >= (unsigned)a.n_pages || (unsigned)head >= (unsigned)a.h_kv) {
      raise_status(a.status, ST_RANGE);
      return -1;
    }
    return pg * a.stride_rows + head * a.page + (key - pi * a.page);
  };

  float o[NT][NB][4][4], m[NT][2], l[NT][2];
  Chunk<KT> kc[2 * MT][NC], vc[NB][4 * MT];
  unsigned ok = 0;  // keys g + 8 i of the unit in kc that are not masked
  // Whole pages of 16-key tiles and channels without padding: a tile's rows are
  // consecutive, so a lane's loads are one pointer and constant offsets.
  const bool tiled = a.dh == DH && (a.page & 15) == 0;

  auto load_k = [&](int row) {
    if (tiled && __all_sync(0xffffffffu, row >= 0)) {
      ok = ~0u;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const KT* p = Kp + (long long)(__shfl_sync(0xffffffffu, row, 16 * mt) + g) * DH + 8 * t4;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          kc[2 * mt][i].load(p + 32 * i);
          kc[2 * mt + 1][i].load(p + 8 * DH + 32 * i);
        }
      }
    } else {
      ok = 0;
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j) {
        const int r = __shfl_sync(0xffffffffu, row, g + 8 * j);
        ok |= r >= 0 ? 1u << j : 0u;
#pragma unroll
        for (int i = 0; i < NC; ++i) kc[j][i].load(Kp, r, dh8, t4 + 4 * i);
      }
    }
  };
  auto load_v = [&](int row, int nb0, int nb1) {
    if (tiled && __all_sync(0xffffffffu, row >= 0)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const KT* p = Vp + (long long)(__shfl_sync(0xffffffffu, row, 16 * mt) + 2 * t4) * DH + 8 * g;
#pragma unroll
        for (int nb = nb0; nb < nb1; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) vc[nb][4 * mt + i].load(p + ((i & 1) + (i >> 1) * 8) * DH + 64 * nb);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4 * MT; ++j) {
        const int r = __shfl_sync(0xffffffffu, row, 2 * t4 + (j & 1) + (j >> 1) * 8);
#pragma unroll
        for (int nb = nb0; nb < nb1; ++nb) vc[nb][j].load(Vp, r, dh8, g + 8 * nb);
      }
    }
  };
  uint2* q_mine = s_q + warp * NT * NK * 3 * 32 + lane;

  // q of an item, split, in the lane's own places of shared memory
  auto begin_item = [&](const PagedAt& p) {
    const int j = p.it / a.NQ, z = p.it - j * a.NQ;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = (z * NT + nt) * 8 + g;
      const float* qr = a.q + (((size_t)p.b * a.rows + j) * a.G + n) * a.dh;
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        const int c = t4 + 4 * (s >> 1);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n < a.G && c < dh8) x = *reinterpret_cast<const float4*>(qr + 8 * c + 4 * (s & 1));
        uint2 h, mm, ll;
        split3(x.x, x.y, h.x, mm.x, ll.x);
        split3(x.z, x.w, h.y, mm.y, ll.y);
        uint2* d = q_mine + (nt * NK + s) * 3 * 32;
        d[0] = h;
        d[32] = mm;
        d[64] = ll;
      }
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][nb][e][i] = 0.f;
    }
  };
  // l summed over the lanes that share its queries
  auto total_l = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x);
  };
  // A partial: per lane its accumulators and (m, l), as 16-byte vectors
  auto put_part = [&](float4* d) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          d[((nt * NB + nb) * 4 + e) * 32 + lane] = make_float4(o[nt][nb][e][0], o[nt][nb][e][1], o[nt][nb][e][2], o[nt][nb][e][3]);
      d[(NT * NB * 4 + nt) * 32 + lane] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
    }
  };
  // `from`: how to read them (shared memory, or another CTA's through L2)
  auto add_part = [&](const float4* d, auto from) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 ml = from(d + (NT * NB * 4 + nt) * 32 + lane);
      const float m2[2] = {ml.x, ml.y}, l2[2] = {ml.z, ml.w};
      float c1[2], c2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mn = fmaxf(m[nt][i], m2[i]), mu = mn == -INFINITY ? 0.f : mn;
        c1[i] = exp2f(m[nt][i] - mu);
        c2[i] = exp2f(m2[i] - mu);
        l[nt][i] = l[nt][i] * c1[i] + l2[i] * c2[i];
        m[nt][i] = mn;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v = from(d + ((nt * NB + nb) * 4 + e) * 32 + lane);
          o[nt][nb][e][0] = o[nt][nb][e][0] * c1[0] + v.x * c2[0];
          o[nt][nb][e][1] = o[nt][nb][e][1] * c1[1] + v.y * c2[1];
          o[nt][nb][e][2] = o[nt][nb][e][2] * c1[0] + v.z * c2[0];
          o[nt][nb][e][3] = o[nt][nb][e][3] * c1[1] + v.w * c2[1];
        }
    }
  };
  const auto shared = [](const float4* p) { return *p; };
  const auto global = [](const float4* p) { return __ldcg(p); };
  auto output = [&](int b, int it) {
    const int j = it / a.NQ, z = it - j * a.NQ;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = (z * NT + nt) * 8 + 2 * t4 + i;
        if (n >= a.G) continue;
        const size_t row = ((size_t)b * a.rows + j) * a.G + n;
        const float inv = l[nt][i] > 0.f || l[nt][i] != l[nt][i] ? 1.f / l[nt][i] : 0.f;  // (NaN stays)
        if (a.lse && g == 0) a.lse[row] = l[nt][i] == 0.f ? -INFINITY : (m[nt][i] + log2f(l[nt][i])) * 0.69314718055994531f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (g + 8 * nb >= dh8) continue;
          float4* d = reinterpret_cast<float4*>(a.out + row * a.dh + 8 * (g + 8 * nb));
          d[0] = make_float4(o[nt][nb][0][i] * inv, o[nt][nb][1][i] * inv, o[nt][nb][2][i] * inv, o[nt][nb][3][i] * inv);
          d[1] = make_float4(o[nt][nb][0][2 + i] * inv, o[nt][nb][1][2 + i] * inv, o[nt][nb][2][2 + i] * inv, o[nt][nb][3][2 + i] * inv);
        }
      }
  };

  bool held = false, started = false;
  PagedAt cur = {0, 0, 0, 0};
  if (wlo < whi) {
    cur = locate(wlo);
    PagedAt nxt = cur;
    const int count = (int)(whi - wlo);
    int row = pool_row(cur);
    if (PRE) {
      load_k(row);
      load_v(row, 0, NB);
    }
    if (count > 1) {
      advance(nxt);
      if (PRE) row = pool_row(nxt);
    }
    started = cur.t == 0;
    begin_item(cur);
#pragma unroll 1
    for (int n = 0; n < count; ++n) {
      const bool more = n + 1 < count;
      if (!PRE) load_k(row);
      // scores of UNIT keys by 8 NT queries
      float s[NT][MT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float hi[MT][2][4] = {}, lo[MT][4] = {};
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const uint2* qd = q_mine + (nt * NK + k) * 3 * 32;
          const uint2 q0 = qd[0], q1 = qd[32], q2 = qd[64];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const Chunk<KT>&x = kc[2 * mt][k >> 1], &y = kc[2 * mt + 1][k >> 1];
            uint32_t f[SPL][4];
            if constexpr (!F32) {
              const int w = (k & 1) * 2;
              f[0][0] = x.word(w);
              f[0][1] = y.word(w);
              f[0][2] = x.word(w + 1);
              f[0][3] = y.word(w + 1);
            } else {
              const int e = (k & 1) * 4;
              split3(__uint_as_float(x.word(e)), __uint_as_float(x.word(e + 1)), f[0][0], f[1][0], f[2][0]);
              split3(__uint_as_float(y.word(e)), __uint_as_float(y.word(e + 1)), f[0][1], f[1][1], f[2][1]);
              split3(__uint_as_float(x.word(e + 2)), __uint_as_float(x.word(e + 3)), f[0][2], f[1][2], f[2][2]);
              split3(__uint_as_float(y.word(e + 2)), __uint_as_float(y.word(e + 3)), f[0][3], f[1][3], f[2][3]);
            }
            mma_bf16(lo[mt], f[0], q2.x, q2.y);
            if constexpr (F32) {
              mma_bf16(lo[mt], f[2], q0.x, q0.y);
              mma_bf16(lo[mt], f[1], q1.x, q1.y);
              mma_bf16(lo[mt], f[1], q0.x, q0.y);
            }
            mma_bf16(lo[mt], f[0], q1.x, q1.y);
            mma_bf16(hi[mt][k & 1], f[0], q0.x, q0.y);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[nt][mt][i] = (ok >> (2 * mt + (i >> 1))) & 1 ? (hi[mt][0][i] + hi[mt][1][i] + lo[mt][i]) * a.scale_log2 : -INFINITY;
      }
      if (PRE && more) load_k(row);
      // running maximum and sum; p in bf16 terms, transposed into B fragments
      uint32_t pf[NT][MT][3][2];
      float corr[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(s[nt][mt][i], s[nt][mt][2 + i]));
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          const float mn = fmaxf(m[nt][i], mx), mu = mn == -INFINITY ? 0.f : mn;
          corr[nt][i] = exp2f(m[nt][i] - mu);
          m[nt][i] = mn;
          float sum = 0.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            s[nt][mt][i] = exp2f(s[nt][mt][i] - mu);
            s[nt][mt][2 + i] = exp2f(s[nt][mt][2 + i] - mu);
            sum += s[nt][mt][i] + s[nt][mt][2 + i];
          }
          l[nt][i] = l[nt][i] * corr[nt][i] + sum;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t h, mm, ll;
            split3(s[nt][mt][2 * hf], s[nt][mt][2 * hf + 1], h, mm, ll);
            pf[nt][mt][0][hf] = transpose8x8(h);
            pf[nt][mt][1][hf] = transpose8x8(mm);
            pf[nt][mt][2][hf] = transpose8x8(ll);
          }
      }
      // o = o corr + V^T p
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (!PRE) load_v(row, nb, nb + 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float c[NT][4] = {};
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const Chunk<KT>* v = vc[nb] + 4 * mt;
            uint32_t f[SPL][4];
            if constexpr (!F32) {
              const uint32_t sel = (e & 1) ? 0x7632u : 0x5410u;
              f[0][0] = __byte_perm(v[0].word(e >> 1), v[1].word(e >> 1), sel);
              f[0][1] = __byte_perm(v[0].word(2 + (e >> 1)), v[1].word(2 + (e >> 1)), sel);
              f[0][2] = __byte_perm(v[2].word(e >> 1), v[3].word(e >> 1), sel);
              f[0][3] = __byte_perm(v[2].word(2 + (e >> 1)), v[3].word(2 + (e >> 1)), sel);
            } else {
              split3(__uint_as_float(v[0].word(e)), __uint_as_float(v[1].word(e)), f[0][0], f[1][0], f[2][0]);
              split3(__uint_as_float(v[0].word(4 + e)), __uint_as_float(v[1].word(4 + e)), f[0][1], f[1][1], f[2][1]);
              split3(__uint_as_float(v[2].word(e)), __uint_as_float(v[3].word(e)), f[0][2], f[1][2], f[2][2]);
              split3(__uint_as_float(v[2].word(4 + e)), __uint_as_float(v[3].word(4 + e)), f[0][3], f[1][3], f[2][3]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t(&pm)[3][2] = pf[nt][mt];
              mma_bf16(c[nt], f[0], pm[2][0], pm[2][1]);
              if constexpr (F32) {
                mma_bf16(c[nt], f[2], pm[0][0], pm[0][1]);
                mma_bf16(c[nt], f[1], pm[1][0], pm[1][1]);
                mma_bf16(c[nt], f[1], pm[0][0], pm[0][1]);
              }
              mma_bf16(c[nt], f[0], pm[1][0], pm[1][1]);
              mma_bf16(c[nt], f[0], pm[0][0], pm[0][1]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][nb][e][i] = fmaf(o[nt][nb][e][i], corr[nt][i & 1], c[nt][i]);
        }
      }
      if (PRE && more) load_v(row, 0, NB);
      const bool ends = cur.t + 1 == cur.nt;
      if (ends || !more) {
        total_l();
        if (started && ends) {
          output(cur.b, cur.it);
        } else if (!started && !lead) {
          put_part(reinterpret_cast<float4*>(s_part + warp * PARTF));
        } else if (ends) {  // an item that earlier CTAs began ends in the first warp
          put_part(reinterpret_cast<float4*>(a.part + (size_t)blockIdx.x * 2 * PARTF));
          if (lane == 0) {
            s_join[0][0] = wlo + n - cur.t;
            s_join[0][1] = wlo + n;
            s_joinat[0][0] = cur.b;
            s_joinat[0][1] = cur.it;
          }
        } else {
          held = true;
        }
      }
      if (more) {
        cur = nxt;
        if (n + 2 < count) advance(nxt);
        if (!PRE) row = pool_row(cur);
        else if (n + 2 < count) row = pool_row(nxt);
        if (ends) {
          started = true;
          begin_item(cur);
        }
      }
    }
  }
  __syncthreads();

  // What crosses warps: the item's first warp in this CTA adds the others' partials
  const long long chi = U * ((long long)(blockIdx.x + 1) * PGA_WARPS) / NW;
  if (held) {
    const long long first = whi - 1 - cur.t, end = first + cur.nt;
    for (int w = warp + 1; w < PGA_WARPS; ++w) {
      const long long lo = U * (blockIdx.x * PGA_WARPS + w) / NW, hi = U * (blockIdx.x * PGA_WARPS + w + 1) / NW;
      if (lo >= hi) continue;
      if (lo >= end) break;
      add_part(reinterpret_cast<const float4*>(s_part + w * PARTF), shared);
    }
    if (started && end <= chi) {
      output(cur.b, cur.it);
    } else {
      const int slot = started ? 1 : 0;
      put_part(reinterpret_cast<float4*>(a.part + ((size_t)blockIdx.x * 2 + slot) * PARTF));
      if (lane == 0) {
        s_join[slot][0] = first;
        s_join[slot][1] = end - 1;
        s_joinat[slot][0] = cur.b;
        s_joinat[slot][1] = cur.it;
      }
    }
  }
  __threadfence();
  __syncthreads();
  // What crosses CTAs: the last to arrive adds the partials of CTAs c0 .. c0 + n - 1
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const long long u0 = s_join[s][0];
    if (u0 < 0) continue;
    const int c0 = (int)(((u0 + 1) * NW - 1) / U) / PGA_WARPS;
    const int n = (int)(((s_join[s][1] + 1) * NW - 1) / U) / PGA_WARPS - c0 + 1;
    if (tid == 0) {
      const unsigned old = atomicAdd(a.tick + c0, 1u);
      s_last = old == (unsigned)(n - 1);
      if (s_last) a.tick[c0] = 0;
      __threadfence();
    }
    __syncthreads();
    if (s_last) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][nb][e][i] = 0.f;
      }
      for (int p = warp; p < n; p += PGA_WARPS)
        add_part(reinterpret_cast<const float4*>(a.part + ((size_t)(c0 + p) * 2 + (p == 0 ? 1 : 0)) * PARTF), global);
      if (warp > 0) put_part(reinterpret_cast<float4*>(s_part + warp * PARTF));
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < PGA_WARPS && w < n; ++w) add_part(reinterpret_cast<const float4*>(s_part + w * PARTF), shared);
        output(s_joinat[s][0], s_joinat[s][1]);
      }
    }
    __syncthreads();
  }
}

}  // namespace dv
