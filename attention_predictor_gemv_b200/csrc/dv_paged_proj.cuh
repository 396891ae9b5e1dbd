// The projections of the head-sparse attention block over a paged cache, bf16
// weights, up to 8 requests: q, k, v of the selected heads (k and v straight
// into their pages) and W^O.
//
// Both stream weight rows once through shared memory (asynchronous 16-byte
// copies, a ring per warp) into mma.sync m16n8k16 with the requests as rows:
// the fp32 operand enters as three bf16 terms (dv_paged.cuh), so the products
// are fp32's. The tensor core's sums are kept to one ring slot and added in
// fp32 outside. The eight warps of a CTA share the products' long axis and add
// their sums in warp order through shared memory: no atomics, results do not
// depend on timing. Bound by reading the weights.
#pragma once

#include "dv_paged.cuh"

namespace dv {

constexpr int PP_WARPS = 8, PP_THREADS = 32 * PP_WARPS;
constexpr int PP_MAX_B = 8;

template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}

// Two consecutive k slots of an operand row as A fragment words: rows 0-7 high
// above middle terms (`a`), low terms in rows 8-15 of `b`; of one request
// (ONE) high and middle in rows 0 and 8, low in row 1, all in `a`.
template <bool ONE>
__device__ __forceinline__ void a_words(float x, float y, int g, uint32_t& a_top, uint32_t& a_low, uint32_t& b_low) {
  uint32_t h, m, l;
  split3(x, y, h, m, l);
  // (masks: choices by row became branches)
  const uint32_t row0 = g == 0 ? ~0u : 0u, row1 = g == 1 ? ~0u : 0u;
  a_top = ONE ? (h & row0) | (l & row1) : h;
  a_low = ONE ? m & row0 : m;
  b_low = l;
}

// ----------------------------------------------------------------------------
// q, k, v. Weight rows Wqkv[head][3][dh][d] of the selected heads (and, with
// `all`, k and v of the others) form tiles of 8 rows; a CTA takes an equal
// share of the tiles, its warps a share of the d channels each. y lies in shared
// memory, since loads of it within the loop queue behind the weights in flight.
// k and v are rounded into slots[b]; without `all` the places of the other heads
// are cleared. Two forms, below.
// 5376 rows of 12288 channels (132 MB), one request: 34 us under a profiler,
// 3.9 TB/s; 7680 rows of 4096 channels (63 MB), four requests: 22 us. Bound by
// the 4 us before the first rows arrive, by CTAs of five tiles where the mean is
// 4.5, by the rows read once more (below, 2 us), and with more requests by the
// loop's instructions.
// ----------------------------------------------------------------------------
struct PagedQkvArgs {
  const __nv_bfloat16* W;
  const float* bias;
  const float* y;
  const int32_t *head_idx, *head_count;
  const int32_t* slots;
  float* q;  // [B][kh_max][dh]
  __nv_bfloat16 *K, *V;
  int* status;
  int B, d, h, dh, kh_max, all, page, stride_rows, n_slots;
};

// A tile's place: its head (-1: none), which of q, k, v, first channel, place in the set
struct QkvTile {
  int head, m, c, j;
};

// The set's size, clamped and flagged, and the heads outside it in order (s_rest, s_nrest); by a whole block, first of
// all: with the first weights on their way it took 6 us more at four requests.
__device__ __forceinline__ int qkv_lists(const PagedQkvArgs& a, short* s_rest, int* s_nrest) {
  const int tid = threadIdx.x, nth = blockDim.x, lane = tid & 31;
  int nsel = *a.head_count;
  if (nsel < 0 || nsel > a.kh_max) {
    if (blockIdx.x == 0 && tid == 0) raise_status(a.status, ST_CLAMPED);
    nsel = nsel < 0 ? 0 : a.kh_max;
  }
  for (int i = tid; i < a.h; i += nth) s_rest[i] = 0;
  __syncthreads();
  for (int j = tid; j < nsel; j += nth) {
    const int head = a.head_idx[j];
    if (head >= 0 && head < a.h) s_rest[head] = 1;
    else if (blockIdx.x == 0) raise_status(a.status, ST_RANGE);
  }
  __syncthreads();
  if (tid < 32) {
    int n = 0;
    for (int i0 = 0; i0 < a.h; i0 += 32) {
      const bool rest = i0 + lane < a.h && !s_rest[min(i0 + lane, a.h - 1)];
      const unsigned in = __ballot_sync(0xffffffffu, rest);
      __syncwarp();
      if (rest) s_rest[n + __popc(in & ((1u << lane) - 1u))] = (short)(i0 + lane);  // (never past what was read)
      __syncwarp();
      n += __popc(in);
    }
    if (lane == 0) *s_nrest = n;
  }
  __syncthreads();
  return nsel;
}

__device__ __forceinline__ QkvTile qkv_tile(const PagedQkvArgs& a, int nsel, const short* s_rest, int t) {
  const int per = a.dh >> 3, sel_tiles = nsel * 3 * per;  // tiles of one head's q, k or v; of the set
  QkvTile p;
  if (t < sel_tiles) {
    p.j = t / (3 * per);
    const int r = t - p.j * 3 * per;
    p.m = r / per;
    p.c = (r - p.m * per) * 8;
    p.head = a.head_idx[p.j];
    if (p.head >= a.h) p.head = -1;
  } else {
    const int u = t - sel_tiles, i = u / (2 * per), r = u - i * 2 * per;
    p.j = -1;
    p.m = 1 + r / per;
    p.c = (r - (p.m - 1) * per) * 8;
    p.head = s_rest[i];
  }
  return p;
}

// Values of k and v next to a rounding border.
//
// One bf16 step of one stored value moves the output by up to 2e-4 of its norm where few keys are attended to, and fp32
// sums in another order fall on the other side of a border for one value in some thousands. So k and v are what the
// exact sum gives, rounded to fp32 and then to bf16, whatever the kernel's form or the number of requests: a sum so
// close to a border that its own error could decide is formed again in 64 bits, its row read once more. The sums'
// errors are 1.4e-7 of a value's spread in the mean square (2048 to 12288 channels). The magnitudes of the eight warps'
// partial sums, added, are 2.3 times that spread for independent terms, but no more than the value itself where one warp
// has all channels, so the largest of the 32 values that a warp stores is taken: 2 to 4 times the spread, and 2^-22 of it
// 4 to 7 times the error (fewer channels have smaller errors).
// About one value in 500 is formed again, by the whole CTA at its end: 2500 cycles each of 4096 channels and 8000 of 12288,
// nearly all of them the loads while other SMs stream. A call with one request of 4096 channels takes 39 us with it and
// 38 without, with four 48.5 for 46, with eight 63 for 60; one request of 12288 channels 53.5 for 52, eight 103 for 96. By
// a warp each, at once, four requests took 53 us and one of 12288 channels 64; the loads through shared memory, all at
// once, the same as this; the loop unrolled by three or six up to 1.5 us more with 4096 channels.
constexpr int QC_ENTRIES = PP_THREADS + 128, QC_ROUND = 32;
struct QkvClose {
  long long to[QC_ENTRIES];  // the value's element of its pool, doubled, odd: of V
  int row[QC_ENTRIES], b[QC_ENTRIES];
  double sum[QC_ROUND][PP_WARPS];
  int n;
};

// Entries' values in 64 bits (products are exact there): each warp takes every eighth 256 channels.
__device__ __forceinline__ void qkv_again(const PagedQkvArgs& a, QkvClose& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = s.n;
  for (int i0 = 0; i0 < n; i0 += QC_ROUND) {
    const int m = min(QC_ROUND, n - i0);
#pragma unroll 1
    for (int i = 0; i < m; ++i) {
      const __nv_bfloat16* w = a.W + (size_t)s.row[i0 + i] * a.d;
      const float* y = a.y + (size_t)s.b[i0 + i] * a.d;
      double part[8] = {};
#pragma unroll 1
      for (int c = 256 * warp + 8 * lane; c < a.d; c += 256 * PP_WARPS) {
        const uint4 u = *reinterpret_cast<const uint4*>(w + c);
        const float4 y0 = *reinterpret_cast<const float4*>(y + c), y1 = *reinterpret_cast<const float4*>(y + c + 4);
        const float ys[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = word_of(u, e >> 1);
          part[e] = fma((double)__uint_as_float(e & 1 ? x & 0xffff0000u : x << 16), (double)ys[e], part[e]);
        }
      }
      double sum = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) s.sum[i][warp] = sum;
    }
    __syncthreads();
    if (tid < m) {
      double v = a.bias ? (double)a.bias[s.row[i0 + tid]] : 0.0;
#pragma unroll
      for (int w = 0; w < PP_WARPS; ++w) v += s.sum[tid][w];
      const long long to = s.to[i0 + tid];
      (to & 1 ? a.V : a.K)[to >> 1] = __float2bfloat16_rn((float)v);
    }
    __syncthreads();
  }
  if (tid == 0) s.n = 0;
}

// Where a sum goes: m 0 to q, 1 to K, 2 to V, at element `to`; -1: nowhere. Formed before the sum, since the loads that it
// and the bias need follow one another.
struct QkvPlace {
  int m, row;  // (weight row)
  long long to;
  float bias;
};

__device__ __forceinline__ QkvPlace qkv_place(const PagedQkvArgs& a, const QkvTile& p, int b, int slot, int r) {
  QkvPlace t = {-1, 0, 0, 0.f};
  if (p.head < 0) return t;
  const int c = p.c + r;
  t.row = (p.head * 3 + p.m) * a.dh + c;
  if (a.bias) t.bias = a.bias[t.row];
  if (p.m == 0) {
    t.m = 0;
    t.to = ((long long)b * a.kh_max + p.j) * a.dh + c;
  } else if (slot >= 0 && slot < a.n_slots) {
    const int pg = slot / a.page;
    t.m = p.m;
    t.to = ((long long)pg * a.stride_rows + p.head * a.page + (slot - pg * a.page)) * a.dh + c;
  } else if (slot >= 0) {
    raise_status(a.status, ST_RANGE);
  }
  return t;
}

// A warp's values to their places: each the sum of the warps' partial sums, `step` floats apart, and the bias
__device__ __forceinline__ void qkv_store(const PagedQkvArgs& a, const QkvPlace& t, int b, const float* part, int step, QkvClose& s) {
  float v = 0.f, mag = 0.f;
  if (t.m >= 0) {
#pragma unroll
    for (int w = 0; w < PP_WARPS; ++w) {
      const float x = part[w * step];
      v += x;
      mag += fabsf(x);
    }
  }
  v += t.bias;
  mag = __uint_as_float(__reduce_max_sync(0xffffffffu, mag < INFINITY ? __float_as_uint(mag) : 0u));
  if (t.m == 0) a.q[t.to] = v;
  if (t.m <= 0) return;
  (t.m == 1 ? a.K : a.V)[t.to] = __float2bfloat16_rn(v);
  const float border = __uint_as_float((__float_as_uint(v) & 0xffff0000u) | 0x8000u);
  if (fabsf(v - border) <= (mag + fabsf(v)) * 0x1p-22f) {
    const int i = atomicAdd(&s.n, 1);
    s.to[i] = 2 * t.to + (t.m == 2);
    s.row[i] = t.row;
    s.b[i] = b;
  }
}

// The places of the heads outside the set
__device__ __forceinline__ void qkv_clear(const PagedQkvArgs& a, const short* s_rest, int n_rest) {
  const int n = n_rest * a.B, vecs = a.dh >> 3;  // (head, request) pairs, 16-byte vectors of each
  for (int x = blockIdx.x * blockDim.x + threadIdx.x; x < n * vecs; x += gridDim.x * blockDim.x) {
    const int pr = x / vecs, v = x - pr * vecs, b = pr % a.B, head = s_rest[pr / a.B];
    const int slot = a.slots[b];
    if (slot < 0 || slot >= a.n_slots) {
      if (slot >= 0) raise_status(a.status, ST_RANGE);
      continue;
    }
    const int pg = slot / a.page;
    const long long row = (long long)pg * a.stride_rows + head * a.page + (slot - pg * a.page);
    reinterpret_cast<uint4*>(a.K)[row * vecs + v] = make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(a.V)[row * vecs + v] = make_uint4(0, 0, 0, 0);
  }
}

// Tiles of 8 rows that a call can have: q, k, v for every entry of the set, and k, v for every head that no valid entry
// names (entries out of range or repeated name none, so a set of h entries can leave all h heads to the rest)
__host__ __device__ constexpr long long qkv_most_tiles(int kh_max, int h, int dh, bool all) {
  return (3ll * kh_max + (all ? 2ll * h : 0)) * (dh / 8);
}
constexpr int PQ_MAX_TILES = 576;  // of a CTA; more on an SM: refused on the host. 1000 entries, 1024 heads of 128 on 148 SMs: 546

// One request: a tile of 8 rows at a time, 512 channels of each row a warp and ring slot, so that what lies together in
// memory is read together; y's terms, formed once, come from shared memory, and limit it to 12288 channels. Whole calls
// with 512, 2048, 4096, 8192 and 12288 channels: 15.2, 19.6, 37.1, 46.0 and 54.3 us; by the other form 15.6, 20.2, 38.5,
// 48.5 and 60.3.
constexpr int PT_CW = 512, PT_PITCH = 2 * PT_CW + 16, PT_SLOT = 8 * PT_PITCH, PT_SLOTS = 2, PT_MAX_D = 12288;
constexpr int PT_HOLD = 8;  // tiles whose sums are kept before the warps' are added
constexpr int PT_RING = PP_WARPS * PT_SLOTS * PT_SLOT, PT_RED = PT_HOLD * PP_WARPS * 8 * 4;
constexpr size_t paged_qkv_one_smem() { return PT_RING + PT_RED + 3 * 2 * (PT_MAX_D + 8); }
static_assert(paged_qkv_one_smem() + 2 * PTK_MAX_H + 4 * PQ_MAX_TILES + sizeof(QkvClose) + 1024 <= 227 * 1024, "shared memory");

__global__ void __launch_bounds__(PP_THREADS, 1) paged_qkv_one_kernel(PagedQkvArgs a) {
  constexpr int CW = PT_CW, SLOTS = PT_SLOTS, PITCH = PT_PITCH, CPR = CW / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(16) char ring[];
  __shared__ short s_rest[PTK_MAX_H];
  __shared__ int s_nrest, s_row[PQ_MAX_TILES];  // a tile's first weight row, -1: none
  __shared__ QkvClose s_close;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  float* red = reinterpret_cast<float*>(ring + PP_WARPS * SLOTS * PT_SLOT);  // [tiles held][warps][8 rows]
  __nv_bfloat16* s_y = reinterpret_cast<__nv_bfloat16*>(ring + PP_WARPS * SLOTS * PT_SLOT + PT_RED);
  if (tid == 0) s_close.n = 0;
  griddep_wait();
  griddep_launch();  // (after the wait: what starts early finds everything before this call complete)
  const int slot_of = a.slots[0];
  const int nsel = qkv_lists(a, s_rest, &s_nrest);
  const int tiles = (nsel * 3 + (a.all ? s_nrest * 2 : 0)) * (a.dh >> 3);
  const int t0 = (int)((long long)tiles * blockIdx.x / gridDim.x), t1 = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  for (int t = t0 + tid; t < t1; t += PP_THREADS) {
    const QkvTile p = qkv_tile(a, nsel, s_rest, t);
    s_row[t - t0] = p.head < 0 ? -1 : (p.head * 3 + p.m) * a.dh + p.c;
  }
  __syncthreads();
  const int blocks = (a.d + CW - 1) / CW, nk = (blocks + PP_WARPS - 1 - warp) / PP_WARPS;  // blocks warp, warp + 8, ...
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring) + warp * SLOTS * PT_SLOT;
  int rt = t0, rk = 0, rs = 0;  // requested next: tile, block, slot
  auto request = [&]() {
    if (rt < t1 && nk > 0) {
      const int row = s_row[rt - t0], ch0 = (warp + rk * PP_WARPS) * CW;
      const uint32_t to = base + rs * PT_SLOT;
      const __nv_bfloat16* src = a.W + (row >= 0 ? (size_t)row * a.d + ch0 : 0);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
#pragma unroll
        for (int c = lane; c < CPR; c += 32) {
          const bool on = row >= 0 && ch0 + 8 * c < a.d;
          copy16_or_zero(to + r * PITCH + c * 16, src + (on ? 8 * c : 0), on);
        }
        if (row >= 0) src += a.d;
      }
      rs = rs + 1 == SLOTS ? 0 : rs + 1;
      if (++rk == nk) rk = 0, ++rt;
    }
    copies_commit();
  };
#pragma unroll
  for (int u = 0; u < SLOTS - 1; ++u) request();
  // y's terms: high, middle, low [B][pitch]
  const int width = blocks * CW, pitch = width + 8;
  for (int c = 4 * tid; c < width; c += 4 * PP_THREADS) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.d) v = *reinterpret_cast<const float4*>(a.y + c);
    uint2 h, m, l;
    split3(v.x, v.y, h.x, m.x, l.x);
    split3(v.z, v.w, h.y, m.y, l.y);
    *reinterpret_cast<uint2*>(s_y + c) = h;
    *reinterpret_cast<uint2*>(s_y + pitch + c) = m;
    *reinterpret_cast<uint2*>(s_y + 2 * pitch + c) = l;
  }
  __syncthreads();
  // row 0's lanes have y's high and middle terms, row 1's the low ones
  const __nv_bfloat16* y_top = s_y + (g == 1 ? 2 * pitch : 0) + warp * CW + 16 * t4;
  const __nv_bfloat16* y_mid = s_y + pitch + warp * CW + 16 * t4;
  const uint32_t on_top = g < 2 ? ~0u : 0u, on_mid = g == 0 ? ~0u : 0u;
  int slot = 0;
#pragma unroll 1
  for (int ta = t0; ta < t1; ta += PT_HOLD) {
    const int held = min(PT_HOLD, t1 - ta);
    QkvPlace place = {-1, 0, 0, 0.f};
    if (tid < held * 8) place = qkv_place(a, qkv_tile(a, nsel, s_rest, ta + (tid >> 3)), 0, slot_of, tid & 7);
#pragma unroll 1
    for (int i = 0; i < held; ++i) {
      float acc[2] = {0.f, 0.f};
#pragma unroll 1
      for (int k = 0; k < nk; ++k) {
        request();
        copies_wait<SLOTS - 1>();
        const char* w = ring + (warp * SLOTS + slot) * PT_SLOT + g * PITCH + t4 * 32;
        slot = slot + 1 == SLOTS ? 0 : slot + 1;
        const int ko = k * PP_WARPS * CW;
        float c[4][4];
#pragma unroll
        for (int p = 0; p < CW / 32; ++p) {  // 16 bytes: eight channels, two steps; four sums side by side
          const int at = 64 * (p >> 1) + 8 * (p & 1);
          const uint4 v = *reinterpret_cast<const uint4*>(w + 2 * at);
          const uint4 h = *reinterpret_cast<const uint4*>(y_top + ko + at), m = *reinterpret_cast<const uint4*>(y_mid + ko + at);
          const uint32_t f0[4] = {h.x & on_top, m.x & on_mid, h.y & on_top, m.y & on_mid};
          const uint32_t f1[4] = {h.z & on_top, m.z & on_mid, h.w & on_top, m.w & on_mid};
          float(&x)[4] = c[2 * (p & 1)], (&z)[4] = c[2 * (p & 1) + 1];
          if (p < 2) {
            mma_bf16_first(x, f0, v.x, v.y);
            mma_bf16_first(z, f1, v.z, v.w);
          } else {
            mma_bf16(x, f0, v.x, v.y);
            mma_bf16(z, f1, v.z, v.w);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
          acc[e] += ((c[0][e] + c[0][2 + e]) + (c[1][e] + c[1][2 + e])) + ((c[2][e] + c[2][2 + e]) + (c[3][e] + c[3][2 + e]));
        __syncwarp();  // the slot is free
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float v = acc[e] + __shfl_xor_sync(0xffffffffu, acc[e], 4);
        if (g == 0) red[(i * PP_WARPS + warp) * 8 + 2 * t4 + e] = v;
      }
    }
    __syncthreads();
    if (warp < PT_HOLD / 4) qkv_store(a, place, 0, red + (tid >> 3) * PP_WARPS * 8 + (tid & 7), 8, s_close);
    __syncthreads();
    if (s_close.n > QC_ENTRIES - PP_THREADS || ta + PT_HOLD >= t1) {
      qkv_again(a, s_close);
      __syncthreads();
    }
  }
  if (!a.all) qkv_clear(a, s_rest, s_nrest);
}

// More requests (or channels): they are the rows; a slot holds four tiles of 128 channels, and y's terms are formed once
// for them, from y in shared memory (a segment of the channels at a time where it is larger than 64 KB). With four
// requests of 4096 channels the form above took 25 us where this took 20; slots of 64 channels of eight tiles, or 16
// warps, the same time.
constexpr int PQ_TILES = 4, PQ_SLOTS = 2, PQ_PITCH = 256 + 16;
constexpr int PQ_SLOT = PQ_TILES * 8 * PQ_PITCH;
constexpr int PQ_STRIDE = 128 * PP_WARPS;                // channels that the warps take side by side
constexpr int PQ_YF = 16384;                             // floats of y at a time
constexpr int PQ_YPAD = 4;                               // of each request's row, in floats
constexpr size_t PQ_RING = (size_t)PP_WARPS * PQ_SLOTS * PQ_SLOT;
constexpr size_t paged_qkv_smem() { return PQ_RING + 4 * (PQ_YF + PP_MAX_B * PQ_YPAD); }
static_assert(paged_qkv_smem() + 2 * PTK_MAX_H + PP_WARPS * PQ_TILES * 8 * 9 * 4 + 4 * PQ_MAX_TILES + sizeof(QkvClose) + 1024 <= 227 * 1024, "shared memory");

__global__ void __launch_bounds__(PP_THREADS, 1) paged_qkv_kernel(PagedQkvArgs a) {
  constexpr int QR = PP_MAX_B;
  extern __shared__ __align__(16) char ring[];
  __shared__ short s_rest[PTK_MAX_H];
  __shared__ float red[PP_WARPS][PQ_TILES * 8][QR + 1];
  __shared__ int s_nrest, s_row[PQ_MAX_TILES];  // a tile's first weight row, -1: none
  __shared__ QkvClose s_close;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  if (tid == 0) s_close.n = 0;
  griddep_wait();
  griddep_launch();  // (after the wait: what starts early finds everything before this call complete)

  // y, a segment of the channels, on its way to shared memory; channels past d become zeros
  float* s_y = reinterpret_cast<float*>(ring + PQ_RING);
  const int seg = min((a.d + PQ_STRIDE - 1) / PQ_STRIDE, PQ_YF / PQ_STRIDE / a.B);  // strides of channels at a time
  const int pitch = seg * PQ_STRIDE + PQ_YPAD;
  auto request_y = [&](int i0) {
    const int n4 = min(seg * PQ_STRIDE, a.d - i0 * PQ_STRIDE) >> 2;
    for (int b = 0; b < a.B; ++b)
      for (int i = tid; i < seg * PQ_STRIDE / 4; i += PP_THREADS)
        copy16_or_zero((uint32_t)__cvta_generic_to_shared(s_y + b * pitch + 4 * i),
                       a.y + (i < n4 ? (size_t)b * a.d + i0 * PQ_STRIDE + 4 * i : 0), i < n4);
    copies_commit();
  };
  request_y(0);

  const int b_of = tid / (PQ_TILES * 8), slot_of = a.slots[min(b_of, a.B - 1)];  // the request whose sums this thread stores
  const int nsel = qkv_lists(a, s_rest, &s_nrest);
  const int tiles = (nsel * 3 + (a.all ? s_nrest * 2 : 0)) * (a.dh >> 3);
  const int t0 = (int)((long long)tiles * blockIdx.x / gridDim.x), t1 = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  for (int t = t0 + tid; t < t1; t += PP_THREADS) {
    const QkvTile p = qkv_tile(a, nsel, s_rest, t);
    s_row[t - t0] = p.head < 0 ? -1 : (p.head * 3 + p.m) * a.dh + p.c;
  }
  __syncthreads();
  if (t1 > t0) {
    const int passes = (t1 - t0 + PQ_TILES - 1) / PQ_TILES, nt = (t1 - t0 + passes - 1) / passes;
    const int blocks = (a.d + 127) >> 7;
    const int nk = (blocks + PP_WARPS - 1 - warp) / PP_WARPS;  // blocks warp, warp + 8, ...: side by side in a row
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(ring) + warp * PQ_SLOTS * PQ_SLOT + (lane >> 4) * PQ_PITCH + (lane & 15) * 16;
    const char* mine = ring + warp * PQ_SLOTS * PQ_SLOT;
    // what is requested next: pass rp, the warp's block rk; its tiles' rows (this lane's first) and which there are
    int rp = 0, rk = 0, rs = 0;
    const char* src[PQ_TILES];
    unsigned there = 0;
    auto rows_of_pass = [&]() {
      there = 0;
#pragma unroll
      for (int i = 0; i < PQ_TILES; ++i) {
        const int t = t0 + rp * nt + i, row = i < nt && t < t1 ? s_row[t - t0] : -1;
        there |= row >= 0 ? 1u << i : 0u;
        src[i] = reinterpret_cast<const char*>(a.W + (row >= 0 ? (size_t)(row + (lane >> 4)) * a.d : 0));
      }
    };
    if (nk > 0) rows_of_pass();
    const size_t two_rows = 4ull * a.d;  // bytes
    auto request = [&]() {
      if (nk > 0 && rp < passes) {
        const int ch = (warp + rk * PP_WARPS) * 128 + (lane & 15) * 8;
        const uint32_t to = at + rs * PQ_SLOT;
#pragma unroll
        for (int i = 0; i < PQ_TILES; ++i) {
          if (i >= nt) break;
          const bool on = (there >> i & 1) && ch < a.d;
          const char* p = src[i] + (on ? 2 * ch : 0);
#pragma unroll
          for (int r = 0; r < 8; r += 2) {
            copy16_or_zero(to + (8 * i + r) * PQ_PITCH, p, on);
            if (on) p += two_rows;
          }
        }
        rs = rs + 1 == PQ_SLOTS ? 0 : rs + 1;
        if (++rk == nk) {
          rk = 0;
          if (++rp < passes) rows_of_pass();
        }
      }
      copies_commit();
    };
#pragma unroll
    for (int u = 0; u < PQ_SLOTS - 1; ++u) request();
    int slot = 0;
    for (int pass = 0; pass < passes; ++pass) {
      float acc[PQ_TILES][2] = {};
      QkvPlace place = {-1, 0, 0, 0.f};
      {
        const int i = (tid >> 3) % PQ_TILES, t = t0 + pass * nt + i;
        if (i < nt && t < t1 && b_of < a.B) place = qkv_place(a, qkv_tile(a, nsel, s_rest, t), b_of, slot_of, tid & 7);
      }
      for (int i0 = 0; i0 * PQ_STRIDE < a.d; i0 += seg) {
        if (pass + i0 == 0) {  // the first segment: all but the ring's groups
          copies_wait<PQ_SLOTS - 1>();
          __syncthreads();
        } else if (seg * PQ_STRIDE < a.d) {
          __syncthreads();
          request_y(i0);
          copies_wait<0>();
          __syncthreads();
        }
#pragma unroll 1
      for (int k = i0; k < min(nk, i0 + seg); ++k) {
        request();
        uint32_t fa[8][4], fb[8][2];
        const float* yp = s_y + g * pitch + (k - i0) * PQ_STRIDE + warp * 128 + 16 * t4;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (g < a.B) x = *reinterpret_cast<const float4*>(yp + 64 * (s >> 2) + 4 * (s & 3));
          split3(x.x, x.y, fa[s][0], fa[s][1], fb[s][0]);
          split3(x.z, x.w, fa[s][2], fa[s][3], fb[s][1]);
        }
        copies_wait<PQ_SLOTS - 1>();
        const char* w = mine + slot * PQ_SLOT + g * PQ_PITCH + t4 * 32;
        slot = slot + 1 == PQ_SLOTS ? 0 : slot + 1;
        float c[PQ_TILES][4];
#pragma unroll
        for (int piece = 0; piece < 4; ++piece) {
          uint4 v[PQ_TILES];
#pragma unroll
          for (int i = 0; i < PQ_TILES; ++i) v[i] = *reinterpret_cast<const uint4*>(w + 8 * i * PQ_PITCH + (piece >> 1) * 128 + (piece & 1) * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int s = 2 * piece + h;
#pragma unroll
            for (int i = 0; i < PQ_TILES; ++i) {
              const uint32_t b0 = h ? v[i].z : v[i].x, b1 = h ? v[i].w : v[i].y;
              if (s == 0) mma_bf16_first(c[i], fa[s], b0, b1);
              else mma_bf16(c[i], fa[s], b0, b1);
            }
            const uint32_t low[4] = {0u, fb[s][0], 0u, fb[s][1]};
#pragma unroll
            for (int i = 0; i < PQ_TILES; ++i) mma_bf16(c[i], low, h ? v[i].z : v[i].x, h ? v[i].w : v[i].y);
          }
        }
#pragma unroll
        for (int i = 0; i < PQ_TILES; ++i) {
          acc[i][0] += c[i][0] + c[i][2];
          acc[i][1] += c[i][1] + c[i][3];
        }
        __syncwarp();  // the slot is free
      }
      }
#pragma unroll
      for (int i = 0; i < PQ_TILES; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) red[warp][8 * i + 2 * t4 + e][g] = acc[i][e];
      __syncthreads();
      static_assert(PQ_TILES * 8 * QR == PP_THREADS, "a sum each");
      qkv_store(a, place, b_of, &red[0][tid % (PQ_TILES * 8)][b_of], PQ_TILES * 8 * (QR + 1), s_close);
      __syncthreads();
      if (s_close.n > QC_ENTRIES - PP_THREADS || pass + 1 == passes) {
        qkv_again(a, s_close);
        __syncthreads();
      }
    }
  }
  if (!a.all) qkv_clear(a, s_rest, s_nrest);
}

// ----------------------------------------------------------------------------
// W^O: out[b][c] (+)= sum_r H[b][r] WOt[row r][c] (+ bO[c]) over the rows of
// the selected heads. A CTA takes 8 NC columns and all rows, its warps a share
// of the rows each, 32 rows a ring slot; the weights are the MMA's columns,
// read by transposing matrix loads. The ring is filled before the wait for the
// attention, which writes H alone. 1792 rows of 12288 columns (44 MB), one
// request: 12 us; 2560 rows of 4096, four requests: 10.5 us; bound by the ring's
// start and the last round of a ring that is as long as the work.
// ----------------------------------------------------------------------------
struct PagedWoArgs {
  const __nv_bfloat16* W;
  const float* bias;
  const float* H;  // [B][kh_max][dh]
  const int32_t *head_idx, *head_count;
  float* out;
  int* status;
  int B, d, h, dh, kh_max, accumulate;
};

template <int NC>
struct PagedWoShape {
  static constexpr int CB = 8 * NC, PITCH = 2 * CB + 16, HPITCH = 36;  // (floats; rows of H in other banks)
  static constexpr int ROWS = 32 * PITCH, SLOT = ROWS + PP_MAX_B * HPITCH * 4;
  static constexpr int FIT = 200 * 1024 / (PP_WARPS * SLOT), SLOTS = FIT < 6 ? FIT : 6;
  static_assert(SLOTS >= 2 && PP_WARPS * SLOTS * SLOT >= PP_WARPS * 8 * CB * 4, "the ring holds the warps' sums at the end");
};

template <int QR, int NC>
__global__ void __launch_bounds__(PP_THREADS, 1) paged_wo_kernel(PagedWoArgs a) {
  constexpr bool ONE = QR == 1;
  using S = PagedWoShape<NC>;
  constexpr int CB = S::CB, PITCH = S::PITCH, SLOTS = S::SLOTS, PIECES = CB / 8;  // 16-byte pieces of a row
  extern __shared__ __align__(16) char ring[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  int nsel = *a.head_count;
  nsel = nsel < 0 ? 0 : min(nsel, a.kh_max);
  const int per = a.dh >> 5, nu = nsel * per;  // units of 32 rows
  const int ulo = nu * warp / PP_WARPS, units = nu * (warp + 1) / PP_WARPS - ulo;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring) + warp * SLOTS * S::SLOT;
  bool waited = false;
  for (int c0 = blockIdx.x * CB; c0 < a.d; c0 += gridDim.x * CB) {
    auto request = [&](int u) {
      if (u < units) {
        const int j = (ulo + u) / per, head = a.head_idx[j];
        const bool good = head >= 0 && head < a.h;
        const __nv_bfloat16* src = a.W + (good ? ((size_t)head * a.dh + (ulo + u - j * per) * 32) * a.d + c0 : 0);
        const uint32_t to = base + (u % SLOTS) * S::SLOT;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const int e = i * 32 + lane, r = e / PIECES, c = e - r * PIECES;
          const bool on = good && c0 + 8 * c < a.d;
          copy16_or_zero(to + r * PITCH + c * 16, src + (on ? (size_t)r * a.d + 8 * c : 0), on);
        }
      }
    };
    // H of its rows, [B][32]
    auto request_h = [&](int u) {
      if (u < units)
        for (int i = lane; i < 8 * a.B; i += 32)
          copy16(base + (u % SLOTS) * S::SLOT + S::ROWS + ((i >> 3) * S::HPITCH + 4 * (i & 7)) * 4,
                 a.H + (size_t)(i >> 3) * a.kh_max * a.dh + (ulo + u) * 32 + 4 * (i & 7));
    };
#pragma unroll
    for (int u = 0; u < SLOTS - 1; ++u) {
      request(u);
      copies_commit();
    }
    if (!waited) griddep_wait(), waited = true;  // H, and the last readers and writers of out
#pragma unroll
    for (int u = 0; u < SLOTS - 1; ++u) request_h(u);
    copies_commit();
    float acc[NC][2] = {};
#pragma unroll 1
    for (int u = 0; u < units; ++u) {
      request(u + SLOTS - 1);
      request_h(u + SLOTS - 1);
      copies_commit();
      if (u == 0) copies_wait<1>();  // (H of the first slots came last)
      else copies_wait<SLOTS - 1>();
      // two steps of 16 rows, k slots 2 t, + 1, + 8, + 9 of each
      uint32_t fa[2][4], fb[2][2];
      const float* hp = reinterpret_cast<const float*>(ring + (warp * SLOTS + u % SLOTS) * S::SLOT + S::ROWS) + (ONE ? 0 : g) * S::HPITCH + 2 * t4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 x = make_float2(0.f, 0.f);
        if (ONE || g < a.B) x = *reinterpret_cast<const float2*>(hp + 8 * i);
        a_words<ONE>(x.x, x.y, g, fa[i >> 1][2 * (i & 1)], fa[i >> 1][2 * (i & 1) + 1], fb[i >> 1][i & 1]);
      }
      const uint32_t w = base + (u % SLOTS) * S::SLOT + ((lane >> 3 & 1) * 8 + (lane & 7)) * PITCH + (lane >> 4) * 16;
#pragma unroll
      for (int n = 0; n < NC; n += 2) {
        float c[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t b[4];
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                       : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                       : "r"(w + 16 * k * PITCH + n * 16)
                       : "memory");
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (k == 0) mma_bf16_first(c[i], fa[k], b[2 * i], b[2 * i + 1]);
            else mma_bf16(c[i], fa[k], b[2 * i], b[2 * i + 1]);
          }
          if constexpr (!ONE) {
            const uint32_t low[4] = {0u, fb[k][0], 0u, fb[k][1]};
#pragma unroll
            for (int i = 0; i < 2; ++i) mma_bf16(c[i], low, b[2 * i], b[2 * i + 1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[n + i][0] += c[i][0] + c[i][2];
          acc[n + i][1] += c[i][1] + c[i][3];
        }
      }
      __syncwarp();  // the slot is free
    }
    copies_wait<0>();
    __syncthreads();  // the rings are free
    float* red = reinterpret_cast<float*>(ring);  // [warps][QR][CB]
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = acc[n][e];
        if constexpr (ONE) v += __shfl_xor_sync(0xffffffffu, v, 4);
        if (!ONE || g == 0) red[(warp * QR + (ONE ? 0 : g)) * CB + 8 * n + 2 * t4 + e] = v;
      }
    __syncthreads();
    for (int i = tid; i < a.B * CB; i += PP_THREADS) {
      const int b = i / CB, c = i - b * CB;
      if (c0 + c >= a.d) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < PP_WARPS; ++w) v += red[(w * QR + b) * CB + c];
      if (a.bias) v += a.bias[c0 + c];
      float* o = a.out + (size_t)b * a.d + c0 + c;
      *o = a.accumulate ? *o + v : v;
    }
    __syncthreads();
  }
  if (!waited) griddep_wait();
  griddep_launch();
}

}  // namespace dv
