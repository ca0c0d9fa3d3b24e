// The paged key-value cache: appending new tokens (with RoPE on the way), choosing the pages a
// decode query reads, and attention of one new token per sequence over its pages.
//
// A pool holds n_pages pages of page_size positions: K and V [page, kv head, row, D] through
// three strides, 16-bit.  A block table row lists a sequence's pages in order, so position p
// of sequence b is row p % page_size of page table[b][p / page_size].  Optional page bounds
// keep the smallest and largest key value per channel, [page, kv head, D].
#pragma once
#include "common.cuh"
#include "misc.cuh"

namespace hymba {

// ----------------------------------------------------------------------------------------
// 16-bit element types of a pool
// ----------------------------------------------------------------------------------------
template <typename E>
struct Elem;
template <>
struct Elem<__half> {
  static constexpr bool IS_F16 = true;
  __device__ static uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
  __device__ static float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }
  // d (16x8 fp32) += a (16x16, row-major) * b (16x8, column-major)
  __device__ static void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    mma_16816(d, a0, a1, a2, a3, b0, b1);
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr bool IS_F16 = false;
  __device__ static uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  __device__ static float2 unpack(uint32_t v) { return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v)); }
  __device__ static void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3)
      : "memory");
}

enum { PDT_F32 = 0, PDT_BF16 = 1, PDT_F16 = 2 };   // element types at the boundary (HYMBA_DT_*)

// two consecutive outputs (d even), rounded once to the output type
__device__ __forceinline__ void store_pair(void* out, int dt, long long i, float a, float b) {
  if (dt == PDT_F32) *reinterpret_cast<float2*>(static_cast<float*>(out) + i) = make_float2(a, b);
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + i) = dt == PDT_F16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}

// ----------------------------------------------------------------------------------------
// Append.  Token i of sequence b is at position p = start[b] + i; its key and query turn by
// p * theta_j (theta_j = base^(-2j/D), the pair (j, j + D/2)), and the rotated key and the
// value, rounded once to the pool's type, go to row p % page_size of the sequence's page.
//
// CTA = (run, kv head): a run is the tokens of one sequence that fall into one page, so one
// CTA alone owns a page's rows and bounds of its head (no atomics, and the bounds need no
// second pass).  The CTA also rotates the G query heads of its group, which share the angles:
// RC rows' cosines and sines are computed once into shared memory (the angle in turns is
// reduced in double precision, so far positions keep their phase) and used by G + 1 heads.
// Threads 0..127 take the chunk's keys (4 pairs each), threads 128..255 its values, then
// all of them the queries.
// ----------------------------------------------------------------------------------------
constexpr int PAP_THREADS = 256;

struct PagedAppendParams {
  const void *q, *k, *v;            // [T] rows of Hq*D, Hkv*D, Hkv*D elements; q may be NULL
  long long q_stride, k_stride, v_stride;
  int src;                          // PDT_* of q, k, v
  int n_slices;                     // fp32 rows as the sum of split-K slices, slice_stride apart
  long long slice_stride;
  void* q_out;                      // [T, Hq, D] in the pool's type
  const int* start;                 // [B] position of each sequence's first new token
  int start_add;                    // added to every start
  const int* cu_new;                // [B+1] first token row of each sequence, or NULL: one each
  const int* table;
  long long table_stride;
  int width, B, T, G, Hkv, n_pages, ps_log2, rotate;
  void *pk, *pv;                    // the pool; pk NULL: only the queries are rotated
  long long page_stride, head_stride, row_stride;
  void *k_lo, *k_hi;                // [n_pages, Hkv, D], or NULL
  DevStatus* status;
  double turns[64];                 // theta_j / (2 pi)
};

// 4 consecutive source elements as floats
__device__ __forceinline__ void pap_load4(const PagedAppendParams& p, const void* base, long long i, float* f) {
  if (p.src == PDT_F32) {
    const float* s = static_cast<const float*>(base) + i;
    float4 a = *reinterpret_cast<const float4*>(s);
    for (int n = 1; n < p.n_slices; ++n) {
      const float4 c = *reinterpret_cast<const float4*>(s + n * p.slice_stride);
      a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
    }
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    float2 a, b;
    if (p.src == PDT_F16) {
      a = Elem<__half>::unpack(r.x);
      b = Elem<__half>::unpack(r.y);
    } else {
      a = Elem<__nv_bfloat16>::unpack(r.x);
      b = Elem<__nv_bfloat16>::unpack(r.y);
    }
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  }
}

template <typename E>
__device__ __forceinline__ void pap_store4(E* dst, const float* f) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(Elem<E>::pack(f[0], f[1]), Elem<E>::pack(f[2], f[3]));
}

// New tokens of sequence b and its first token row; 0 tokens (and a report) where cu_new does
// not name rows of this call.
__device__ __forceinline__ int pap_count(const PagedAppendParams& p, int b, int* row0) {
  if (p.cu_new == nullptr) {
    *row0 = b;
    return 1;
  }
  const int r0 = p.cu_new[b], r1 = p.cu_new[b + 1];
  *row0 = r0;
  if (r0 < 0 || r1 < r0 || r1 > p.T) {
    report_error(p.status, DEV_ERR_BOUNDS, 611);
    return 0;
  }
  return r1 - r0;
}
// pages the new tokens of sequence b touch
__device__ __forceinline__ int pap_runs(const PagedAppendParams& p, int b) {
  int r0;
  const int n = pap_count(p, b, &r0);
  const int s = p.start[b] + p.start_add;
  if (n == 0) return 0;
  if (s < 0 || s > 0x7fffffff - n) {   // refused whole: neither keys nor queries of this sequence
    report_error(p.status, DEV_ERR_BOUNDS, 612);
    return 0;
  }
  return ((s + n - 1) >> p.ps_log2) - (s >> p.ps_log2) + 1;
}

template <typename E, int D>
__global__ void __launch_bounds__(PAP_THREADS) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr int H2 = D / 2;
  constexpr int RC = 1024 / D;         // rows per chunk: 128 key items of 4 pairs
  constexpr int PARTS = H2 / 4;
  __shared__ float2 cs_tab[RC][H2];
  __shared__ float red[4][2][D];
  __shared__ int wsum[PAP_THREADS / 32];
  __shared__ int pick[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y;

  // 1. this CTA's run: sequence b and its page number within the sequence's new tokens
  int b, run;
  if (p.cu_new == nullptr) {
    b = blockIdx.x;
    run = 0;
    if (pap_runs(p, b) == 0) return;
  } else {
    const int per = (p.B + PAP_THREADS - 1) / PAP_THREADS;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    int mine = 0;
    for (int i = b0; i < b1; ++i) mine += pap_runs(p, i);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) wsum[warp] = inc;
    if (tid == 0) pick[0] = -1;
    __syncthreads();
    int before = inc - mine;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    const int u = blockIdx.x;
    if (u >= before && u < before + mine) {
      int i = b0, left = u - before;
      for (; i < b1; ++i) {
        const int r = pap_runs(p, i);
        if (left < r) break;
        left -= r;
      }
      pick[0] = i;
      pick[1] = left;
    }
    __syncthreads();
    b = pick[0];
    run = pick[1];
    if (b < 0) return;   // past the last run (the grid is sized for the most there can be)
  }
  int row0;
  const int n = pap_count(p, b, &row0);
  const int s0 = p.start[b] + p.start_add;
  const int ps = 1 << p.ps_log2;
  const int page_no = (s0 >> p.ps_log2) + run;            // page index within the sequence
  // (64-bit: the last page of the position range may end at 2^31)
  const int pos0 = run == 0 ? s0 : page_no << p.ps_log2;
  const long long pos1 = min((long long)s0 + n, ((long long)page_no + 1) << p.ps_log2);
  const int rows = (int)(pos1 - pos0);
  const int tok0 = row0 + (pos0 - s0);
  int page = -1;
  if (p.pk != nullptr) {
    if (page_no < p.width) page = p.table[(long long)b * p.table_stride + page_no];
    if (page < 0 || page >= p.n_pages) {   // nowhere to write: reported, queries still rotated
      if (tid == 0) report_error(p.status, DEV_ERR_BOUNDS, 613);
      page = -1;
    }
  }
  E* pk = static_cast<E*>(p.pk) + (page < 0 ? 0 : (long long)page * p.page_stride + g * p.head_stride);
  E* pv = static_cast<E*>(p.pv) + (page < 0 ? 0 : (long long)page * p.page_stride + g * p.head_stride);
  const int in_page = pos0 & (ps - 1);

  float lo[8], hi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo[e] = INFINITY;
    hi[e] = -INFINITY;
  }
  const int item = tid & 127, irow = item / PARTS, part = item % PARTS;
  for (int c0 = 0; c0 < rows; c0 += RC) {
    const int nr = min(RC, rows - c0);
    if (p.rotate) {
      for (int i = tid; i < nr * H2; i += PAP_THREADS) {
        const int r = i / H2, j = i % H2;
        const double t = (double)(pos0 + c0 + r) * p.turns[j];
        float sn, cs;
        sincospif(2.f * (float)(t - rint(t)), &sn, &cs);
        cs_tab[r][j] = make_float2(cs, sn);
      }
      __syncthreads();
    }
    // the pair elements x1 (j..j+3) and x2 (j+H2..) of row r, rotated
    auto rot = [&](int r, int j, float* x1, float* x2) {
      if (!p.rotate) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = cs_tab[r][j + e];
        const float a = x1[e] * t.x - x2[e] * t.y;
        x2[e] = x2[e] * t.x + x1[e] * t.y;
        x1[e] = a;
      }
    };
    auto guard = [&](const float* x1, const float* x2) {
      if constexpr (Elem<E>::IS_F16) {
        f16_range_guard<4>(x1, p.status, 614);
        f16_range_guard<4>(x2, p.status, 614);
      }
    };
    if (page >= 0 && irow < nr) {
      const long long src = (long long)(tok0 + c0 + irow);
      const long long dst = (in_page + c0 + irow) * p.row_stride + part * 4;
      float x1[4], x2[4];
      if (tid < 128) {
        const long long at = src * p.k_stride + g * D + part * 4;
        pap_load4(p, p.k, at, x1);
        pap_load4(p, p.k, at + H2, x2);
        rot(irow, part * 4, x1, x2);
        guard(x1, x2);
        pap_store4<E>(pk + dst, x1);
        pap_store4<E>(pk + dst + H2, x2);
        // rounding keeps the order, so the bounds of the stored keys are the rounded bounds
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = fminf(lo[e], x1[e]);
          hi[e] = fmaxf(hi[e], x1[e]);
          lo[e + 4] = fminf(lo[e + 4], x2[e]);
          hi[e + 4] = fmaxf(hi[e + 4], x2[e]);
        }
      } else {
        const long long at = src * p.v_stride + g * D + part * 4;
        pap_load4(p, p.v, at, x1);
        pap_load4(p, p.v, at + H2, x2);
        guard(x1, x2);
        pap_store4<E>(pv + dst, x1);
        pap_store4<E>(pv + dst + H2, x2);
      }
    }
    if (p.q != nullptr) {
      const int per_head = nr * PARTS;
      for (int i = tid; i < p.G * per_head; i += PAP_THREADS) {
        const int h = g * p.G + i / per_head, r = (i % per_head) / PARTS, j = (i % PARTS) * 4;
        const long long tok = tok0 + c0 + r;
        float x1[4], x2[4];
        const long long at = tok * p.q_stride + h * D + j;
        pap_load4(p, p.q, at, x1);
        pap_load4(p, p.q, at + H2, x2);
        rot(r, j, x1, x2);
        guard(x1, x2);
        E* qo = static_cast<E*>(p.q_out) + (tok * p.Hkv * p.G + h) * D + j;
        pap_store4<E>(qo, x1);
        pap_store4<E>(qo + H2, x2);
      }
    }
    if (p.rotate) __syncthreads();   // the next chunk rewrites the table
  }

  // 2. page bounds: over the run's rows, and over what an earlier call wrote when the run
  //    does not begin the page
  if (p.k_lo != nullptr && page >= 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = PARTS; o < 32; o <<= 1) {
        lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
        hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
      }
    }
    if (tid < 128 && lane < PARTS) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = (e < 4 ? 0 : H2) + lane * 4 + (e & 3);
        red[warp][0][d] = lo[e];
        red[warp][1][d] = hi[e];
      }
    }
    __syncthreads();
    if (tid < D) {
      const long long at = ((long long)page * p.Hkv + g) * D + tid;
      E* blo = static_cast<E*>(p.k_lo) + at;
      E* bhi = static_cast<E*>(p.k_hi) + at;
      float l = fminf(fminf(red[0][0][tid], red[1][0][tid]), fminf(red[2][0][tid], red[3][0][tid]));
      float h = fmaxf(fmaxf(red[0][1][tid], red[1][1][tid]), fmaxf(red[2][1][tid], red[3][1][tid]));
      if (in_page > 0) {
        l = fminf(l, (float)*blo);
        h = fmaxf(h, (float)*bhi);
      }
      *blo = (E)l;
      *bhi = (E)h;
    }
  }
}

// ----------------------------------------------------------------------------------------
// Page selection.  The largest value that q_h . k can take over keys k inside a page's box
// lo <= k <= hi is sum_d max(q_hd lo_d, q_hd hi_d); summed over the G query heads of a group
// it is
//   score(page) = sum_d up_d hi_d + dn_d lo_d,   up_d = sum_h max(q_hd, 0), dn_d = sum_h min(q_hd, 0)
// so a group costs one pair of dot products whatever G is.
//
// Ranks must not depend on rounding, so the scores are held in 64 bits.  A 16-bit value is put
// into a double by moving its bits (sign, exponent and mantissa, the exponent not rebiased):
// that is the value times 2^(bias - 1023) exactly, subnormals included, at two integer
// operations instead of a conversion; up and dn carry the inverse scale up to a factor that is
// the same for every page.  (An infinity reads as the power of two above the largest finite
// value.)
// ----------------------------------------------------------------------------------------
template <typename E>
__device__ __forceinline__ double raw_double(uint32_t h) {   // h: 16 bits
  constexpr int SH = Elem<E>::IS_F16 ? 10 : 13;              // 20 - mantissa bits
  return __hiloint2double((int)(((h & 0x8000u) << 16) | ((h & 0x7fffu) << SH)), 0);
}
template <typename E>
__device__ __forceinline__ double q_scale() {   // 2^1000 or 2^880: |up| stays below 2^1024
  return Elem<E>::IS_F16 ? __hiloint2double((1023 + 1000) << 20, 0) : __hiloint2double((1023 + 880) << 20, 0);
}

struct PagedSelectParams {
  const void *k_lo, *k_hi;   // [n_pages, Hkv, D]
  const void* q;             // [B] rows of Hq*D
  long long q_stride;
  const int* table;
  long long table_stride;
  const int* lens;
  int width, B, Hkv, G, n_pages, ps_log2, n_first, n_last, top;
  unsigned long long* keys;  // [B, Hkv, width] scores in an order-preserving integer form
  int* page_idx;             // [B, Hkv, top]
  DevStatus* status;
};

__device__ __forceinline__ int paged_len(int len, int width, int ps_log2) {
  const long long cap = (long long)width << ps_log2;
  return len < 0 ? 0 : (int)min((long long)len, cap);
}

constexpr int PSC_PAGES = 64;     // pages per warp
constexpr int PSC_THREADS = 128;

template <typename E, int D>
__global__ void __launch_bounds__(PSC_THREADS) paged_score_kernel(const PagedSelectParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr int LPP = D / 8;          // lanes per page: 8 dims each
  constexpr int PPI = 32 / LPP;       // pages per warp and iteration
  const int lane = threadIdx.x & 31;
  const int n_chunks = (p.width + PSC_PAGES - 1) / PSC_PAGES;
  const long long w = (long long)blockIdx.x * (PSC_THREADS / 32) + (threadIdx.x >> 5);
  const int g = (int)(w % p.Hkv), chunk = (int)(w / p.Hkv % n_chunks);
  const long long bl = w / p.Hkv / n_chunks;
  if (bl >= p.B) return;
  const int b = (int)bl;
  const int raw_len = p.lens[b];
  const int len = paged_len(raw_len, p.width, p.ps_log2);
  if (len != raw_len && lane == 0) report_error(p.status, DEV_ERR_BOUNDS, 621);
  const int n = (int)(((long long)len + (1 << p.ps_log2) - 1) >> p.ps_log2);
  const int j0 = chunk * PSC_PAGES, j1 = min(n, j0 + PSC_PAGES);
  if (j0 >= n) return;
  const int d0 = (lane % LPP) * 8, sub = lane / LPP;
  double up[8], dn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) up[e] = dn[e] = 0.0;
  const E* q = static_cast<const E*>(p.q) + b * p.q_stride + (long long)g * p.G * D + d0;
  for (int h = 0; h < p.G; ++h) {
    const uint4 r = *reinterpret_cast<const uint4*>(q + h * D);
    const uint32_t wds[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = Elem<E>::unpack(wds[e / 2]);
      const float x = (e & 1) ? f.y : f.x;
      if (x > 0.f) up[e] += (double)x;
      else dn[e] += (double)x;
    }
  }
  const double qs = q_scale<E>();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    up[e] *= qs;
    dn[e] *= qs;
  }
  unsigned long long* keys = p.keys + ((long long)b * p.Hkv + g) * p.width;
#pragma unroll 2
  for (int j = j0; j < j1; j += PPI) {
    const int jj = j + sub;
    double s = 0.0;
    if (jj < j1) {
      int page = p.table[(long long)b * p.table_stride + jj];
      if (page < 0 || page >= p.n_pages) {   // ranked last; reading it is reported by the attention too
        report_error(p.status, DEV_ERR_BOUNDS, 622);
        s = -__hiloint2double(0x7fe00000, 0);
      } else {
        const long long at = ((long long)page * p.Hkv + g) * D + d0;
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.k_hi) + at);
        const uint4 c = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.k_lo) + at);
        const uint32_t hw[4] = {a.x, a.y, a.z, a.w}, lw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s = fma(up[e], raw_double<E>((hw[e / 2] >> (16 * (e & 1))) & 0xffffu), s);
          s = fma(dn[e], raw_double<E>((lw[e / 2] >> (16 * (e & 1))) & 0xffffu), s);
        }
      }
    }
#pragma unroll
    for (int o = LPP / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (jj < j1 && lane % LPP == 0) {
      const unsigned long long u = (unsigned long long)__double_as_longlong(s + 0.0);   // -0 becomes +0
      keys[jj] = (u >> 63) ? ~u : u | 0x8000000000000000ull;
    }
  }
}

// The top pages of one (sequence, kv head): the first n_first and last n_last are taken, and
// of the rest the largest keys, ties to the lowest index; the list is written in ascending
// order and filled up with -1.  Radix selection from the top digit down, on keys rebased to
// the smallest one so that the first digit already spreads them: `base` and `bits` bound the
// bin that holds the last page taken, `need` counts the pages still to take from it.
constexpr int PPK_THREADS = 512;
template <int THREADS>
__device__ __forceinline__ unsigned long long block_red_u64(unsigned long long v, bool take_max,
                                                            unsigned long long* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
    v = take_max ? max(v, w) : min(v, w);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
  for (int i = 1; i < THREADS / 32; ++i) v = take_max ? max(v, sh[i]) : min(v, sh[i]);
  return v;
}

__global__ void __launch_bounds__(PPK_THREADS) paged_pick_kernel(const PagedSelectParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ unsigned long long ppk_keys[];
  __shared__ unsigned long long red[PPK_THREADS / 32];
  __shared__ int hist[256];
  __shared__ int found[2];
  __shared__ int wsum[PPK_THREADS / 32][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bg = blockIdx.x, b = bg / p.Hkv;
  const int len = paged_len(p.lens[b], p.width, p.ps_log2);
  const int n = (int)(((long long)len + (1 << p.ps_log2) - 1) >> p.ps_log2);
  int* out = p.page_idx + (long long)bg * p.top;
  if (n <= p.top) {   // every page
    for (int i = tid; i < p.top; i += PPK_THREADS) out[i] = i < n ? i : -1;
    return;
  }
  const unsigned long long* keys = p.keys + (long long)bg * p.width;
  // n > top >= n_first + n_last: the forced pages do not overlap
  const int f0 = p.n_first, f1 = n - p.n_last;
  unsigned long long mn = ~0ull, mx = 0;
  for (int i = tid; i < n; i += PPK_THREADS) {
    const unsigned long long k = keys[i];
    ppk_keys[i] = k;
    if (i >= f0 && i < f1) {
      mn = min(mn, k);
      mx = max(mx, k);
    }
  }
  mn = block_red_u64<PPK_THREADS>(mn, false, red);
  mx = block_red_u64<PPK_THREADS>(mx, true, red);
  int need = p.top - p.n_first - p.n_last;
  unsigned long long base = mn;
  int bits = 64 - __clzll((long long)(mx - mn));
  bool whole = need == 0;   // every key >= base is taken (need == 0: none, base above all)
  if (need == 0) base = mx + 1;   // (mx < 2^64 - 1: scores are finite)
  while (!whole && bits > 0) {
    const int shift = max(bits - 8, 0);
    for (int i = tid; i < 256; i += PPK_THREADS) hist[i] = 0;
    __syncthreads();
    for (int i = f0 + tid; i < f1; i += PPK_THREADS) {
      const unsigned long long r = ppk_keys[i] - base;
      if (ppk_keys[i] >= base && (bits == 64 || (r >> bits) == 0)) atomicAdd(&hist[(int)(r >> shift)], 1);
    }
    __syncthreads();
    if (warp == 0) {   // the bin where the count from the top reaches `need`
      int c[8], s = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = hist[255 - (lane * 8 + e)];
        s += c[e];
      }
      int inc = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      int above = inc - s;
      if (above < need && inc >= need) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (above < need && above + c[e] >= need) {
            found[0] = 255 - (lane * 8 + e);
            found[1] = above;
          }
          above += c[e];
        }
      }
    }
    __syncthreads();
    const int d = found[0];
    need -= found[1];
    whole = hist[d] == need;
    base += (unsigned long long)d << shift;
    bits = shift;
    __syncthreads();
  }
  // taken: forced, key above the bin's single value, or (not whole) among the first `need`
  // equal to it
  const int per = (n + PPK_THREADS - 1) / PPK_THREADS;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const unsigned long long k = ppk_keys[i];
    if (i < f0 || i >= f1 || k > base || (whole && k == base)) ++gt;
    else if (k == base) ++eq;
  }
  int ig = gt, ie = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, ig, o), c = __shfl_up_sync(0xffffffffu, ie, o);
    if (lane >= o) {
      ig += a;
      ie += c;
    }
  }
  if (lane == 31) {
    wsum[warp][0] = ig;
    wsum[warp][1] = ie;
  }
  __syncthreads();
  int bg_ = ig - gt, be = ie - eq;
  for (int k = 0; k < warp; ++k) {
    bg_ += wsum[k][0];
    be += wsum[k][1];
  }
  for (int i = i0; i < i1; ++i) {
    const unsigned long long k = ppk_keys[i];
    if (i < f0 || i >= f1 || k > base || (whole && k == base)) {
      out[bg_ + min(be, need)] = i;
      ++bg_;
    } else if (k == base) {
      if (be < need) out[bg_ + be] = i;
      ++be;
    }
  }
}

// ----------------------------------------------------------------------------------------
// Attention of one new token per sequence over its pages ([JJ] eq. (1) for one query row):
//   o = sum_j e_j v_j / sum_j e_j,  e_j = 2^(scale log2(e) q.k_j - m)
// over the visible positions j < lens[b]: all of them, those with j < M or j >= lens[b] - W
// (meta tokens and window), or those of the listed pages.
//
// The keys of (sequence, kv head) are cut into tiles of 64 positions, and the tiles of all of
// them, in order, are dealt to the CTAs as equal contiguous shares: a long sequence is split
// over many CTAs and short ones share one, whatever the lengths are (they are known on the
// device only, and a replayed graph sees new ones).  A (sequence, head) that one CTA covers
// alone is finished there; of one that is cut, each CTA leaves its running maximum, sum and
// weighted values, which paged_attn_join_kernel merges in CTA order.  A CTA has at most two
// such parts: one that an earlier CTA began and one that a later CTA ends.
//
// A producer warp walks the share: its lanes look up the pages and issue one TMA box per page
// piece (128-byte swizzled rows; D = 128 as two 64-wide halves), with the visibility of the
// tile's 64 positions as a bit mask beside it; a page that does not exist gets an
// out-of-range coordinate, which TMA fills with zeros.  Four consumer warps take 16 positions
// of every tile each.  The group's query heads are rows of 16 x 16 x 8 tensor-core products:
// rows 0..7 hold up to 8 heads, and rows 8..15, otherwise empty, take in the second product
// the rounding error of the probabilities (p = hi + lo, both 16 bits), so P V costs the same
// number of instructions and keeps about twice the mantissa.  With 9 to 16 heads (NHB = 2)
// rows 8..15 of Q K^T are heads 8..15, and P V runs once per 8 heads.
// ----------------------------------------------------------------------------------------
constexpr int PA_KT = 64;
constexpr int PA_CONSUMERS = 128;
constexpr int PA_THREADS = PA_CONSUMERS + 32;
constexpr int PA_MAX_GRID = 148 * 3;   // CTAs of any variant (sizes the workspace)

template <int D, int NHB>
struct PaShape {
  static constexpr int STAGES = D == 64 ? 3 : (NHB == 1 ? 3 : 5);
  static constexpr int PER_SM = NHB == 1 ? (D == 64 ? 3 : 2) : (D == 64 ? 2 : 1);
  static constexpr int HALF = PA_KT * 128;                 // bytes of 64 positions x 64 dims
  static constexpr int STAGE = 2 * (D / 64) * HALF;        // K then V
  static constexpr int QB = 8 * NHB * D * 2;
  static constexpr int SMEM = STAGES * STAGE + 1024;
};

struct PagedAttnParams {
  const void* q;
  long long q_stride;
  void* out;
  int out_dt;
  long long out_stride;
  float* lse;                 // [B, Hq] natural log of the softmax's denominator, or NULL
  const int* table;
  long long table_stride;
  const int* lens;
  int len_add;                // added to every length
  const int* page_idx;        // [B, Hkv, top] page numbers within the sequence, or NULL
  int top, width, B, Hq, Hkv, G, n_pages, ps_log2, M, W;
  int dim_row, dim_head;      // tensor-map dimensions (1..3) of rows and heads; pages have the other
  float scale_log2;
  float* part;                // [grid][2][G][D + 2]
  int2* desc;                 // [grid]: (item, parts) of the cut item that this CTA begins
  DevStatus* status;
};

struct PaTiles {
  int len;      // positions of the sequence
  int n_tiles;  // at least 1
  int head;     // window: the first tiles (meta); tile t >= head stands for tile t + skip
  int skip;
};
__device__ __forceinline__ PaTiles pa_tiles(const PagedAttnParams& p, int raw_len) {
  PaTiles r;
  r.len = paged_len(raw_len, p.width, p.ps_log2);
  const int all = (int)(((long long)r.len + PA_KT - 1) / PA_KT);
  r.head = all;
  r.skip = 0;
  r.n_tiles = all;
  if (p.page_idx != nullptr) {
    const int pages = (int)(((long long)r.len + (1 << p.ps_log2) - 1) >> p.ps_log2);
    r.n_tiles = (int)((((long long)min(pages, p.top) << p.ps_log2) + PA_KT - 1) / PA_KT);
  } else if (p.W > 0) {
    const int w0 = max(0, r.len - p.W) / PA_KT;           // the window's first tile
    r.head = min(w0, (p.M + PA_KT - 1) / PA_KT);
    r.skip = w0 - r.head;
    r.n_tiles = all - r.skip;
  }
  if (r.n_tiles < 1) r.n_tiles = 1;                       // an empty sequence: one tile without keys
  return r;
}
__device__ __forceinline__ int pa_len(const PagedAttnParams& p, int b) {
  const int l = p.lens[b];
  return l > 0x7fffffff - p.len_add ? l : l + p.len_add;
}
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
}

struct PaMeta {
  unsigned long long mask;   // visible positions of the tile
  int item;                  // sequence * Hkv + kv head
  int flags;                 // PA_FIRST, PA_LAST of the item's tiles in this CTA, PA_WHOLE, part slot
};
enum { PA_FIRST = 1, PA_LAST = 2, PA_WHOLE = 4, PA_SLOT1 = 8 };

template <typename E, int D, int NHB>
__global__ void __launch_bounds__(PA_THREADS, PaShape<D, NHB>::PER_SM)
    paged_attn_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                      const __grid_constant__ PagedAttnParams p) {
  using S = PaShape<D, NHB>;
  constexpr int STAGES = S::STAGES;
  constexpr int NH = D / 64;
  extern __shared__ uint8_t pa_smem_raw[];
  uint8_t* ring = align_smem<1024>(pa_smem_raw);
  __shared__ uint64_t full[STAGES], empty[STAGES], merge_bar;
  __shared__ __align__(16) PaMeta meta[STAGES];
  __shared__ __align__(128) uint8_t qbuf[STAGES][S::QB];
  __shared__ __align__(16) float mo[2][8][D + 4];   // pairwise merge of the warps (padded rows)
  __shared__ float mm[2][8], ml[2][8];
  __shared__ long long wsum[PA_THREADS / 32];
  __shared__ long long start_at;                     // tile offset of the share inside sequence start_b
  __shared__ int start_b, abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], PA_CONSUMERS / 32);
    }
    mbar_init(&merge_bar, PA_CONSUMERS / 32);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
  }
  pdl_wait();
  pdl_trigger();

  // 1. this CTA's share of the tiles, and the sequence it starts in
  const int per = (p.B + PA_THREADS - 1) / PA_THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int i = b0; i < b1; ++i) {
    const int l = pa_len(p, i);
    const PaTiles t = pa_tiles(p, l);
    if (t.len != l && blockIdx.x == 0) report_error(p.status, DEV_ERR_BOUNDS, 601);
    mine += t.n_tiles;
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  long long before = inc - mine, total = 0;
  for (int w = 0; w < PA_THREADS / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  total *= p.Hkv;
  const long long n_cta = min((long long)gridDim.x, total);
  if (blockIdx.x >= n_cta) {
    if (tid == 0) p.desc[blockIdx.x] = make_int2(0, 0);
    return;
  }
  const long long t0 = blockIdx.x * total / n_cta, t1 = (blockIdx.x + 1) * total / n_cta;
  if (t0 >= before * p.Hkv && t0 < (before + mine) * p.Hkv) {
    long long left = t0 - before * p.Hkv;
    int i = b0;
    for (; i < b1; ++i) {
      const long long c = (long long)pa_tiles(p, pa_len(p, i)).n_tiles * p.Hkv;
      if (left < c) break;
      left -= c;
    }
    start_b = i;
    start_at = left;
  }
  __syncthreads();
  const long long n_mine = t1 - t0;

  if (warp == PA_CONSUMERS / 32) {
    // ------------------------------ producer warp ------------------------------
    const int ps = 1 << p.ps_log2;
    const int R = min(ps, PA_KT), n_chunk = PA_KT / R;    // a tile's page pieces
    int b = start_b;
    PaTiles sq = pa_tiles(p, pa_len(p, b));
    int g = (int)(start_at / sq.n_tiles), t = (int)(start_at % sq.n_tiles);
    int next_len = b + 1 < p.B ? pa_len(p, b + 1) : 0;
    int2 desc = make_int2(0, 0);
    bool ok = true;
    // one tile's page piece of this lane: pool page (out of range where there is nothing to
    // read), first row in the page, and the visible rows as bits
    struct Piece {
      int page, row;
      unsigned long long bits;
    };
    auto look = [&]() {
      Piece r;
      r.page = p.n_pages;
      r.row = 0;
      r.bits = 0;
      if (lane < n_chunk) {
        const int key = t * PA_KT + lane * R;             // < 2^31: tiles of at most len + 63 positions
        int logical, pos;
        bool in = true;
        if (p.page_idx != nullptr) {
          const int e = key >> p.ps_log2;
          const int pages = (int)(((long long)sq.len + ps - 1) >> p.ps_log2);
          logical = e < min(pages, p.top) ? p.page_idx[((long long)b * p.Hkv + g) * p.top + e] : -1;
          in = logical >= 0 && logical < pages;
          pos = in ? (logical << p.ps_log2) + (key & (ps - 1)) : 0;
        } else {
          pos = (t < sq.head ? key : key + sq.skip * PA_KT);
          logical = pos >> p.ps_log2;
        }
        r.row = pos & (ps - 1);
        if (in && pos < sq.len) {
          r.bits = low_bits(min(R, sq.len - pos));
          if (p.W > 0) r.bits &= low_bits(p.M - pos) | ~low_bits((sq.len - pos) - p.W);
          if (r.bits != 0) {
            const int page = p.table[(long long)b * p.table_stride + logical];
            if (page >= 0 && page < p.n_pages) {
              r.page = page;
            } else {
              report_error(p.status, DEV_ERR_BOUNDS, 602);
              r.bits = 0;
            }
          }
        }
      }
      return r;
    };
    Piece cur = look();
    int seg_first = 1;
    long long i = 0;
    for (; i < n_mine; ++i) {
      const int stg = (int)(i % STAGES);
      // this tile's place in its item
      const int item = b * p.Hkv + g;
      const bool first = seg_first, last = i + 1 == n_mine || t + 1 == sq.n_tiles;
      int flags = (first ? PA_FIRST : 0) | (last ? PA_LAST : 0);
      if (first && t == 0) {
        const long long end = t0 + i + sq.n_tiles;         // the item's end in the order of all tiles
        if (end > t1) desc = make_int2(item, (int)((end * n_cta - 1) / total) - (int)blockIdx.x + 1);
      }
      // PA_WHOLE / PA_SLOT1 matter on the last tile: begun here at tile 0?
      const long long seg_len_before = t;                  // tiles of the item before this one
      const bool begun_here = seg_len_before <= i;         // its tile 0 is in this share
      if (begun_here && t + 1 == sq.n_tiles) flags |= PA_WHOLE;
      if (begun_here) flags |= PA_SLOT1;
      const int cb = b, cg = g;
      // step to the next tile and start its look-up before waiting for a free stage
      seg_first = 0;
      if (++t == sq.n_tiles) {
        t = 0;
        seg_first = 1;
        if (++g == p.Hkv) {
          g = 0;
          ++b;
          sq = pa_tiles(p, next_len);
          next_len = b + 1 < p.B ? pa_len(p, b + 1) : 0;
        }
      }
      Piece nxt;
      nxt.page = p.n_pages;
      nxt.row = 0;
      nxt.bits = 0;
      if (i + 1 < n_mine) nxt = look();
      if (i >= STAGES) {
        ok = mbar_wait(&empty[stg], (uint32_t)(i / STAGES - 1) & 1u, &abort_flag, p.status, 603);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      unsigned long long mask = cur.bits << (lane < n_chunk ? lane * R : 0);
      mask |= __shfl_xor_sync(0xffffffffu, mask, 1);
      mask |= __shfl_xor_sync(0xffffffffu, mask, 2);
      uint8_t* kt = ring + stg * S::STAGE;
      if (lane == 0) {
        meta[stg].mask = mask;
        meta[stg].item = item;
        meta[stg].flags = flags;
        const uint32_t q_bytes = first ? (uint32_t)(p.G * D * 2) : 0u;
        mbar_arrive_expect_tx(&full[stg], S::STAGE + q_bytes);
        if (first)
          bulk_load(qbuf[stg], static_cast<const E*>(p.q) + cb * p.q_stride + (long long)cg * p.G * D, q_bytes,
                    &full[stg]);
      }
      __syncwarp();
      if (lane < n_chunk) {
        auto coord = [&](int dim) { return p.dim_row == dim ? cur.row : (p.dim_head == dim ? cg : cur.page); };
        const int c1 = coord(1), c2 = coord(2), c3 = coord(3);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          tma_load_4d(kt + h * S::HALF + lane * R * 128, &mapK, &full[stg], h * 64, c1, c2, c3);
          tma_load_4d(kt + (NH + h) * S::HALF + lane * R * 128, &mapV, &full[stg], h * 64, c1, c2, c3);
        }
      }
      cur = nxt;
    }
    if (lane == 0) {
      p.desc[blockIdx.x] = desc;
      // loads still in flight (all of them, if the consumers gave up) land before the CTA exits
      for (long long j = i > STAGES ? i - STAGES : 0; j < i; ++j)
        mbar_wait(&full[j % STAGES], (uint32_t)(j / STAGES) & 1u, nullptr, p.status, 604);
    }
    return;
  }

  // ------------------------------ consumer warps ------------------------------
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t ring_u32 = smem_u32(ring);
  const int k_row = warp * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, k_chk = (lane >> 3) & 1;
  const int v_row = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, v_chk = (lane >> 4) & 1;
  uint32_t qa[D / 16][2 * NHB];
  float m_run[NHB], l_run[NHB], o[NHB][D / 8][4];
  uint32_t merge_phase = 0;
  bool ok = true;
  auto merge_sync = [&]() {   // the four consumer warps; bounded, so that a warp that gave up holds no one
    __syncwarp();
    if (lane == 0) mbar_arrive(&merge_bar);
    const bool r = mbar_wait(&merge_bar, merge_phase & 1u, &abort_flag, p.status, 605);
    ++merge_phase;
    return __all_sync(0xffffffffu, r) != 0;
  };
  for (long long i = 0; i < n_mine && ok; ++i) {
    const int stg = (int)(i % STAGES);
    ok = mbar_wait(&full[stg], (uint32_t)(i / STAGES) & 1u, &abort_flag, p.status, 606);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const unsigned long long mask = meta[stg].mask;
    const int item = meta[stg].item, flags = meta[stg].flags;
    if (flags & PA_FIRST) {
      const E* q = reinterpret_cast<const E*>(qbuf[stg]);
#pragma unroll
      for (int hb = 0; hb < NHB; ++hb) {
        m_run[hb] = -INFINITY;
        l_run[hb] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[hb][j][0] = o[hb][j][1] = o[hb][j][2] = o[hb][j][3] = 0.f;
        const bool row = hb * 8 + gq < p.G;
        const E* qr = q + (hb * 8 + gq) * D + 2 * tq;
#pragma unroll
        for (int st = 0; st < D / 16; ++st) {
          qa[st][2 * hb] = row ? *reinterpret_cast<const uint32_t*>(qr + st * 16) : 0u;
          qa[st][2 * hb + 1] = row ? *reinterpret_cast<const uint32_t*>(qr + st * 16 + 8) : 0u;
        }
      }
    }
    const uint32_t m16 = (uint32_t)(mask >> (warp * 16)) & 0xffffu;
    if (m16 != 0) {
      const uint32_t kt = ring_u32 + stg * S::STAGE, vt = kt + NH * S::HALF;
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int st = 0; st < D / 16; ++st) {
        uint32_t f0, f1, f2, f3;
        ldsm_x4(sw128_addr(kt + (st / 4) * S::HALF, k_row, 2 * (st & 3) + k_chk), f0, f1, f2, f3);
        const uint32_t a1 = NHB == 2 ? qa[st][2 * NHB - 2] : 0u, a3 = NHB == 2 ? qa[st][2 * NHB - 1] : 0u;
        Elem<E>::mma(s0, qa[st][0], a1, qa[st][1], a3, f0, f1);
        Elem<E>::mma(s1, qa[st][0], a1, qa[st][1], a3, f2, f3);
      }
      // this lane's positions: 2tq, 2tq + 1, 2tq + 8, 2tq + 9 of the warp's 16
      const uint32_t mb = m16 >> (2 * tq);
      const bool vis[4] = {(mb & 1u) != 0, (mb & 2u) != 0, (mb & 0x100u) != 0, (mb & 0x200u) != 0};
      uint32_t pa[NHB][4];
#pragma unroll
      for (int hb = 0; hb < NHB; ++hb) {
        float v[4] = {s0[2 * hb] * p.scale_log2, s0[2 * hb + 1] * p.scale_log2, s1[2 * hb] * p.scale_log2,
                      s1[2 * hb + 1] * p.scale_log2};
        if (m16 != 0xffffu) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = vis[e] ? v[e] : -INFINITY;
        }
        float tm = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
        const float m_new = fmaxf(m_run[hb], tm);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;   // every score so far is -inf
        const float al = ex2_approx(m_run[hb] - m_use);
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = ex2_approx(v[k] - m_use);
        m_run[hb] = m_new;
        l_run[hb] = l_run[hb] * al + ((e[0] + e[1]) + (e[2] + e[3]));
        if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[hb][j][0] *= al; o[hb][j][1] *= al; o[hb][j][2] *= al; o[hb][j][3] *= al;
          }
        }
        pa[hb][0] = Elem<E>::pack(e[0], e[1]);
        pa[hb][2] = Elem<E>::pack(e[2], e[3]);
        const float2 h0 = Elem<E>::unpack(pa[hb][0]), h2 = Elem<E>::unpack(pa[hb][2]);
        pa[hb][1] = Elem<E>::pack(e[0] - h0.x, e[1] - h0.y);
        pa[hb][3] = Elem<E>::pack(e[2] - h2.x, e[3] - h2.y);
      }
      // a hidden position's probability is 0, but its value may be anything (0 * NaN): its
      // fragment halves are cleared
      const uint32_t vm0 = (vis[0] ? 0xffffu : 0u) | (vis[1] ? 0xffff0000u : 0u);
      const uint32_t vm1 = (vis[2] ? 0xffffu : 0u) | (vis[3] ? 0xffff0000u : 0u);
#pragma unroll
      for (int j = 0; j < D / 8; j += 2) {
        uint32_t f0, f1, f2, f3;
        ldsm_x4_t(sw128_addr(vt + (j / 8) * S::HALF, v_row, (j & 7) + v_chk), f0, f1, f2, f3);
        if (m16 != 0xffffu) {
          f0 &= vm0; f1 &= vm1; f2 &= vm0; f3 &= vm1;
        }
#pragma unroll
        for (int hb = 0; hb < NHB; ++hb) {
          Elem<E>::mma(o[hb][j], pa[hb][0], pa[hb][1], pa[hb][2], pa[hb][3], f0, f1);
          Elem<E>::mma(o[hb][j + 1], pa[hb][0], pa[hb][1], pa[hb][2], pa[hb][3], f2, f3);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stg]);   // this warp is done with the stage
    if (!(flags & PA_LAST)) continue;

    // the item's tiles in this CTA are done: merge the four warps (2 and 3 into 0 and 1, then
    // 1 into 0), warp 0 writes
    const int b = item / p.Hkv, g = item % p.Hkv;
#pragma unroll
    for (int hb = 0; hb < NHB; ++hb) {
      float m = m_run[hb], l = l_run[hb];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      float acc[D / 8][2];
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        acc[j][0] = o[hb][j][0] + o[hb][j][2];
        acc[j][1] = o[hb][j][1] + o[hb][j][3];
      }
      auto put = [&](int slot) {
        if (tq == 0) {
          mm[slot][gq] = m;
          ml[slot][gq] = l;
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<float2*>(&mo[slot][gq][8 * j + 2 * tq]) = make_float2(acc[j][0], acc[j][1]);
      };
      auto take = [&](int slot) {
        const float m2 = mm[slot][gq], l2 = ml[slot][gq];
        const float mn = fmaxf(m, m2), mu = mn == -INFINITY ? 0.f : mn;
        const float wa = ex2_approx(m - mu), wb = ex2_approx(m2 - mu);
        m = mn;
        l = l * wa + l2 * wb;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const float2 x = *reinterpret_cast<const float2*>(&mo[slot][gq][8 * j + 2 * tq]);
          acc[j][0] = acc[j][0] * wa + x.x * wb;
          acc[j][1] = acc[j][1] * wa + x.y * wb;
        }
      };
      if (warp >= 2) put(warp - 2);
      if (ok) ok = merge_sync();
      if (!ok) break;
      if (warp < 2) take(warp);
      if (warp == 1) put(1);       // slot 1 was warp 1's own to read
      ok = merge_sync();
      if (!ok) break;
      if (warp == 0) take(1);
      ok = merge_sync();           // the slots are free again
      if (!ok) break;
      const int hh = hb * 8 + gq;  // query head within the group
      if (warp == 0 && hh < p.G) {
        if (flags & PA_WHOLE) {
          const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // no key: zeros; NaN stays
          const long long at = b * p.out_stride + (long long)(g * p.G + hh) * D + 2 * tq;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) store_pair(p.out, p.out_dt, at + 8 * j, acc[j][0] * inv, acc[j][1] * inv);
          if (p.lse != nullptr && tq == 0)
            p.lse[(long long)b * p.Hq + g * p.G + hh] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
        } else {
          float* dst = p.part + (((long long)blockIdx.x * 2 + ((flags & PA_SLOT1) ? 1 : 0)) * p.G + hh) * (D + 2);
          if (tq == 0) *reinterpret_cast<float2*>(dst) = make_float2(m, l);
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(dst + 2 + 8 * j + 2 * tq) = make_float2(acc[j][0], acc[j][1]);
        }
      }
    }
  }
}

// Join of an item that was cut: CTA x of the grid's first dimension stands for the attention
// CTA that began the item, y for the query head.  The parts are its slot 1 and the slot 0 of
// the CTAs after it; o = sum_i w_i o_i / sum_i w_i l_i, w_i = 2^(m_i - max m), added up by PJ
// fixed interleaved groups of threads and then in group order, so the result does not depend
// on scheduling.
constexpr int PJ_THREADS = 256;
template <int D>
__global__ void __launch_bounds__(PJ_THREADS) paged_attn_join_kernel(const PagedAttnParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr int GROUPS = PJ_THREADS / D;
  __shared__ float so[GROUPS][D], sl[GROUPS], sm[PJ_THREADS / 32];
  const int2 desc = p.desc[blockIdx.x];
  const int n = desc.y;
  if (n == 0) return;
  const int tid = threadIdx.x, hh = blockIdx.y;
  const long long pstride = 2LL * p.G * (D + 2);
  const float* first = p.part + (((long long)blockIdx.x * 2 + 1) * p.G + hh) * (D + 2);
  const float* rest = p.part + ((long long)blockIdx.x * 2 * p.G + hh) * (D + 2);   // + i * pstride, i >= 1
  auto src = [&](int i) { return i == 0 ? first : rest + i * pstride; };
  float m = -INFINITY;
  for (int i = tid; i < n; i += PJ_THREADS) m = fmaxf(m, src(i)[0]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) sm[tid >> 5] = m;
  __syncthreads();
  for (int w = 0; w < PJ_THREADS / 32; ++w) m = fmaxf(m, sm[w]);
  const float mu = m == -INFINITY ? 0.f : m;
  const int grp = tid / D, d = tid % D;
  float O = 0.f, L = 0.f;
#pragma unroll 8
  for (int i = grp; i < n; i += GROUPS) {
    const float* s = src(i);
    const float w = ex2_approx(s[0] - mu);
    L += w * s[1];
    O += w * s[2 + d];
  }
  so[grp][d] = O;
  if (d == 0) sl[grp] = L;
  __syncthreads();
  if (tid < D / 2) {
    float a = 0.f, c = 0.f, l = 0.f;
    for (int k = 0; k < GROUPS; ++k) {
      a += so[k][2 * tid];
      c += so[k][2 * tid + 1];
      l += sl[k];
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int b = desc.x / p.Hkv, h = desc.x % p.Hkv * p.G + hh;
    store_pair(p.out, p.out_dt, b * p.out_stride + (long long)h * D + 2 * tid, a * inv, c * inv);
    if (p.lse != nullptr && tid == 0)
      p.lse[(long long)b * p.Hq + h] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
  }
}

}  // namespace hymba
