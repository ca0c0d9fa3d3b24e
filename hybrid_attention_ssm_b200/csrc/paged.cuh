// The paged key-value cache: appending new tokens (with RoPE on the way), choosing the pages a
// decode query reads, and attention of one new token per sequence over its pages.
//
// A pool holds n_pages pages of page_size positions: K and V [page, kv head, row, D] through
// three strides, 16-bit.  A block table row lists a sequence's pages in order, so position p
// of sequence b is row p % page_size of page table[b][p / page_size].  Optional page bounds
// keep the smallest and largest key value per channel, [page, kv head, D].
#pragma once
#include <type_traits>

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
  __device__ static uint32_t min2(uint32_t a, uint32_t b) {
    const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static constexpr uint32_t INF2 = 0x7c007c00u;
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
  __device__ static uint32_t min2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static constexpr uint32_t INF2 = 0x7f807f80u;
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
// A thread owns some pairs of a token: it computes their angles once and applies them to the
// key and to the query heads of its kv head; the value is copied.  Angles are phases in units
// of 2^-64 turns, pos * turn_j modulo 2^64 in integers, so far positions keep theirs.
//
// One token per sequence (paged_append_step_kernel): thread = (sequence, kv head, 4 pairs), and
// each page's bounds are widened by the thread that owns the channels.
//
// Several (paged_append_kernel): persistent CTAs, three per SM, take the items (run, kv head) in
// turn, a run being the tokens of one sequence that fall into one page: one CTA alone owns a
// page's rows and bounds of a head, so there are no atomics and no second pass, and the heads
// of a run, whose rows are neighbours in memory, are under way at the same time (equal
// contiguous shares instead: 61 against 57 us at 4 x 8320 tokens).  A producer warp streams the
// items' rows through a ring by TMA, 8 tokens to a box, so the bytes in flight cost neither
// registers nor instructions; eight consumer warps take a stage's rows, 4 pairs of a row per
// thread.
//
// Bound by its bytes: 4 x 8320 tokens of 25 + 5 + 5 heads of 64 move 298 MB in 59 us, 5.0 TB/s
// where a plain copy reaches 6.55 (45 us); ncu reads 57% of DRAM and half of the issue slots,
// the rest is ramp and the mix of reads and writes.  Before the rows came by TMA (loads into
// registers, a CTA per run) it took 140 us, then 64 with 4 pairs per thread in flight.  One
// token for each of 64 sequences takes 6 us on the device, all of it latency.
// ----------------------------------------------------------------------------------------
constexpr int PAP_STEP_THREADS = 64;
constexpr int PAP_CONSUMERS = 256;
constexpr int PAP_THREADS = PAP_CONSUMERS + 32;
constexpr int PAP_PER_SM = 3;
constexpr int PAP_BOX = 8;                 // tokens per TMA box
constexpr int PAP_STAGES = 2;
constexpr int PAP_STAGE_BYTES = 32768;     // (one box of the widest group needs more)
constexpr int PAP_SMEM_MAX = PAP_STAGES * PAP_BOX * (16 + 2) * 128 * 4;

struct PagedAppendParams {
  const void *q, *k, *v;            // [T] rows of Hq*D, Hkv*D, Hkv*D elements; q may be NULL
  long long q_stride, k_stride, v_stride;
  int src;                          // PDT_* of q, k, v
  int n_slices;                     // fp32 rows as the sum of split-K slices, slice_stride apart
  long long slice_stride;
  void* q_out;                      // [T, Hq, D] in the pool's type
  const int* start;                 // [B] position of each sequence's first new token
  const int* cu_new;                // [B+1] first token row of each sequence, or NULL: one each
  const int* table;
  long long table_stride;
  int width, B, T, G, Hkv, n_pages, ps_log2, rotate;
  int chunk;                        // several tokens: rows of a stage
  void *pk, *pv;                    // the pool; pk NULL: only the queries are rotated
  long long page_stride, head_stride, row_stride;
  void *k_lo, *k_hi;                // [n_pages, Hkv, D], or NULL
  unsigned* clear;                  // n_clear words that the step kernel zeroes (the counters of an
  int n_clear;                      // attention that follows in the same call: it then needs no
                                    // initialised workspace), or NULL
  DevStatus* status;
  unsigned long long turns[64];     // theta_j / (2 pi) in units of 2^-64
};

// 4 consecutive source elements, as they are loaded; as two packed fp32 pairs, and rounded
template <int SRC>
struct PapRaw {
  using T = typename std::conditional<SRC == PDT_F16, __half, __nv_bfloat16>::type;
  uint2 r;
  __device__ void load(const PagedAppendParams&, const void* base, long long i) {
    r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
  }
  __device__ void get(uint64_t* f) const {
    const float2 a = Elem<T>::unpack(r.x), b = Elem<T>::unpack(r.y);
    f[0] = f2_pack(a.x, a.y);
    f[1] = f2_pack(b.x, b.y);
  }
};
template <>
struct PapRaw<PDT_F32> {
  using T = float;
  float4 r;
  __device__ void load(const PagedAppendParams& p, const void* base, long long i) {
    const float* s = static_cast<const float*>(base) + i;
    r = *reinterpret_cast<const float4*>(s);
    for (int n = 1; n < p.n_slices; ++n) {   // split-K slices, in order
      const float4 c = *reinterpret_cast<const float4*>(s + n * p.slice_stride);
      r.x += c.x; r.y += c.y; r.z += c.z; r.w += c.w;
    }
  }
  __device__ void get(uint64_t* f) const {
    f[0] = f2_pack(r.x, r.y);
    f[1] = f2_pack(r.z, r.w);
  }
};
// Rounded to the pool's type.  big: the largest magnitudes stored so far (fp16 pools).
template <typename E>
__device__ __forceinline__ void pap_keep(const uint2& a, uint32_t& big) {
  if constexpr (Elem<E>::IS_F16) big = Elem<E>::max2(big, Elem<E>::max2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu));
}
template <typename E>
__device__ __forceinline__ uint2 pap_round(const uint64_t* f, uint32_t& big) {
  const uint2 a = make_uint2(Elem<E>::pack(f2_lo(f[0]), f2_hi(f[0])), Elem<E>::pack(f2_lo(f[1]), f2_hi(f[1])));
  pap_keep<E>(a, big);
  return a;
}

// cos and sin of the 4 pairs from j0 on at a position, as packed fp32 pairs.  The phase's
// nearest quarter turn is split off in integers; the rest, at most 1/8 turn, goes into the
// Taylor polynomials of sin(2 pi r) and cos(2 pi r) (remainders below 2e-9 and 2e-10).
struct PapTurn {
  uint64_t cs[2], sn[2], neg[2];   // neg = -sn
  __device__ __forceinline__ void at(const PagedAppendParams& p, int pos, int j0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t quarter[2];
      float r[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t ph = (uint32_t)(((unsigned long long)(uint32_t)pos * p.turns[j0 + 2 * e + k]) >> 32);
        quarter[k] = (ph + 0x20000000u) >> 30;
        r[k] = (float)(int)(ph - (quarter[k] << 30)) * 0x1p-32f;
      }
      const uint64_t x = f2_pack(r[0], r[1]), x2 = f2_mul(x, x);
      auto c2 = [](float v) { return f2_pack(v, v); };
      uint64_t s = f2_fma(x2, c2(42.058693944897655f), c2(-76.70585975306136f));
      s = f2_fma(s, x2, c2(81.60524927607504f));
      s = f2_fma(s, x2, c2(-41.34170224039976f));
      s = f2_mul(f2_fma(s, x2, c2(6.283185307179586f)), x);
      uint64_t c = f2_fma(x2, c2(-26.426256783374388f), c2(60.244641371876656f));
      c = f2_fma(c, x2, c2(-85.45681720669373f));
      c = f2_fma(c, x2, c2(64.93939402266829f));
      c = f2_fma(c, x2, c2(-19.739208802178716f));
      c = f2_fma(c, x2, c2(1.f));
      float sv[2] = {f2_lo(s), f2_hi(s)}, cv[2] = {f2_lo(c), f2_hi(c)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {   // sin and cos of r + quarter / 4
        const float a = (quarter[k] & 1u) ? cv[k] : sv[k], b = (quarter[k] & 1u) ? sv[k] : cv[k];
        sv[k] = __uint_as_float(__float_as_uint(a) ^ ((quarter[k] & 2u) << 30));
        cv[k] = __uint_as_float(__float_as_uint(b) ^ (((quarter[k] + 1u) & 2u) << 30));
      }
      cs[e] = f2_pack(cv[0], cv[1]);
      sn[e] = f2_pack(sv[0], sv[1]);
      neg[e] = f2_pack(-sv[0], -sv[1]);
    }
  }
  // (a, b) of pair 2e and 2e + 1 turned
  __device__ __forceinline__ void apply(int e, uint64_t& a, uint64_t& b) const {
    const uint64_t x = f2_fma(b, neg[e], f2_mul(a, cs[e]));
    b = f2_fma(a, sn[e], f2_mul(b, cs[e]));
    a = x;
  }
};

// One token and kv head of a thread: the key and value into the pool's row (element offset,
// head included; -1: no place), the group's query heads into q_out.  k returns the stored key
// (low and high channels), big the largest magnitudes rounded so far.
template <typename E, int D, int SRC>
__device__ __forceinline__ void pap_token(const PagedAppendParams& p, const PapTurn& turn, long long tok,
                                          long long row, int g, int part, uint2* k, uint32_t& big) {
  constexpr int H2 = D / 2, QB = 4;   // query heads whose loads are in flight together
  PapRaw<SRC> kr[2], vr[2], qr[QB][2];
  if (row >= 0) {
    const long long ka = tok * p.k_stride + g * D + part * 4, va = tok * p.v_stride + g * D + part * 4;
    kr[0].load(p, p.k, ka);
    kr[1].load(p, p.k, ka + H2);
    vr[0].load(p, p.v, va);
    vr[1].load(p, p.v, va + H2);
  }
  const long long qa = tok * p.q_stride + g * p.G * D + part * 4;
  auto load_q = [&](int h0) {
#pragma unroll
    for (int h = 0; h < QB; ++h) {
      if (h0 + h < p.G) {
        qr[h][0].load(p, p.q, qa + (h0 + h) * D);
        qr[h][1].load(p, p.q, qa + (h0 + h) * D + H2);
      }
    }
  };
  if (p.q != nullptr) load_q(0);
  auto rotate = [&](const PapRaw<SRC>* raw, uint2* out) {
    uint64_t a[2], b[2];
    raw[0].get(a);
    raw[1].get(b);
    if (p.rotate) {
#pragma unroll
      for (int e = 0; e < 2; ++e) turn.apply(e, a[e], b[e]);
    }
    out[0] = pap_round<E>(a, big);
    out[1] = pap_round<E>(b, big);
  };
  if (row >= 0) {
    E* pv = static_cast<E*>(p.pv) + row + part * 4;
    if constexpr (std::is_same<typename PapRaw<SRC>::T, E>::value) {   // no rounding: the bits as they are
      *reinterpret_cast<uint2*>(pv) = vr[0].r;
      *reinterpret_cast<uint2*>(pv + H2) = vr[1].r;
      pap_keep<E>(vr[0].r, big);
      pap_keep<E>(vr[1].r, big);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint64_t f[2];
        vr[e].get(f);
        *reinterpret_cast<uint2*>(pv + e * H2) = pap_round<E>(f, big);
      }
    }
    rotate(kr, k);
    E* pk = static_cast<E*>(p.pk) + row + part * 4;
    *reinterpret_cast<uint2*>(pk) = k[0];
    *reinterpret_cast<uint2*>(pk + H2) = k[1];
  }
  if (p.q == nullptr) return;
  E* qo = static_cast<E*>(p.q_out) + (tok * p.Hkv + g) * p.G * D + part * 4;
  for (int h0 = 0;;) {
#pragma unroll
    for (int h = 0; h < QB; ++h) {
      if (h0 + h < p.G) {
        uint2 y[2];
        rotate(qr[h], y);
        *reinterpret_cast<uint2*>(qo + (h0 + h) * D) = y[0];
        *reinterpret_cast<uint2*>(qo + (h0 + h) * D + H2) = y[1];
      }
    }
    h0 += QB;
    if (h0 >= p.G) break;
    load_q(h0);
  }
}
// Values that rounded to an infinity: |v| >= 65520 in an fp16 pool.
template <typename E>
__device__ __forceinline__ void pap_report(const PagedAppendParams& p, uint32_t big) {
  if constexpr (Elem<E>::IS_F16)
    if ((big & 0xffffu) == (Elem<E>::INF2 & 0xffffu) || (big >> 16) == (Elem<E>::INF2 >> 16))
      report_error(p.status, DEV_ERR_FP16_RANGE, 614);
}

// The page of a sequence's page number page_no, or -1 (reported) where there is none.
__device__ __forceinline__ int pap_page(const PagedAppendParams& p, int b, int page_no) {
  const int page = page_no < p.width ? p.table[(long long)b * p.table_stride + page_no] : -1;
  if (page >= 0 && page < p.n_pages) return page;
  report_error(p.status, DEV_ERR_BOUNDS, 613);
  return -1;
}

// Bounds of 4 channels of a page and head: widened by [l, h] (old), or set to it.
template <typename E>
__device__ __forceinline__ void pap_bounds(const PagedAppendParams& p, long long at, bool old, uint2 l, uint2 h) {
  uint2* lo = reinterpret_cast<uint2*>(static_cast<E*>(p.k_lo) + at);
  uint2* hi = reinterpret_cast<uint2*>(static_cast<E*>(p.k_hi) + at);
  if (old) {
    const uint2 a = *lo, b = *hi;
    l = make_uint2(Elem<E>::min2(l.x, a.x), Elem<E>::min2(l.y, a.y));
    h = make_uint2(Elem<E>::max2(h.x, b.x), Elem<E>::max2(h.y, b.y));
  }
  *lo = l;
  *hi = h;
}

template <typename E, int D, int SRC>
__global__ void __launch_bounds__(PAP_STEP_THREADS) paged_append_step_kernel(const __grid_constant__ PagedAppendParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr int PARTS = D / 8;
  const long long i = (long long)blockIdx.x * PAP_STEP_THREADS + threadIdx.x;
  const int part = (int)(i % PARTS), g = (int)(i / PARTS % p.Hkv);
  const long long bl = i / PARTS / p.Hkv;
  if (p.clear != nullptr)
    for (long long k = i; k < p.n_clear; k += (long long)gridDim.x * PAP_STEP_THREADS) p.clear[k] = 0;
  if (bl >= p.B) return;
  const int b = (int)bl;
  const int pos = p.start[b];
  if (pos < 0) {   // refused whole: neither keys nor queries of this sequence
    report_error(p.status, DEV_ERR_BOUNDS, 612);
    return;
  }
  const int in_page = pos & ((1 << p.ps_log2) - 1);
  const int page = p.pk != nullptr ? pap_page(p, b, pos >> p.ps_log2) : -1;
  PapTurn turn;
  if (p.rotate) turn.at(p, pos, part * 4);
  uint2 k[2];
  uint32_t big = 0;
  pap_token<E, D, SRC>(p, turn, b,
                       page < 0 ? -1 : (long long)page * p.page_stride + g * p.head_stride + (long long)in_page * p.row_stride,
                       g, part, k, big);
  pap_report<E>(p, big);
  if (p.k_lo != nullptr && page >= 0) {
    const long long at = ((long long)page * p.Hkv + g) * D + part * 4;
    pap_bounds<E>(p, at, in_page > 0, k[0], k[0]);
    pap_bounds<E>(p, at + D / 2, in_page > 0, k[1], k[1]);
  }
}

// New tokens of sequence b and its first token row; 0 tokens (and a report) where cu_new does
// not name rows of this call.
__device__ __forceinline__ int pap_count(const PagedAppendParams& p, int b, int* row0) {
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
  const int s = p.start[b];
  if (n == 0) return 0;
  if (s < 0 || s > 0x7fffffff - n) {   // refused whole: neither keys nor queries of this sequence
    report_error(p.status, DEV_ERR_BOUNDS, 612);
    return 0;
  }
  return ((s + n - 1) >> p.ps_log2) - (s >> p.ps_log2) + 1;
}

// 4 source elements in shared memory as two packed fp32 pairs
template <int SRC>
__device__ __forceinline__ void pap_get4(const uint8_t* s, uint64_t* f) {
  if constexpr (SRC == PDT_F32) {
    const float4 a = *reinterpret_cast<const float4*>(s);
    f[0] = f2_pack(a.x, a.y);
    f[1] = f2_pack(a.z, a.w);
  } else {
    PapRaw<SRC> raw;
    raw.r = *reinterpret_cast<const uint2*>(s);
    raw.get(f);
  }
}
// what a stage's rows need besides their bytes
struct PapMeta {
  long long row;     // element offset of the first row in the pool (head included), or -1: no place
  int tok, pos;      // first token row and position
  int rows, g;
  int page;
  int old, last;     // the page was begun by an earlier call; the run's last stage
};

template <typename E, int D, int SRC>
__global__ void __launch_bounds__(PAP_THREADS, PAP_PER_SM)
    paged_append_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                        const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ PagedAppendParams p) {
  constexpr int H2 = D / 2, PARTS = D / 8;      // threads of a row: 4 pairs each
  constexpr int ESZ = SRC == PDT_F32 ? 4 : 2;
  constexpr int HB = D * ESZ;                   // bytes of a head
  constexpr int NW = PAP_THREADS / 32;
  extern __shared__ __align__(128) uint8_t pap_smem[];   // stages of k, v [chunk][D] and q [chunk / 8][G][8][D]
  __shared__ __align__(8) uint32_t red[2][PAP_CONSUMERS];
  __shared__ uint64_t full[PAP_STAGES], empty[PAP_STAGES], sync_bar;
  __shared__ PapMeta metas[PAP_STAGES];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < PAP_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], PAP_CONSUMERS / 32);
    }
    mbar_init(&sync_bar, PAP_CONSUMERS / 32);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
    tma_prefetch_desc(&mapQ);
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  const int stage_bytes = p.chunk * HB * ((p.q != nullptr ? p.G : 0) + (p.k != nullptr ? 2 : 0));
  int stg = 0;
  uint32_t phase = 0;

  if (warp == NW - 1) {
    // ------------------------------ producer warp ------------------------------
    int b = 0, run = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv, filled = 0;   // run: counted from sequence b's first
    bool ok = true;
    // moves b to the sequence that holds the run, 32 sequences at a step; false past the last
    auto seek = [&]() {
      for (; b < p.B; b += 32) {
        const int c = b + lane < p.B ? pap_runs(p, b + lane) : 0;
        int inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > run);
        if (hit != 0) {
          const int l = __ffs(hit) - 1;
          run -= __shfl_sync(0xffffffffu, inc - c, l);
          b += l;
          return true;
        }
        run -= __shfl_sync(0xffffffffu, inc, 31);
      }
      return false;
    };
    while (ok && seek()) {
      int row0;
      const int n = pap_count(p, b, &row0), s0 = p.start[b];
      const int page_no = (s0 >> p.ps_log2) + run;          // page number within the sequence
      const int pos0 = run == 0 ? s0 : page_no << p.ps_log2;
      // (64-bit: the last page of the position range may end at 2^31)
      const int rows = (int)(min((long long)s0 + n, ((long long)page_no + 1) << p.ps_log2) - pos0);
      const int in_page = pos0 & ((1 << p.ps_log2) - 1);
      const int page = p.pk != nullptr ? pap_page(p, b, page_no) : -1;
      const long long base = (long long)page * p.page_stride + g * p.head_stride + (long long)in_page * p.row_stride;
      const int tok0 = row0 + (pos0 - s0);
      for (int c0 = 0; c0 < rows && ok; c0 += p.chunk) {
        const int nr = min(p.chunk, rows - c0);
        if (filled >= PAP_STAGES) ok = mbar_wait(&empty[stg], phase ^ 1u, &abort_flag, p.status, 615);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* sk = pap_smem + stg * stage_bytes;
        uint8_t* sv = sk + (p.k != nullptr ? p.chunk * HB : 0);
        uint8_t* sq = sv + (p.k != nullptr ? p.chunk * HB : 0);
        const int boxes = (nr + PAP_BOX - 1) / PAP_BOX, q_heads = p.q != nullptr ? p.G : 0;
        if (lane == 0) {
          PapMeta& m = metas[stg];
          m.row = page < 0 ? -1 : base + c0 * p.row_stride;
          m.tok = tok0 + c0;
          m.pos = pos0 + c0;
          m.rows = nr;
          m.g = g;
          m.page = page;
          m.old = in_page > 0;
          m.last = c0 + nr >= rows;
          mbar_arrive_expect_tx(&full[stg], boxes * PAP_BOX * HB * ((page >= 0 ? 2 : 0) + q_heads));
        }
        __syncwarp();
        const int per_box = q_heads + 2;   // per 8 tokens the boxes of the query heads, k and v, [8][D] each
        for (int x = lane; x < boxes * per_box; x += 32) {
          const int bx = x / per_box, h = x % per_box, tok = tok0 + c0 + bx * PAP_BOX;
          if (h < q_heads) {
            tma_load_2d(sq + (bx * p.G + h) * PAP_BOX * HB, &mapQ, &full[stg], (g * p.G + h) * D, tok);
          } else if (page >= 0) {
            tma_load_2d((h == q_heads ? sk : sv) + bx * PAP_BOX * HB, h == q_heads ? &mapK : &mapV, &full[stg], g * D,
                        tok);
          }
        }
        ++filled;
        if (++stg == PAP_STAGES) {
          stg = 0;
          phase ^= 1u;
        }
      }
      g += gridDim.x % p.Hkv;
      run += gridDim.x / p.Hkv;
      if (g >= p.Hkv) {
        g -= p.Hkv;
        ++run;
      }
    }
    if (lane == 0) {
      // the loads in flight land before the CTA can exit (also when the consumers gave up) ...
      int back = stg;
      uint32_t back_phase = phase;
      for (int k = min(filled, PAP_STAGES); k > 0; --k) {
        if (--back < 0) {
          back = PAP_STAGES - 1;
          back_phase ^= 1u;
        }
        mbar_wait(&full[back], back_phase, nullptr, p.status, 617);
      }
      // ... and one more stage, without rows, ends the consumers' walk
      if (ok && filled >= PAP_STAGES) ok = mbar_wait(&empty[stg], phase ^ 1u, &abort_flag, p.status, 616);
      if (ok) {
        metas[stg].rows = 0;
        mbar_arrive(&full[stg]);
      }
    }
    return;
  }

  // ------------------------------ consumer warps ------------------------------
  constexpr int PAIRS = D / 2, ROWS_AT_ONCE = PAP_CONSUMERS / PAIRS;   // bounds: threads by two channels and row
  constexpr uint32_t LO0 = Elem<E>::INF2, HI0 = Elem<E>::INF2 | 0x80008000u;
  uint32_t big = 0, lo = LO0, hi = HI0, sync_phase = 0;
  auto group_sync = [&]() {   // bounded, so that a warp that gave up holds no one for long
    __syncwarp();
    if (lane == 0) mbar_arrive(&sync_bar);
    const bool r = mbar_wait(&sync_bar, sync_phase & 1u, &abort_flag, p.status, 618);
    ++sync_phase;
    return __all_sync(0xffffffffu, r) != 0;
  };
  for (;;) {
    bool ok = mbar_wait(&full[stg], phase, &abort_flag, p.status, 619);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const PapMeta m = metas[stg];
    if (m.rows == 0) break;
    uint8_t* sk = pap_smem + stg * stage_bytes;
    const uint8_t* sv = sk + (p.k != nullptr ? p.chunk * HB : 0);
    const uint8_t* sq = sv + (p.k != nullptr ? p.chunk * HB : 0);
    const bool bounds = p.k_lo != nullptr && m.page >= 0;
    for (int i = tid; i < m.rows * PARTS; i += PAP_CONSUMERS) {
      const int r = i / PARTS, part = i % PARTS;
      const int at = r * HB + part * 4 * ESZ;
      PapTurn turn;
      if (p.rotate) turn.at(p, m.pos + r, part * 4);
      auto rotate = [&](const uint8_t* s, uint2* out) {
        uint64_t a[2], c[2];
        pap_get4<SRC>(s, a);
        pap_get4<SRC>(s + H2 * ESZ, c);
        if (p.rotate) {
#pragma unroll
          for (int e = 0; e < 2; ++e) turn.apply(e, a[e], c[e]);
        }
        out[0] = pap_round<E>(a, big);
        out[1] = pap_round<E>(c, big);
      };
      if (m.page >= 0) {
        const long long dst = m.row + r * p.row_stride + part * 4;
        uint2 y[2];
        uint64_t f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          pap_get4<SRC>(sv + at + e * H2 * ESZ, f);
          *reinterpret_cast<uint2*>(static_cast<E*>(p.pv) + dst + e * H2) = pap_round<E>(f, big);
        }
        rotate(sk + at, y);
        *reinterpret_cast<uint2*>(static_cast<E*>(p.pk) + dst) = y[0];
        *reinterpret_cast<uint2*>(static_cast<E*>(p.pk) + dst + H2) = y[1];
        if (bounds) {   // the stored key, over its source (which this thread alone reads)
          *reinterpret_cast<uint2*>(sk + at) = y[0];
          *reinterpret_cast<uint2*>(sk + at + H2 * ESZ) = y[1];
        }
      }
      if (p.q != nullptr) {
        E* qo = static_cast<E*>(p.q_out) + ((long long)(m.tok + r) * p.Hkv + m.g) * p.G * D + part * 4;
        const uint8_t* qs = sq + ((r / PAP_BOX) * p.G * PAP_BOX + r % PAP_BOX) * HB + part * 4 * ESZ;
#pragma unroll 2
        for (int h = 0; h < p.G; ++h) {
          uint2 y[2];
          rotate(qs + h * PAP_BOX * HB, y);
          *reinterpret_cast<uint2*>(qo + h * D) = y[0];
          *reinterpret_cast<uint2*>(qo + h * D + H2) = y[1];
        }
      }
    }
    if (bounds) {
      if (!group_sync()) break;
      // channels 2c, 2c + 1: of the 4 of a part, at 16-bit steps behind the part's first byte
      const int c = tid % PAIRS, half = c / (H2 / 2), x = c % (H2 / 2);
      const uint8_t* col = sk + half * H2 * ESZ + (x / 2) * 4 * ESZ + (x % 2) * 4;
      for (int r = tid / PAIRS; r < m.rows; r += ROWS_AT_ONCE) {
        const uint32_t k = *reinterpret_cast<const uint32_t*>(col + r * HB);
        lo = Elem<E>::min2(lo, k);
        hi = Elem<E>::max2(hi, k);
      }
      fence_proxy_async_smem();   // the kept keys were written through the generic proxy
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stg]);   // this warp is done with the stage
    if (bounds && m.last) {
      // over the run's rows, and over what an earlier call wrote when the run does not begin
      // the page (red is free again by the next stage's group_sync)
      red[0][tid] = lo;
      red[1][tid] = hi;
      lo = LO0;
      hi = HI0;
      if (!group_sync()) break;
      if (tid < D / 4) {
        uint2 l = *reinterpret_cast<const uint2*>(&red[0][2 * tid]), h = *reinterpret_cast<const uint2*>(&red[1][2 * tid]);
#pragma unroll
        for (int k = 1; k < ROWS_AT_ONCE; ++k) {
          const uint2 l2 = *reinterpret_cast<const uint2*>(&red[0][k * PAIRS + 2 * tid]);
          const uint2 h2 = *reinterpret_cast<const uint2*>(&red[1][k * PAIRS + 2 * tid]);
          l = make_uint2(Elem<E>::min2(l.x, l2.x), Elem<E>::min2(l.y, l2.y));
          h = make_uint2(Elem<E>::max2(h.x, h2.x), Elem<E>::max2(h.y, h2.y));
        }
        pap_bounds<E>(p, ((long long)m.page * p.Hkv + m.g) * D + tid * 4, m.old != 0, l, h);
      }
    }
    if (++stg == PAP_STAGES) {
      stg = 0;
      phase ^= 1u;
    }
  }
  pap_report<E>(p, big);
}

// ----------------------------------------------------------------------------------------
// Page selection.  The largest value that q_h . k can take over keys k inside a page's box
// lo <= k <= hi is sum_d max(q_hd lo_d, q_hd hi_d); summed over the G query heads of a group
// it is
//   score(page) = sum_d up_d hi_d + dn_d lo_d,   up_d = sum_h max(q_hd, 0), dn_d = sum_h min(q_hd, 0)
// so a group costs one pair of dot products whatever G is.
//
// The scores are held in 64 bits, so that ranks depend on rounding only where scores agree to
// about 15 digits.  A 16-bit value is put
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

// A cluster of 1 to 8 CTAs serves a (sequence, kv head): each scores a share of the pages, 8
// channels per lane, into the first CTA's shared memory, and that CTA ranks them: a radix
// selection from the top digit down, on keys (the scores' bits in an order-preserving form)
// rebased to the smallest one so that the first digit already spreads them, until at most 32
// candidates share the digits of the last page taken; a warp ranks those.
//
// Bound by latency: a chain of length, table, bounds, cluster barrier and four block-wide
// steps.  2049 pages x 5 heads of one sequence take 12 us, 64 sequences of up to 512 pages 14 us
// (22 MB of bounds, 3.4 us at 6.55 TB/s); as two launches with a key buffer they took 20 and 24.
// 512 threads per CTA were faster for one sequence (13.4 against 14.1 us cold) and slower for 64
// (23.5 against 16.8), two page groups in flight instead of four slower for both.
struct PagedSelectParams {
  const void *k_lo, *k_hi;   // [n_pages, Hkv, D]
  const void* q;             // [B] rows of Hq*D
  long long q_stride;
  const int* table;
  long long table_stride;
  const int* lens;
  int len_add;               // added to every length
  int width, cap, B, Hkv, G, n_pages, ps_log2, n_first, n_last, top;
  int* page_idx;             // [B, Hkv, top]
  DevStatus* status;
};

// Sequence lengths: lens[b] + add, clamped to 0 .. cap, the positions that the table holds.
__device__ __forceinline__ int paged_len(int len, int cap) { return max(0, min(len, cap)); }
__device__ __forceinline__ int paged_pages(int len, int ps_log2) {
  return (int)(((unsigned)len + (1u << ps_log2) - 1u) >> ps_log2);
}

__device__ __forceinline__ int paged_raw_len(const int* lens, int b, int add) {
  const int l = lens[b];
  return l > 0x7fffffff - add ? l : l + add;
}

constexpr int PSEL_THREADS = 256;
constexpr int PSEL_WARPS = PSEL_THREADS / 32;

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <typename E, int D>
__global__ void __launch_bounds__(PSEL_THREADS, 2)
    paged_select_kernel(const __grid_constant__ PagedSelectParams p, int cluster) {
  constexpr int LPP = D / 8;          // lanes per page
  constexpr int PPI = 32 / LPP;       // pages per warp at a time
  extern __shared__ unsigned long long psel_keys[];   // one per page, in the cluster's first CTA
  __shared__ unsigned long long red[2][PSEL_WARPS], cand_key[32], last_key;
  __shared__ int hist[256], found[2], cand_idx[32], n_cand, last_idx, wsum[PSEL_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, bg = blockIdx.x / cluster, b = bg / p.Hkv, g = bg % p.Hkv;
  const int d0 = (lane % LPP) * 8, sub = lane / LPP;
  pdl_wait();
  pdl_trigger();
  constexpr int QB = 8;   // query heads whose loads are in flight together, with the length's
  const E* q = static_cast<const E*>(p.q) + b * p.q_stride + (long long)g * p.G * D + d0;
  uint4 qr[QB];
#pragma unroll
  for (int h = 0; h < QB; ++h)
    if (h < p.G) qr[h] = *reinterpret_cast<const uint4*>(q + h * D);
  const int raw_len = paged_raw_len(p.lens, b, p.len_add);
  const int len = paged_len(raw_len, p.cap);
  if (len != raw_len && tid == 0) report_error(p.status, DEV_ERR_BOUNDS, 621);
  const int n = paged_pages(len, p.ps_log2);
  int* out = p.page_idx + (long long)bg * p.top;
  if (n <= p.top) {   // every page (the whole cluster takes this branch)
    if (rank == 0)
      for (int i = tid; i < p.top; i += PSEL_THREADS) out[i] = i < n ? i : -1;
    return;
  }

  // 1. scores of this CTA's share, a chunk of up to 32 pages per warp at a time
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  {
    const int share = (n + cluster - 1) / cluster, s0 = min(n, rank * share), s1 = min(n, s0 + share);
    int chunk = 32;   // small shares: fewer, so that every warp has some
    while (chunk > PPI && chunk * PSEL_WARPS >= 2 * share) chunk >>= 1;
    double up[8], dn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) up[e] = dn[e] = 0.0;
    for (int h0 = 0; h0 < p.G; h0 += QB) {
#pragma unroll
      for (int h = 0; h < QB; ++h) {
        if (h0 + h >= p.G) break;
        const uint4 r = h0 == 0 ? qr[h] : *reinterpret_cast<const uint4*>(q + (h0 + h) * D);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Elem<E>::unpack(w[e]);
          up[2 * e] += (double)fmaxf(f.x, 0.f);
          up[2 * e + 1] += (double)fmaxf(f.y, 0.f);
          dn[2 * e] += (double)fminf(f.x, 0.f);
          dn[2 * e + 1] += (double)fminf(f.y, 0.f);
        }
      }
    }
    const double qs = q_scale<E>();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      up[e] *= qs;
      dn[e] *= qs;
    }
    const uint32_t keys0 = smem_cluster_addr(psel_keys, 0);
    // the first CTA has started before its shared memory is written
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int j0 = s0 + warp * chunk; j0 < s1; j0 += PSEL_WARPS * chunk) {
      const int nj = min(chunk, s1 - j0);
      int entry = -1;
      if (lane < nj) {
        entry = p.table[(long long)b * p.table_stride + j0 + lane];
        if (entry < 0 || entry >= p.n_pages) {   // not in the pool: ranked last
          report_error(p.status, DEV_ERR_BOUNDS, 622);
          entry = -1;
        }
      }
      constexpr int UN = 4;   // page groups whose loads are in flight together
      for (int i0 = 0; i0 < nj; i0 += UN * PPI) {
        int page[UN];
        uint4 hi[UN], lo[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          page[u] = __shfl_sync(0xffffffffu, entry, (i0 + u * PPI + sub) & 31);
          const long long at = ((long long)max(page[u], 0) * p.Hkv + g) * D + d0;   // (page 0 in the place of none)
          hi[u] = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.k_hi) + at);
          lo[u] = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.k_lo) + at);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          const uint32_t hw[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w}, lw[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w};
          double s = 0.0, t = 0.0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s = fma(up[e], raw_double<E>((hw[e / 2] >> (16 * (e & 1))) & 0xffffu), s);
            t = fma(dn[e], raw_double<E>((lw[e / 2] >> (16 * (e & 1))) & 0xffffu), t);
          }
          s += t;
#pragma unroll
          for (int o = LPP / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          const int i = i0 + u * PPI + sub;
          if (i < nj && lane % LPP == 0) {
            const unsigned long long v = (unsigned long long)__double_as_longlong(s + 0.0);   // -0 becomes +0
            st_cluster_u64(keys0 + (j0 + i) * 8,
                           page[u] < 0 ? 0ull : ((v >> 63) ? ~v : v | 0x8000000000000000ull));
          }
        }
      }
    }
  }
  cluster_sync();
  if (rank != 0) return;

  // 2. the range of the keys of the pages that are not forced (n > top >= n_first + n_last: the
  //    forced ones do not overlap)
  const int f0 = p.n_first, f1 = n - p.n_last;
  unsigned long long mn = ~0ull, mx = 0;
  // (the loops of the selection run once a call: unrolled, they would cost more in instruction
  // fetches than they save)
#pragma unroll 1
  for (int i = f0 + tid; i < f1; i += PSEL_THREADS) {
    mn = min(mn, psel_keys[i]);
    mx = max(mx, psel_keys[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (lane == 0) {
    red[0][warp] = mn;
    red[1][warp] = mx;
  }
  hist[tid] = 0;
  if (tid == 0) n_cand = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < PSEL_WARPS; ++w) {
    mn = min(mn, red[0][w]);
    mx = max(mx, red[1][w]);
  }

  // 3. the last page taken: (key, number), no other page that is taken ranks lower.  The pages
  //    with base <= key < base + 2^bits are still undecided, `need` of them are taken.
  int need = p.top - p.n_first - p.n_last, count = f1 - f0;
  unsigned long long base = mn;
  int bits = 64 - __clzll((long long)(mx - mn));
  auto undecided = [&](unsigned long long k) { return k >= base && (bits == 64 || ((k - base) >> bits) == 0); };
  if (need == 0) {
    if (tid == 0) {
      last_key = ~0ull;
      last_idx = -1;
    }
  } else {
    while (count > 32 && bits > 0) {
      const int shift = max(bits - 8, 0);
#pragma unroll 1
      for (int i = f0 + tid; i < f1; i += PSEL_THREADS) {
        const unsigned long long k = psel_keys[i];
        if (undecided(k)) atomicAdd(&hist[(int)((k - base) >> shift)], 1);
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
      count = hist[d];
      base += (unsigned long long)d << shift;
      bits = shift;
      __syncthreads();
      hist[tid] = 0;
      __syncthreads();
    }
    if (count <= 32) {   // rank the candidates
#pragma unroll 1
      for (int i = f0 + tid; i < f1; i += PSEL_THREADS) {
        const unsigned long long k = psel_keys[i];
        if (undecided(k)) {
          const int at = atomicAdd(&n_cand, 1);
          cand_key[at] = k;
          cand_idx[at] = i;
        }
      }
      __syncthreads();
      if (warp == 0) {
        const bool in = lane < count;
        const unsigned long long k = in ? cand_key[lane] : 0;
        const int idx = in ? cand_idx[lane] : 0;
        int above = 0;
#pragma unroll 1
        for (int o = 0; o < count; ++o) {
          const unsigned long long k2 = __shfl_sync(0xffffffffu, k, o);
          const int i2 = __shfl_sync(0xffffffffu, idx, o);
          above += k2 > k || (k2 == k && i2 < idx) ? 1 : 0;
        }
        if (in && above == need - 1) {
          last_key = k;
          last_idx = idx;
        }
      }
    } else if (warp == 0) {   // more than 32 pages of one score: the need-th of them
      int seen = 0;
      for (int i = f0; i < f1; i += 32) {
        const bool eq = i + lane < f1 && psel_keys[i + lane] == base;
        const unsigned m = __ballot_sync(0xffffffffu, eq);
        if (eq && seen + __popc(m & ((1u << lane) - 1)) == need - 1) {
          last_key = base;
          last_idx = i + lane;
        }
        seen += __popc(m);
      }
    }
  }
  __syncthreads();

  // 4. the list: every warp writes the pages of its stretch in order
  const unsigned long long lk = last_key;
  const int li = last_idx;
  auto taken = [&](int i) {
    if (i >= n) return false;
    if (i < f0 || i >= f1) return true;
    const unsigned long long k = psel_keys[i];
    return k > lk || (k == lk && i <= li);
  };
  const int stretch = (n + PSEL_THREADS - 1) / PSEL_THREADS * 32, i0 = warp * stretch, i1 = min(n, i0 + stretch);
  int mine = 0;
#pragma unroll 1
  for (int i = i0; i < i1; i += 32) mine += __popc(__ballot_sync(0xffffffffu, taken(i + lane)));
  if (lane == 0) wsum[warp] = mine;
  __syncthreads();
  int at = 0;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) at += wsum[w];
#pragma unroll 1
  for (int i = i0; i < i1; i += 32) {
    const bool t = taken(i + lane);
    const unsigned m = __ballot_sync(0xffffffffu, t);
    if (t) out[at + __popc(m & ((1u << lane) - 1))] = i + lane;
    at += __popc(m);
  }
}

// ----------------------------------------------------------------------------------------
// Attention of one new token per sequence over its pages ([JJ] eq. (1) for one query row):
//   o = sum_j e_j v_j / sum_j e_j,  e_j = 2^(scale log2(e) q.k_j - m)
// over the visible positions j < lens[b]: all of them, those with j < M or j >= lens[b] - W
// (meta tokens and window), or those of the listed pages.
//
// The keys of (sequence, kv head), an item, are cut into tiles of 64 positions, and the tiles
// of all items, in order, are dealt to the CTAs (one per SM) as equal contiguous shares, and
// a CTA's share to its groups: a long sequence is split over many CTAs and short ones share a
// group, whatever the lengths are (they are known on the device only, and a replayed graph
// sees new ones).  An item that one group covers alone is finished there.  Of a cut item every
// group leaves its running maximum, sum and weighted values in shared memory; when the CTA's
// groups are done it merges the parts of the same item, and if other CTAs have a share of the
// item too it leaves one part in the workspace and counts it, and the CTA that completes the
// count merges the parts in CTA order: the result does not depend on which one that is.  One
// CTA per SM (instead of three small ones) keeps that last join to at most 148 parts and gives
// it all of the CTA's threads (131073 keys of one sequence: 61 us with three, 44 with one).
//
// A group is a producer warp and four consumer warps with a ring of stages of their own.  The
// producer walks the group's tiles: its lanes look up the pages and issue one TMA box per page
// piece (128-byte swizzled rows; D = 128 as two 64-wide halves), with the visibility of the
// tile's 64 positions as a bit mask beside it; a page that does not exist gets an
// out-of-range coordinate, which TMA fills with zeros.  The consumer warps take 16 positions
// of every tile each.  The item's query heads are rows of 16 x 16 x 8 tensor-core products:
// rows 0..7 hold up to 8 heads, and rows 8..15, otherwise empty, take in the second product
// the rounding error of the probabilities (p = hi + lo, both 16 bits), so P V costs the same
// number of instructions and keeps about twice the mantissa: 22 bits in fp16, of 2^15 p, so
// that many small ones beside a large one count too (a bare p below 2^-25 would round to 0).
// bf16's 16 bits show in an fp32 output (1.2e-6 of it against 3.8e-7), so there, and only there,
// what is left goes through a second product (97.8 -> 98.8 us at 8 x 65537 keys).  With 9 to 16
// heads (NHB = 2) rows 8..15 of Q K^T are heads 8..15, and P V runs once per 8 heads.
//
// Bound by the keys' and values' bytes, read once (ncu: 310 MB for 307).  Long runs stream at
// 6.6 TB/s (2.7 GB in 410 us; a plain copy reaches 6.55), to which a call adds about 10 us: 3 to
// the first copy, 2 to its data, the spread of the SMs at the end, and 3 to publish and join
// cut items.  Back to back, with inputs that change from call to call, 8 x 65537 keys in bf16
// take 101 us (floor 88), 64 x up to 8320 58 (47), one sequence of 131073 37 (26), a window of
// 1024 + 128 for 64 sequences 28 (15), 48 listed pages of 32 for 64 32 (18).  A fourth stage or two
// groups of five changed nothing or cost 3%; two stages are 3% slower at D = 64 and 1% faster
// at D = 128.  9 to 16 heads per kv head are bound by the latency of the consumer warps' own
// chains, of which fewer fit (255 registers a thread at D = 128, one consumer warp per scheduler:
// issue slots 22% busy, DRAM 38%): 8 x up to 131073 keys, 16 heads x 64, 42 us in fp16 and 45 in bf16
// (floor 22; 8 heads 35), 8 x up to 65537, 32/2 heads x 128, 78 and 88 us (44; 16/2 heads 56).
// ----------------------------------------------------------------------------------------
constexpr int PA_KT = 64;
constexpr int PA_MAX_GRID = 148;   // CTAs (sizes the workspace)
constexpr int PA_PART_WORDS = (PA_MAX_GRID + 3) / 4;   // words of the CTAs' part counters in the status
static_assert(PA_MAX_GRID < 256 && PA_PART_WORDS <= sizeof(DevStatus::parts) / sizeof(unsigned),
              "a counter counts up to one part per CTA in 8 bits");

template <int D, int NHB>
struct PaShape {
  static constexpr int GROUPS = NHB == 1 ? (D == 64 ? 3 : 2) : (D == 64 ? 2 : 1);
  static constexpr int STAGES = D == 64 ? (NHB == 1 ? 3 : 4) : (NHB == 1 ? 2 : 5);
  static constexpr int CWARPS = 4 * GROUPS;                // consumer warps
  static constexpr int THREADS = (CWARPS + GROUPS) * 32;
  static constexpr int HALF = PA_KT * 128;                 // bytes of 64 positions x 64 dims
  static constexpr int STAGE = 2 * (D / 64) * HALF;        // K then V
  static constexpr int QB = 8 * NHB * D * 2;
  static constexpr int LD = D + 4;                         // floats of a part's row: values, max, sum
  static constexpr int SMEM = GROUPS * (STAGES * STAGE + 4 * 8 * LD * 4) + 1024;   // rings, merge rows, alignment
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
  int top, width, cap, B, Hq, Hkv, G, n_pages, ps_log2, M, W;
  int dim_row, dim_head;      // tensor-map dimensions (1..3) of rows and heads; pages have the other
  float scale_log2;
  float* part;                // [grid][2][G][D + 4]: slot 1 the item that begins in the CTA
  DevStatus* status;          // its counter c: parts of the cut item that CTA c began
};

struct PaTiles {
  int len;      // positions of the sequence
  int n_tiles;  // at least 1
  int head;     // window: the first tiles (meta); tile t >= head stands for tile t + skip
  int skip;
};
__device__ __forceinline__ PaTiles pa_tiles(const PagedAttnParams& p, int raw_len) {
  PaTiles r;
  r.len = paged_len(raw_len, p.cap);
  const int all = (int)(((unsigned)r.len + PA_KT - 1) / PA_KT);
  r.head = all;
  r.skip = 0;
  r.n_tiles = all;
  if (p.page_idx != nullptr) {
    const unsigned rows = (unsigned)min(paged_pages(r.len, p.ps_log2), p.top) << p.ps_log2;   // at most 2^31
    r.n_tiles = (int)((rows + PA_KT - 1) / PA_KT);
  } else if (p.W > 0) {
    const int w0 = max(0, r.len - p.W) / PA_KT;           // the window's first tile
    r.head = min(w0, (int)(((unsigned)p.M + PA_KT - 1) / PA_KT));   // (M may be up to 2^31 - 1)
    r.skip = w0 - r.head;
    r.n_tiles = all - r.skip;
  }
  if (r.n_tiles < 1) r.n_tiles = 1;                       // an empty sequence: one tile without keys
  return r;
}
__device__ __forceinline__ int pa_len(const PagedAttnParams& p, int b) { return paged_raw_len(p.lens, b, p.len_add); }
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
}
// Shares of `total` tiles for n CTAs: the first total % n of them get one more.  (The host keeps
// the number of tiles below 2^31.)
struct PaShares {
  int q, r;
  __device__ PaShares(int total, int n) : q(total / n), r(total % n) {}
  __device__ int begin(int c) const { return c * q + min(c, r); }
  __device__ int owner(int x) const { return x < r * (q + 1) ? x / (q + 1) : r + (x - r * (q + 1)) / q; }
};

// what a stage's tile needs besides its bytes
struct PaMeta {
  unsigned long long mask;   // visible positions
  int item;                  // sequence * Hkv + kv head
  int last;                  // the item's last tile in this group; only then:
  int cut;                   // the group has a part of the item only: 1 begun earlier, 2 begun here
  int ends;                  // the item ends here
  int c0, parts;             // the CTA that begins the item, and how many CTAs share it
};
// a group's part of a cut item, in shared memory
struct PaPart {
  int item;                  // -1: none
  int c0, parts;
};

// The running maximum and sum of a query head's softmax and 4 of its D weighted values; in memory
// a row of D values, then the maximum and the sum.
template <int D>
struct PaAcc {
  float m, l, x[4];
  __device__ void clear() {
    m = -INFINITY;
    l = x[0] = x[1] = x[2] = x[3] = 0.f;
  }
  __device__ void add(float m2, float l2, const float4& y) {
    const float mn = fmaxf(m, m2), mu = mn == -INFINITY ? 0.f : mn;
    const float wa = ex2_approx(m - mu), wb = ex2_approx(m2 - mu);
    m = mn;
    l = l * wa + l2 * wb;
    x[0] = x[0] * wa + y.x * wb;
    x[1] = x[1] * wa + y.y * wb;
    x[2] = x[2] * wa + y.z * wb;
    x[3] = x[3] * wa + y.w * wb;
  }
  __device__ void add(const float* row, int quad) {
    add(row[D], row[D + 1], *reinterpret_cast<const float4*>(row + 4 * quad));
  }
  __device__ void put(float* row, int quad) const {
    *reinterpret_cast<float4*>(row + 4 * quad) = make_float4(x[0], x[1], x[2], x[3]);
    if (quad == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m, l);
  }
};
__device__ __forceinline__ float pa_inverse(float l) {   // no key: zeros; a NaN stays one
  return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
}
__device__ __forceinline__ float pa_lse(float m, float l) {
  return l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
}
// 4 values of query head hh of an item, and its lse
template <int D>
__device__ __forceinline__ void pa_finish(const PagedAttnParams& p, int item, int hh, int quad, const PaAcc<D>& a) {
  const int b = item / p.Hkv, h = item % p.Hkv * p.G + hh;
  const float inv = pa_inverse(a.l);
  const long long at = b * p.out_stride + (long long)h * D + 4 * quad;
  const float y[4] = {a.x[0] * inv, a.x[1] * inv, a.x[2] * inv, a.x[3] * inv};
  if (p.out_dt == PDT_F16) f16_range_guard<4>(y, p.status, 609);
  store_pair(p.out, p.out_dt, at, y[0], y[1]);
  store_pair(p.out, p.out_dt, at + 2, y[2], y[3]);
  if (p.lse != nullptr && quad == 0) p.lse[(long long)b * p.Hq + h] = pa_lse(a.m, a.l);
}

// Count a part of the item that CTA c0 began; true for the last of `parts`, which also returns
// the counter to zero.  Releases what the caller's CTA wrote before (after a barrier), and
// acquires what the others did.  Four counters share a word: they lie in the status, which every
// workspace has and no other call touches, so a workspace may serve calls of other kinds in
// between.
__device__ __forceinline__ bool pa_arrive(const PagedAttnParams& p, int c0, int parts) {
  unsigned* word = p.status->parts + c0 / 4;
  const int sh = c0 % 4 * 8;
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(word), "r"(1u << sh) : "memory");
  if (((old >> sh) & 255u) != (unsigned)(parts - 1)) return false;
  atomicSub(word, (unsigned)parts << sh);
  return true;
}
// A CTA counts each of its two parts once: whoever takes its flag does.  (After a wait that gave
// up, another group may still be on its way to publish.)
__device__ __forceinline__ bool pa_claim(int* counted) { return atomicExch(counted, 1) == 0; }
// After a wait that gave up, the counts are completed all the same, so that the next call on
// the workspace finds them at zero: count this CTA's parts of cut items that nobody has claimed
// (counted[0]: of an item begun earlier, [1]: of one that goes on), walking the items.
__device__ __noinline__ void pa_arrive_rest(const PagedAttnParams& p, int t0, int t1, const PaShares& sh, int* counted) {
  int beg = 0;
  for (int b = 0; b < p.B && beg < t1; ++b) {
    const int nt = pa_tiles(p, pa_len(p, b)).n_tiles;
    for (int g = 0; g < p.Hkv && beg < t1; ++g, beg += nt) {
      const int end = beg + nt;
      if (end <= t0 || (beg >= t0 && end <= t1) || !pa_claim(counted + (beg < t0 ? 0 : 1))) continue;
      const int c0 = sh.owner(beg);
      pa_arrive(p, c0, sh.owner(end - 1) - c0 + 1);
    }
  }
}

// Merge the CTAs' parts of n_jobs items, by the CTA's consumer threads: D / 4 lanes (4 values
// each) per part and head, per_head such groups of lanes to a head, each with every per_head-th
// part, then a head's groups through sh (a row of LD floats each).  per_head follows from an
// item's parts alone (pa_join_width), so that the order of its sums does not depend on which
// CTA joins it or what else that one has to join.  The loads go past L1, which may hold an older
// line of a neighbouring part.
constexpr int PA_JOIN_UN = 8;   // parts whose loads are in flight together
template <int D, int CWARPS>
__device__ __forceinline__ int pa_join_width(int parts, int G) {   // a batch of loads in one group, or all groups
  constexpr int SUBS = CWARPS * 32 / (D / 4);
  return parts <= PA_JOIN_UN ? 1 : SUBS / min(G, SUBS);
}
template <int D, int CWARPS, typename Sync>
__device__ __forceinline__ bool pa_join(const PagedAttnParams& p, const PaPart* jobs, int n_jobs, int per_head, int tid,
                                        float* sh, Sync& sync) {
  constexpr int LPR = D / 4, SUBS = CWARPS * 32 / LPR, LD = D + 4;
  const int sub = tid / LPR, quad = tid % LPR;
  const int n_heads = n_jobs * p.G, heads = min(n_heads, SUBS / per_head);   // heads: at a time
  const int hs = sub / per_head, s0 = sub % per_head;
#pragma unroll 1
  for (int h0 = 0; h0 < n_heads; h0 += heads) {
    PaAcc<D> a;
    a.clear();
    const int h = h0 + hs;
    if (hs < heads && h < n_heads) {
      const PaPart j = jobs[h / p.G];
      const float* src = p.part + ((long long)j.c0 * 2 * p.G + h % p.G) * LD;
      constexpr int UN = PA_JOIN_UN;
#pragma unroll 1
      for (int i0 = s0; i0 < j.parts; i0 += UN * per_head) {
        float2 ml[UN];
        float4 x[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          const int i = min(i0 + u * per_head, j.parts - 1);   // (past the end: the last one, not added)
          const float* row = src + ((long long)i * 2 + (i == 0 ? 1 : 0)) * p.G * LD;
          ml[u] = __ldcg(reinterpret_cast<const float2*>(row + D));
          x[u] = __ldcg(reinterpret_cast<const float4*>(row) + quad);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u)
          if (i0 + u * per_head < j.parts) a.add(ml[u].x, ml[u].y, x[u]);
      }
    }
    a.put(sh + sub * LD, quad);
    if (!sync()) return false;
    if (sub < heads && h0 + sub < n_heads) {
      PaAcc<D> t;
      t.clear();
#pragma unroll 1
      for (int k = 0; k < per_head; ++k) t.add(sh + (sub * per_head + k) * LD, quad);
      pa_finish<D>(p, jobs[(h0 + sub) / p.G].item, (h0 + sub) % p.G, quad, t);
    }
    if (!sync()) return false;   // the rows are free again
  }
  return true;
}

template <typename E, int D, int NHB>
__global__ void __launch_bounds__(PaShape<D, NHB>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                      const __grid_constant__ PagedAttnParams p) {
  using S = PaShape<D, NHB>;
  constexpr int STAGES = S::STAGES, GROUPS = S::GROUPS, CWARPS = S::CWARPS, LD = S::LD;
  constexpr int NH = D / 64;
  constexpr int NWARPS = S::THREADS / 32;
  constexpr float P_SCALE = Elem<E>::IS_F16 ? 32768.f : 1.f;   // of the probabilities in P V
  extern __shared__ uint8_t pa_smem_raw[];
  uint8_t* rings = align_smem<1024>(pa_smem_raw);
  float (*mos)[4][8][LD] =                                             // a group's warps' parts of an item
      reinterpret_cast<float (*)[4][8][LD]>(rings + GROUPS * STAGES * S::STAGE);
  __shared__ uint64_t full_bars[GROUPS][STAGES], empty_bars[GROUPS][STAGES], merge_bars[GROUPS], fin_bar;
  __shared__ __align__(16) PaMeta metas[GROUPS][STAGES];
  __shared__ __align__(128) uint8_t qbufs[GROUPS][2][S::QB];         // the queries of every other item
  __shared__ __align__(16) float prows[GROUPS][2][8 * NHB][LD];      // the groups' parts of cut items: one
                                                                     // begun earlier, one begun in the group
  __shared__ PaPart pinfo[GROUPS][2];
  __shared__ int wsum[NWARPS];                       // tiles of a warp's sequences
  __shared__ int counted[2], abort_flag;             // whether the part of slot 0 / 1 is counted (pa_claim)
  __shared__ PaPart joins[2];                        // the cut items that this CTA joins
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int k = 0; k < GROUPS; ++k) {
      for (int i = 0; i < STAGES; ++i) {
        mbar_init(&full_bars[k][i], 1);
        mbar_init(&empty_bars[k][i], 4);
      }
      mbar_init(&merge_bars[k], 4);
      pinfo[k][0].item = pinfo[k][1].item = -1;
    }
    mbar_init(&fin_bar, CWARPS);
    joins[0].item = joins[1].item = -1;
    abort_flag = counted[0] = counted[1] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
  }
  pdl_wait();
  pdl_trigger();

  // 1. the shares of this CTA and of its groups, and the sequences they start in
  const int per = (p.B + S::THREADS - 1) / S::THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int mine = 0;
  for (int i = b0; i < b1; ++i) {
    const int l = pa_len(p, i);
    const PaTiles t = pa_tiles(p, l);
    if (t.len != l && blockIdx.x == 0) report_error(p.status, DEV_ERR_BOUNDS, 601);
    mine += t.n_tiles * p.Hkv;
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  // tiles up to and with a thread's sequences, in its warp: a copy for each producer warp, where
  // its ring will be
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) reinterpret_cast<int*>(rings + k * STAGES * S::STAGE)[tid] = inc;
  fence_proxy_async_smem();
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int wins = lane < NWARPS ? wsum[lane] : 0;   // tiles up to and with warp `lane`'s sequences
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, wins, o);
    if (lane >= o) wins += up;
  }
  const int total = __shfl_sync(0xffffffffu, wins, NWARPS - 1);
  const int n_cta = min((int)gridDim.x, total);
  if ((int)blockIdx.x >= n_cta) return;
  const PaShares shares(total, n_cta);
  const int t0 = shares.begin(blockIdx.x), t1 = shares.begin(blockIdx.x + 1);
  const bool producer = warp >= CWARPS;
  const int grp = producer ? warp - CWARPS : warp / 4;
  const int gq0 = (t1 - t0) / GROUPS, gr0 = (t1 - t0) % GROUPS;
  const int u0 = t0 + grp * gq0 + min(grp, gr0), n_mine = gq0 + (grp < gr0 ? 1 : 0), u1 = u0 + n_mine;
  uint64_t* full = full_bars[grp];
  uint64_t* empty = empty_bars[grp];
  uint8_t* ring = rings + grp * STAGES * S::STAGE;

  if (producer) {
    // ------------------------------ producer warp ------------------------------
    if (n_mine == 0) return;
    const int ps = 1 << p.ps_log2;
    const int R = min(ps, PA_KT), n_chunk = PA_KT / R;    // a tile's page pieces
    // the sequence, kv head and tile that the group starts at: the warp, the thread and the
    // sequence that hold tile u0
    int b, g, t, left = u0;
    {
      const int* upto = reinterpret_cast<const int*>(ring);
      const int w = __ffs(__ballot_sync(0xffffffffu, wins > left)) - 1;
      const int skip = __shfl_sync(0xffffffffu, wins, max(w - 1, 0));
      if (w > 0) left -= skip;
      const unsigned hit = __ballot_sync(0xffffffffu, upto[w * 32 + lane] > left);
      const int owner = w * 32 + __ffs(hit) - 1;
      if (owner > w * 32) left -= upto[owner - 1];
      b = owner * per;
      __syncwarp();
      fence_proxy_async_smem();   // from here on the ring belongs to the copies
    }
    PaTiles sq = pa_tiles(p, pa_len(p, b));
    while (left >= sq.n_tiles * p.Hkv && b + 1 < p.B) {
      left -= sq.n_tiles * p.Hkv;
      sq = pa_tiles(p, pa_len(p, ++b));
    }
    g = left / sq.n_tiles;
    t = left - g * sq.n_tiles;
    int next_len = b + 1 < p.B ? pa_len(p, b + 1) : 0;
    bool ok = true;
    // One tile's page piece of this lane: the table's page (checked when it is used, so that the
    // look-up of the next tile stays in flight meanwhile), the first row in it, and the visible
    // rows as bits (0: nothing to read).
    struct Piece {
      int page, row;
      unsigned long long bits;
    };
    auto look = [&]() {
      Piece r;
      r.page = -1;
      r.row = 0;
      r.bits = 0;
      if (lane < n_chunk) {
        const int key = t * PA_KT + lane * R;             // < 2^31: tiles of at most len + 63 positions
        int logical, pos;
        bool in = true;
        if (p.page_idx != nullptr) {
          const int e = key >> p.ps_log2;
          const int pages = paged_pages(sq.len, p.ps_log2);
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
          if (r.bits != 0) r.page = p.table[(long long)b * p.table_stride + logical];
        }
      }
      return r;
    };
    Piece cur = look();
    bool first = true;
    int q_tile[2] = {-STAGES, -STAGES};   // the tiles that came with the queries in the two buffers
    int q_at = 0, stg = 0, i = 0;
    uint32_t phase = 0;                   // of the current round through the ring
    for (; i < n_mine; ++i) {
      // this tile's place in its item
      const int item = b * p.Hkv + g, cb = b, cg = g;
      const bool q_due = first, last = i + 1 == n_mine || t + 1 == sq.n_tiles;
      const int beg = u0 + i - t, end = beg + sq.n_tiles;   // the item's span in the order of all tiles
      // step to the next tile and start its look-up before waiting for a free stage
      first = false;
      if (++t == sq.n_tiles) {
        t = 0;
        first = true;
        if (++g == p.Hkv) {
          g = 0;
          b = min(b + 1, p.B - 1);   // (the last step is past the share's end)
          sq = pa_tiles(p, next_len);
          next_len = b + 1 < p.B ? pa_len(p, b + 1) : 0;
        }
      }
      Piece nxt = cur;
      if (i + 1 < n_mine) nxt = look();
      if (i >= STAGES) ok = mbar_wait(&empty[stg], phase ^ 1u, &abort_flag, p.status, 603);
      if (q_due) {   // the queries two items ago must have been taken: their tile released
        const int back = i - q_tile[q_at];
        if (ok && back < STAGES) {
          const int qs = stg - back < 0 ? stg - back + STAGES : stg - back;
          ok = mbar_wait(&empty[qs], stg - back < 0 ? phase ^ 1u : phase, &abort_flag, p.status, 608);
        }
        q_tile[q_at] = i;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      int page = p.n_pages;                 // out of range: zeros
      if (cur.bits != 0) {
        if (cur.page >= 0 && cur.page < p.n_pages) {
          page = cur.page;
        } else {
          report_error(p.status, DEV_ERR_BOUNDS, 602);
          cur.bits = 0;
        }
      }
      unsigned long long mask = cur.bits << (lane < n_chunk ? lane * R : 0);
      mask |= __shfl_xor_sync(0xffffffffu, mask, 1);
      mask |= __shfl_xor_sync(0xffffffffu, mask, 2);
      uint8_t* kt = ring + stg * S::STAGE;
      if (lane == 0) {
        PaMeta& mt = metas[grp][stg];
        mt.mask = mask;
        mt.last = last ? 1 : 0;
        if (last) {
          mt.item = item;
          mt.cut = beg < u0 ? 1 : (end > u1 ? 2 : 0);
          mt.ends = end <= u1 ? 1 : 0;
          mt.c0 = beg < t0 ? shares.owner(beg) : (int)blockIdx.x;
          mt.parts = (end > t1 ? shares.owner(end - 1) : (int)blockIdx.x) - mt.c0 + 1;
        }
        const uint32_t q_bytes = q_due ? (uint32_t)(p.G * D * 2) : 0u;
        mbar_arrive_expect_tx(&full[stg], S::STAGE + q_bytes);
        if (q_due)
          bulk_load(qbufs[grp][q_at], static_cast<const E*>(p.q) + cb * p.q_stride + (long long)cg * p.G * D, q_bytes,
                    &full[stg]);
      }
      __syncwarp();
      if (lane < n_chunk) {
        auto coord = [&](int dim) { return p.dim_row == dim ? cur.row : (p.dim_head == dim ? cg : page); };
        const int x1 = coord(1), x2 = coord(2), x3 = coord(3);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          tma_load_4d(kt + h * S::HALF + lane * R * 128, &mapK, &full[stg], h * 64, x1, x2, x3);
          tma_load_4d(kt + (NH + h) * S::HALF + lane * R * 128, &mapV, &full[stg], h * 64, x1, x2, x3);
        }
      }
      if (q_due) q_at ^= 1;
      cur = nxt;
      if (++stg == STAGES) {
        stg = 0;
        phase ^= 1u;
      }
    }
    // loads still in flight (all of them, if the consumers gave up) land before the CTA exits
    if (lane == 0) {
      for (int k = min(i, STAGES); k > 0; --k) {
        if (--stg < 0) {
          stg = STAGES - 1;
          phase ^= 1u;
        }
        mbar_wait(&full[stg], phase, nullptr, p.status, 604);
      }
    }
    return;
  }

  // ------------------------------ consumer warps ------------------------------
  const int wg = warp & 3;                   // warp within the group
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t ring_u32 = smem_u32(ring);
  const int k_row = wg * 16 + (lane & 7) + ((lane >> 4) & 1) * 8, k_chk = (lane >> 3) & 1;
  const int v_row = wg * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, v_chk = (lane >> 4) & 1;
  uint32_t merge_phase = 0, fin_phase = 0, phase = 0;
  const bool third = !Elem<E>::IS_F16 && p.out_dt == PDT_F32;   // a third part of the probabilities
  int stg = 0, i = 0;
  bool ok = true;
  // barriers of the group's and of all consumer warps; bounded, so that a warp that gave up
  // holds no one for long
  auto merge_sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&merge_bars[grp]);
    const bool r = mbar_wait(&merge_bars[grp], merge_phase & 1u, &abort_flag, p.status, 605);
    ++merge_phase;
    return __all_sync(0xffffffffu, r) != 0;
  };
  auto fin_sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&fin_bar);
    const bool r = mbar_wait(&fin_bar, fin_phase & 1u, &abort_flag, p.status, 607);
    ++fin_phase;
    return __all_sync(0xffffffffu, r) != 0;
  };
  for (int q_at = 0; i < n_mine && ok; q_at ^= 1) {   // one item's tiles in this group
    uint32_t qa[D / 16][2 * NHB];
    float m_run[NHB], l_run[NHB], o[NHB][D / 8][4];
#pragma unroll
    for (int hb = 0; hb < NHB; ++hb) {
      m_run[hb] = -INFINITY;
      l_run[hb] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) o[hb][j][0] = o[hb][j][1] = o[hb][j][2] = o[hb][j][3] = 0.f;
    }
    PaMeta mt;
    mt.item = mt.cut = mt.ends = mt.c0 = mt.parts = 0;
    for (bool first = true, last = false; !last; first = false, ++i) {
      ok = mbar_wait(&full[stg], phase, &abort_flag, p.status, 606);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const unsigned long long mask = metas[grp][stg].mask;
      last = metas[grp][stg].last != 0;
      if (last) mt = metas[grp][stg];
      if (first) {
        const E* q = reinterpret_cast<const E*>(qbufs[grp][q_at]);
#pragma unroll
        for (int hb = 0; hb < NHB; ++hb) {
          const bool row = hb * 8 + gq < p.G;
          const E* qr = q + (hb * 8 + gq) * D + 2 * tq;
#pragma unroll
          for (int st = 0; st < D / 16; ++st) {
            qa[st][2 * hb] = row ? *reinterpret_cast<const uint32_t*>(qr + st * 16) : 0u;
            qa[st][2 * hb + 1] = row ? *reinterpret_cast<const uint32_t*>(qr + st * 16 + 8) : 0u;
          }
        }
      }
      const uint32_t m16 = (uint32_t)(mask >> (wg * 16)) & 0xffffu;
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
        uint32_t pa[NHB][4], pb[NHB][2];   // p = hi + lo (+ the rest)
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
          if constexpr (Elem<E>::IS_F16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] *= P_SCALE;
          }
          pa[hb][0] = Elem<E>::pack(e[0], e[1]);
          pa[hb][2] = Elem<E>::pack(e[2], e[3]);
          const float2 h0 = Elem<E>::unpack(pa[hb][0]), h2 = Elem<E>::unpack(pa[hb][2]);
          const float r[4] = {e[0] - h0.x, e[1] - h0.y, e[2] - h2.x, e[3] - h2.y};
          pa[hb][1] = Elem<E>::pack(r[0], r[1]);
          pa[hb][3] = Elem<E>::pack(r[2], r[3]);
          if (third) {
            const float2 l0 = Elem<E>::unpack(pa[hb][1]), l2 = Elem<E>::unpack(pa[hb][3]);
            pb[hb][0] = Elem<E>::pack(r[0] - l0.x, r[1] - l0.y);
            pb[hb][1] = Elem<E>::pack(r[2] - l2.x, r[3] - l2.y);
          }
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
            if (third) {
              Elem<E>::mma(o[hb][j], pb[hb][0], 0u, pb[hb][1], 0u, f0, f1);
              Elem<E>::mma(o[hb][j + 1], pb[hb][0], 0u, pb[hb][1], 0u, f2, f3);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stg]);   // this warp is done with the stage
      if (++stg == STAGES) {
        stg = 0;
        phase ^= 1u;
      }
    }
    if (!ok) break;

    // the item's tiles in this group are done: the four warps' states through shared memory,
    // merged by 4 values per thread into the result or the group's part
    constexpr int QUADS = D / 4;
    // a part of an item shared with other CTAs of which this group has all that is here (the
    // end in the first group, the beginning in the last) leaves at once, while the rest goes on
    const bool early =
        mt.parts > 1 && (mt.cut == 1 ? grp == 0 && mt.c0 != (int)blockIdx.x && mt.ends : mt.cut == 2 && u1 == t1);
#pragma unroll
    for (int hb = 0; hb < NHB; ++hb) {
      float l = l_run[hb];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      float* row = mos[grp][wg][gq];
      if (tq == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m_run[hb], l);
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<float2*>(row + 8 * j + 2 * tq) =
            make_float2((o[hb][j][0] + o[hb][j][2]) * (1.f / P_SCALE), (o[hb][j][1] + o[hb][j][3]) * (1.f / P_SCALE));
      ok = merge_sync();
      if (!ok) break;
      for (int k = tid & 127; k < min(8, p.G - hb * 8) * QUADS; k += 128) {
        const int h = k / QUADS, quad = k % QUADS, hh = hb * 8 + h;   // query head within the group of heads
        PaAcc<D> a;
        a.clear();
#pragma unroll
        for (int w = 0; w < 4; ++w) a.add(mos[grp][w][h], quad);
        if (mt.cut == 0) pa_finish<D>(p, mt.item, hh, quad, a);
        else if (early) a.put(p.part + (((long long)blockIdx.x * 2 + mt.cut - 1) * p.G + hh) * LD, quad);
        else a.put(prows[grp][mt.cut - 1][hh], quad);
      }
      ok = merge_sync();   // the rows are free again, the part is whole
      if (!ok) break;
    }
    if (ok && mt.cut != 0 && wg == 0 && lane == 0) {
      PaPart pi;
      pi.item = mt.item;
      pi.c0 = mt.c0;
      pi.parts = mt.parts;
      if (early) {
        if (pa_claim(counted + mt.cut - 1) && pa_arrive(p, mt.c0, mt.parts))
          joins[mt.cut - 1] = pi;                    // joined when the CTA's groups are done
      } else {
        pinfo[grp][mt.cut - 1] = pi;
      }
    }
  }

  // ------------------------------ cut items ------------------------------
  // The groups' parts, in the order of the tiles; those of one item are neighbours and are merged.
  // At most one item began in an earlier CTA (slot 0) and at most one goes on in a later one (1).
  if (ok) ok = fin_sync();
  if (ok) {
    constexpr int QUADS = D / 4, NP = 2 * GROUPS;
    int item[NP], heads[NP], n_items = 0;   // heads: a part that is the first of its item
    bool far = false;
#pragma unroll
    for (int f = 0, prev = -1; f < NP; ++f) {
      item[f] = pinfo[f >> 1][f & 1].item;
      heads[f] = item[f] >= 0 && item[f] != prev ? 1 : 0;
      if (item[f] >= 0) {
        prev = item[f];
        far = far || pinfo[f >> 1][f & 1].parts > 1;
      }
      n_items += heads[f];
    }
    for (int k = tid; k < n_items * p.G * QUADS; k += CWARPS * 32) {
      const int hq = k / QUADS, quad = k % QUADS, hh = hq % p.G;
      int left = hq / p.G, first = 0;
#pragma unroll
      for (int f = 0; f < NP; ++f)
        if (heads[f] && left-- == 0) first = f;
      const PaPart pi = pinfo[first >> 1][first & 1];
      PaAcc<D> a;
      a.clear();
#pragma unroll
      for (int f = 0; f < NP; ++f)
        if (item[f] == pi.item) a.add(prows[f >> 1][f & 1][hh], quad);
      if (pi.parts == 1) pa_finish<D>(p, pi.item, hh, quad, a);
      else a.put(p.part + (((long long)blockIdx.x * 2 + (pi.c0 == (int)blockIdx.x ? 1 : 0)) * p.G + hh) * LD, quad);
    }
    if (far) {
      ok = fin_sync();
      if (ok && tid == 0) {
#pragma unroll 1
        for (int f = 0; f < NP; ++f) {
          const PaPart pi = pinfo[f >> 1][f & 1];
          const int slot = pi.c0 == (int)blockIdx.x ? 1 : 0;
          if (pi.item >= 0 && pi.parts > 1 && pa_claim(counted + slot)) {   // (several groups' parts of one item)
            if (pa_arrive(p, pi.c0, pi.parts)) joins[slot] = pi;
          }
        }
      }
      if (ok) ok = fin_sync();
    }
    // (the rings are scratch now: every load has landed and been read; the groups' part rows are
    // not, another warp may still be reading them)
    // two items of few parts are joined together
    int width[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      width[s] = joins[s].item < 0 ? 0 : pa_join_width<D, CWARPS>(joins[s].parts, p.G);
    const bool both = width[0] == 1 && width[1] == 1;
#pragma unroll 1
    for (int s = 0; s < 2 && ok; ++s)
      if (width[s] > 0 && !(both && s == 1))
        ok = pa_join<D, CWARPS>(p, joins + s, both ? 2 : 1, width[s], tid, reinterpret_cast<float*>(rings), fin_sync);
  }
  if (!ok && tid == 0) pa_arrive_rest(p, t0, t1, shares, counted);
}

}  // namespace hymba
