// Host side of the paged key-value cache: argument checks, workspace layout and launches
// (included by hymba.cu, whose helpers it uses).
#pragma once

namespace {

constexpr int PAGED_MAX_SELECT_WIDTH = 16384;   // one CTA ranks a sequence's pages in shared memory
constexpr int PSEL_TWO_PER_SM_WIDTH = 14000;    // up to here two such CTAs fit into an SM's shared memory

struct PagedWs {
  size_t part, total;
};
// The attention's parts follow the status word.  The other calls use the status word only.
PagedWs paged_layout(int head_dim, int group) {
  PagedWs w;
  w.part = 256;
  w.total = align256(w.part + (size_t)PA_MAX_GRID * 2 * group * (head_dim + 4) * 4);
  return w;
}

int check_paged_sizes(const hymba_paged_kv* kv) {
  if (kv == nullptr) return fail(HYMBA_ERR_INVALID_ARG, "paged cache is NULL");
  if (kv->dtype != HYMBA_DT_F16 && kv->dtype != HYMBA_DT_BF16)
    return fail(HYMBA_ERR_UNSUPPORTED, "paged cache type %d (16-bit types only)", kv->dtype);
  if (kv->head_dim != 64 && kv->head_dim != 128)
    return fail(HYMBA_ERR_UNSUPPORTED, "paged cache head_dim %d (64 or 128)", kv->head_dim);
  if (kv->page_size < 16 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1)))
    return fail(HYMBA_ERR_UNSUPPORTED, "page_size %d (16, 32, 64, 128 or 256)", kv->page_size);
  if (kv->n_pages < 1 || kv->n_kv_heads < 1 || kv->n_kv_heads > 1024)
    return fail(HYMBA_ERR_INVALID_ARG, "paged cache sizes");
  return HYMBA_OK;
}
// Rows, heads and pages by ascending stride, the order a tensor map wants its dimensions in.
struct PagedDims {
  long long stride[3];
  int size[3], box[3];
  int at_row, at_head;   // their places, 0..2
};
PagedDims paged_dims(const hymba_paged_kv* kv) {
  const long long s[3] = {kv->row_stride, kv->head_stride, kv->page_stride};
  const int n[3] = {kv->page_size, kv->n_kv_heads, kv->n_pages};
  int idx[3] = {0, 1, 2};
  std::stable_sort(idx, idx + 3, [&](int a, int b) { return s[a] < s[b]; });
  PagedDims r;
  for (int i = 0; i < 3; ++i) {
    r.stride[i] = s[idx[i]];
    r.size[i] = n[idx[i]];
    r.box[i] = idx[i] == 0 ? std::min(kv->page_size, PA_KT) : 1;
    if (idx[i] == 0) r.at_row = i;
    if (idx[i] == 1) r.at_head = i;
  }
  return r;
}
int check_paged(const hymba_paged_kv* kv, bool need_kv) {
  HY_TRY(check_paged_sizes(kv));
  if (need_kv) {
    if (kv->k == nullptr || kv->v == nullptr || !aligned16(kv->k) || !aligned16(kv->v))
      return fail(HYMBA_ERR_INVALID_ARG, "paged cache k/v NULL or not 16-byte aligned");
    // every row is a 16-byte aligned run of head_dim elements (TMA boxes, 8-byte stores)
    const long long strides[3] = {kv->page_stride, kv->head_stride, kv->row_stride};
    for (long long s : strides)
      if (s < kv->head_dim || s % 8 || s >= (1LL << 38))
        return fail(HYMBA_ERR_INVALID_ARG, "paged cache stride %lld (a multiple of 8, at least head_dim)", s);
    const PagedDims o = paged_dims(kv);
    if (o.stride[1] % o.stride[0] || o.stride[2] % o.stride[1])
      return fail(HYMBA_ERR_INVALID_ARG, "paged cache strides: each must be a multiple of the next smaller one");
  }
  if ((kv->k_lo == nullptr) != (kv->k_hi == nullptr) || !aligned16(kv->k_lo) || !aligned16(kv->k_hi))
    return fail(HYMBA_ERR_INVALID_ARG, "page bounds: both or neither, 16-byte aligned");
  return HYMBA_OK;
}
int check_table(const hymba_page_table* t) {
  if (t == nullptr || t->pages == nullptr || (reinterpret_cast<uintptr_t>(t->pages) & 3u) || t->batch < 1 ||
      t->batch > (1 << 20) || t->width < 1 || t->stride < t->width)
    return fail(HYMBA_ERR_INVALID_ARG, "page table (NULL, misaligned, or sizes)");
  return HYMBA_OK;
}
int check_select(const hymba_paged_kv* kv, const hymba_page_table* table, int n_first, int n_last, int top_pages) {
  if (kv->k_lo == nullptr) return fail(HYMBA_ERR_INVALID_ARG, "page selection needs the cache's page bounds");
  if (table->width > PAGED_MAX_SELECT_WIDTH)
    return fail(HYMBA_ERR_UNSUPPORTED, "page selection over %d pages (at most %d)", table->width,
                PAGED_MAX_SELECT_WIDTH);
  if (n_first < 0 || n_last < 0 || top_pages < 1 || (long long)n_first + n_last > top_pages)
    return fail(HYMBA_ERR_INVALID_ARG, "top_pages %d with %d first and %d last", top_pages, n_first, n_last);
  return HYMBA_OK;
}
int check_paged_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u)) return fail(HYMBA_ERR_INVALID_ARG, "workspace");
  if (ws_bytes < need) return fail(HYMBA_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
  return HYMBA_OK;
}
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// positions that a table row can name, at most 2^31 - 1
inline int paged_cap(int width, int page_size) {
  return (int)std::min<long long>((long long)width * page_size, 0x7fffffff);
}
inline int log2_int(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// kernel launch by the pool's type and head_dim: F is a functor template over (type, D)
template <typename F>
int paged_dispatch(const hymba_paged_kv* kv, F&& f) {
  if (kv->dtype == HYMBA_DT_F16) {
    if (kv->head_dim == 64) return f(__half{}, std::integral_constant<int, 64>{});
    return f(__half{}, std::integral_constant<int, 128>{});
  }
  if (kv->head_dim == 64) return f(__nv_bfloat16{}, std::integral_constant<int, 64>{});
  return f(__nv_bfloat16{}, std::integral_constant<int, 128>{});
}

// Enqueue the append kernel; p holds everything but the pool's fields.
int launch_paged_append(const hymba_paged_kv* kv, PagedAppendParams& p, float rope_base, int sms, cudaStream_t st) {
  p.Hkv = kv->n_kv_heads;
  p.n_pages = kv->n_pages;
  p.ps_log2 = log2_int(kv->page_size);
  p.page_stride = kv->page_stride;
  p.head_stride = kv->head_stride;
  p.row_stride = kv->row_stride;
  if (p.k != nullptr) {
    p.pk = kv->k;
    p.pv = kv->v;
    p.k_lo = kv->k_lo;
    p.k_hi = kv->k_hi;
  }
  p.rotate = rope_base > 0.f ? 1 : 0;
  const int h2 = kv->head_dim / 2;
  if (p.rotate) {   // turn_j = base^(-j / h2) / (2 pi), its fraction in units of 2^-64 (80-bit floats)
    const long double step = std::exp2(-std::log2((long double)rope_base) / h2);
    long double t = 0.159154943091895335768883763372514362L;
    for (int j = 0; j < h2; ++j, t *= step) {
      const long double f = t < 1.L ? t : t - std::floor(t);
      p.turns[j] = (unsigned long long)(f * 18446744073709551616.0L);
    }
  }
  // the most runs there can be (only a bound: the kernel counts them): a sequence of n tokens touches at most (n + 2 ps - 2) / ps
  // pages, and no more than it has tokens
  long long runs = ((long long)p.T + (long long)p.B * (2 * kv->page_size - 2)) / kv->page_size;
  if (runs > p.T) runs = p.T;
  const bool step = p.cu_new == nullptr;
  const long long items = step ? (long long)p.B * (kv->head_dim / 8) * p.Hkv : runs * p.Hkv;
  if (items > 0x7fffffff) return fail(HYMBA_ERR_UNSUPPORTED, "%d tokens of %d sequences: too many for one call", p.T, p.B);
  const int threads = step ? PAP_STEP_THREADS : PAP_THREADS;
  const int blocks = step ? cdiv(items, threads) : (int)std::min<long long>(items, PAP_PER_SM * sms);
  const int esz = p.src == PDT_F32 ? 4 : 2, head_bytes = kv->head_dim * esz;
  const int row_bytes = ((p.q != nullptr ? p.G : 0) + (p.k != nullptr ? 2 : 0)) * head_bytes;
  // a stage: one 4-pair item per consumer thread, in whole boxes, within its bytes
  p.chunk = std::max(PAP_BOX, std::min({kv->page_size, PAP_CONSUMERS * 8 / kv->head_dim,
                                        PAP_STAGE_BYTES / row_bytes / PAP_BOX * PAP_BOX}));
  const size_t smem = step ? 0 : (size_t)PAP_STAGES * p.chunk * row_bytes;
  // tensor maps of the source rows [T, heads * D], boxes of one head
  CUtensorMap mk, mv, mq;
  auto map_rows = [&](CUtensorMap* m, const void* base, int heads, long long stride) {
    const CUtensorMapDataType dt = p.src == PDT_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : p.src == PDT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t dims[2] = {(uint64_t)heads * kv->head_dim, (uint64_t)p.T};
    const uint64_t str[1] = {(uint64_t)stride * esz};
    const uint32_t box[2] = {(uint32_t)kv->head_dim, (uint32_t)PAP_BOX};
    return make_map(m, base, dt, 2, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  if (!step) {
    if (p.n_slices > 1) return fail(HYMBA_ERR_UNSUPPORTED, "split-K slices go with one token per sequence");
    if (p.k != nullptr) {
      HY_TRY(map_rows(&mk, p.k, p.Hkv, p.k_stride));
      HY_TRY(map_rows(&mv, p.v, p.Hkv, p.v_stride));
    }
    if (p.q != nullptr) HY_TRY(map_rows(&mq, p.q, p.Hkv * p.G, p.q_stride));
    if (p.k == nullptr) mk = mv = mq;
    if (p.q == nullptr) mq = mk;
  }
  return paged_dispatch(kv, [&](auto e, auto d) {
    using E = decltype(e);
    constexpr int D = decltype(d)::value;
    auto run = [&](auto src) {
      constexpr int SRC = decltype(src)::value;
      if (step) {
        prof_begin("paged_append", st);
        HY_CUDA(launch_pdl(paged_append_step_kernel<E, D, SRC>, dim3((unsigned)blocks), dim3(threads), 0, st, p));
        prof_end(st);
        return (int)HYMBA_OK;
      }
      auto kern = paged_append_kernel<E, D, SRC>;
      static bool attr[64] = {false};
      int dcur = 0;
      HY_CUDA(cudaGetDevice(&dcur));
      if (!attr[dcur & 63]) {
        HY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PAP_SMEM_MAX));
        attr[dcur & 63] = true;
      }
      prof_begin("paged_append", st);
      HY_CUDA(launch_pdl(kern, dim3((unsigned)blocks), dim3(threads), smem, st, mk, mv, mq, p));
      prof_end(st);
      return (int)HYMBA_OK;
    };
    if (p.src == PDT_F32) return run(std::integral_constant<int, PDT_F32>{});
    if (p.src == PDT_F16) return run(std::integral_constant<int, PDT_F16>{});
    return run(std::integral_constant<int, PDT_BF16>{});
  });
}

template <typename E, int D, int NHB>
int launch_paged_attn_inst(const CUtensorMap& mk, const CUtensorMap& mv, const PagedAttnParams& p, int sms,
                           cudaStream_t st) {
  using S = PaShape<D, NHB>;
  static bool attr[64] = {false};
  int d = 0;
  HY_CUDA(cudaGetDevice(&d));
  auto kern = paged_attn_kernel<E, D, NHB>;
  if (!attr[d & 63]) {
    HY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM));
    attr[d & 63] = true;
  }
  const int grid = std::min(sms, PA_MAX_GRID);
  prof_begin("paged_attn", st);
  HY_CUDA(launch_pdl(kern, dim3(grid), dim3(S::THREADS), S::SMEM, st, mk, mv, p));
  prof_end(st);
  return HYMBA_OK;
}

// Enqueue the attention over a pool; p holds everything but the pool's and the workspace's fields.
int launch_paged_attn(const hymba_paged_kv* kv, PagedAttnParams& p, uint8_t* ws, const PagedWs& L, int sms,
                      cudaStream_t st) {
  p.Hkv = kv->n_kv_heads;
  p.n_pages = kv->n_pages;
  p.ps_log2 = log2_int(kv->page_size);
  p.cap = paged_cap(p.width, kv->page_size);
  p.part = reinterpret_cast<float*>(ws + L.part);
  // tiles are counted in 32 bits (2^31 of them are 16 TB of keys of one head)
  const long long reach = p.page_idx != nullptr ? std::min(p.top, p.width) : p.width;
  if ((double)p.B * p.Hkv * ((double)reach * kv->page_size / PA_KT + 2) >= 2147483648.0)
    return fail(HYMBA_ERR_UNSUPPORTED, "%d sequences of %lld pages: too many keys for one call", p.B, reach);
  CUtensorMap mk, mv;
  const PagedDims o = paged_dims(kv);
  p.dim_row = o.at_row + 1;
  p.dim_head = o.at_head + 1;
  const uint64_t dims[4] = {(uint64_t)kv->head_dim, (uint64_t)o.size[0], (uint64_t)o.size[1], (uint64_t)o.size[2]};
  const uint64_t str[3] = {(uint64_t)o.stride[0] * 2, (uint64_t)o.stride[1] * 2, (uint64_t)o.stride[2] * 2};
  const uint32_t box[4] = {64, (uint32_t)o.box[0], (uint32_t)o.box[1], (uint32_t)o.box[2]};
  const CUtensorMapDataType dt =
      kv->dtype == HYMBA_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  HY_TRY(make_map(&mk, kv->k, dt, 4, dims, str, box));
  HY_TRY(make_map(&mv, kv->v, dt, 4, dims, str, box));
  return paged_dispatch(kv, [&](auto e, auto d) {
    using E = decltype(e);
    constexpr int D = decltype(d)::value;
    return p.G <= 8 ? launch_paged_attn_inst<E, D, 1>(mk, mv, p, sms, st)
                    : launch_paged_attn_inst<E, D, 2>(mk, mv, p, sms, st);
  });
}

// Enqueue the selection; p holds everything but the pool's fields.
int launch_paged_select(const hymba_paged_kv* kv, PagedSelectParams& p, cudaStream_t st) {
  p.k_lo = kv->k_lo;
  p.k_hi = kv->k_hi;
  p.Hkv = kv->n_kv_heads;
  p.n_pages = kv->n_pages;
  p.ps_log2 = log2_int(kv->page_size);
  p.cap = paged_cap(p.width, kv->page_size);
  const long long lists = (long long)p.B * p.Hkv;
  return paged_dispatch(kv, [&](auto e, auto d) {
    auto kern = paged_select_kernel<decltype(e), decltype(d)::value>;
    static bool attr[64] = {false};
    int dcur = 0;
    HY_CUDA(cudaGetDevice(&dcur));
    if (!attr[dcur & 63]) {
      HY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PAGED_MAX_SELECT_WIDTH * 8));
      attr[dcur & 63] = true;
    }
    // CTAs of a cluster share a list's pages; what they cannot share (the start, the ranking) makes
    // larger clusters worth less the shorter the lists are, and clusters that the device does not
    // hold at once come in a second wave.  So: the largest cluster that leaves at least 64 pages to a
    // CTA, while no more than n + n width / 4096 of them are needed, n being what the device holds:
    // 33, 71 and 148 clusters of 8, 4 and 2 on a B200 (two CTAs per SM), half of that for tables of
    // more than 14000 pages (the keys of the widest take 128 KB of every CTA's SM), and at most two
    // such waves, or four of the halves.  Measured (us, all lists full | lengths spread):
    //   lists x pages    of 8            of 4            of 2            of 1
    //    60 x  1024      17.4 |  15.8    11.7 |  11.2    12.2 |  12.0    16.9 |  16.6
    //   100 x  1024      23.8 |  22.0    17.9 |  16.0    15.0 |  14.6    17.1 |  18.5
    //   240 x  1024      52.8 |  42.4    38.4 |  28.7    32.3 |  24.3    26.0 |  21.7
    //    42 x  4096      31.5 |  22.3    29.4 |  24.3    37.4 |  32.1    63.7 |  49.3
    //   100 x  4096      56.8 |  43.6    51.8 |  40.4    48.4 |  44.9    69.0 |  69.5
    //   180 x  4096      92.3 |  67.3    81.0 |  57.3    88.0 |  56.5    83.1 |  77.4
    //    36 x 15000     116   |  76.7   134   |  79.0   132   | 130     232   | 231
    static std::atomic<int> resident[64][2][4];   // by device, table class, log2 of the cluster: 0 not asked yet
    const int wide = p.width > PSEL_TWO_PER_SM_WIDTH ? 1 : 0;
    int cluster = 8;
    for (int l = 3; cluster > 1; --l, cluster >>= 1) {
      if (p.width < 64 * cluster) continue;
      int n = resident[dcur & 63][wide][l].load(std::memory_order_relaxed);
      if (n == 0) {
        cudaLaunchAttribute dim{};
        dim.id = cudaLaunchAttributeClusterDimension;
        dim.val.clusterDim.x = cluster;
        dim.val.clusterDim.y = dim.val.clusterDim.z = 1;
        cudaLaunchConfig_t q{};
        q.gridDim = dim3((unsigned)cluster);
        q.blockDim = dim3(PSEL_THREADS);
        q.dynamicSmemBytes = (size_t)(wide ? PAGED_MAX_SELECT_WIDTH : PSEL_TWO_PER_SM_WIDTH) * 8;
        q.attrs = &dim;
        q.numAttrs = 1;
        HY_CUDA(cudaOccupancyMaxActiveClusters(&n, kern, &q));
        n = std::max(n, 1);
        resident[dcur & 63][wide][l].store(n, std::memory_order_relaxed);
      }
      if (lists <= n + std::min((long long)n * p.width / 4096, (long long)n * (wide ? 3 : 1))) break;
    }
    if (lists * cluster > 0x7fffffff) return fail(HYMBA_ERR_UNSUPPORTED, "batch too large");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(lists * cluster));
    cfg.blockDim = dim3(PSEL_THREADS);
    cfg.dynamicSmemBytes = (size_t)p.width * 8;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    prof_begin("paged_select", cfg.stream);
    HY_CUDA(cudaLaunchKernelEx(&cfg, kern, p, cluster));
    prof_end(cfg.stream);
    return (int)HYMBA_OK;
  });
}

int paged_group(const hymba_paged_kv* kv, int n_q_heads, int* group) {
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads || n_q_heads / kv->n_kv_heads > 16)
    return fail(HYMBA_ERR_UNSUPPORTED, "%d query heads over %d KV heads (1 to 16 per KV head)", n_q_heads,
                kv->n_kv_heads);
  *group = n_q_heads / kv->n_kv_heads;
  return HYMBA_OK;
}

// ---- a mixer's decode step over a paged cache -------------------------------------------
struct PagedDecode {
  const hymba_paged_kv* kv;
  const hymba_page_table* table;
  int top_pages;   // 0: every page
};
// Workspace after the decode step's own buffers (laid out as for one key: no key splits).
struct PagedDecodeWs {
  size_t q, part, idx, total;
};
DecodeWs paged_decode_base(const Dims& m, int B) { return decode_layout(m, B, true, 1); }
PagedDecodeWs paged_decode_layout(const Dims& m, int B, int top_pages) {
  PagedDecodeWs w;
  size_t off = paged_decode_base(m, B).total;
  auto take = [&](size_t bytes) { size_t o = off; off = align256(off + bytes); return o; };
  w.q = take((size_t)B * m.qw * 2);
  w.part = take((size_t)PA_MAX_GRID * 2 * (m.Hq / m.Hkv) * (m.D + 4) * 4);
  w.idx = take((size_t)B * m.Hkv * top_pages * 4);
  w.total = off;
  return w;
}
// first pages to select whatever their scores: those of the meta tokens
int paged_meta_pages(const hymba_paged_kv* kv, int n_meta) { return cdiv(n_meta, kv->page_size); }

int check_paged_decode(const PagedDecode& d, const hymba_layer_cfg* cfg) {
  HY_TRY(check_paged(d.kv, true));
  HY_TRY(check_table(d.table));
  if (d.kv->n_kv_heads != cfg->n_kv_heads || d.kv->head_dim != cfg->head_dim)
    return fail(HYMBA_ERR_INVALID_ARG, "paged cache of %d heads x %d for a layer of %d x %d", d.kv->n_kv_heads,
                d.kv->head_dim, cfg->n_kv_heads, cfg->head_dim);
  if (d.top_pages < 0 || (d.top_pages > 0 && !cfg->is_global))
    return fail(HYMBA_ERR_INVALID_ARG, "top_pages %d (page selection is for global layers)", d.top_pages);
  if (d.top_pages > 0) HY_TRY(check_select(d.kv, d.table, paged_meta_pages(d.kv, cfg->n_meta), 1, d.top_pages));
  return HYMBA_OK;
}

// RoPE and append of the new tokens from in_proj's split-K slices, the page selection, and the
// attention into o [B, Hq*D] fp32, on `st`.
int launch_paged_decode(const PagedDecode& d, const hymba_layer_cfg* cfg, const Dims& m, int B, const int* positions,
                        const float* proj, int n_slices, bool own_kv, const PagedDecodeWs& L, uint8_t* ws, float* o,
                        const DeviceInfo& dev, cudaStream_t st) {
  const hymba_page_table* t = d.table;
  DevStatus* status = reinterpret_cast<DevStatus*>(ws);
  PagedAppendParams ap{};
  ap.q = proj;
  ap.k = own_kv ? proj + m.qw : nullptr;
  ap.v = own_kv ? proj + m.qw + m.kvw : nullptr;
  ap.q_stride = ap.k_stride = ap.v_stride = m.P;
  ap.src = PDT_F32;
  ap.n_slices = n_slices;
  ap.slice_stride = (long long)B * m.P;
  ap.q_out = ws + L.q;
  ap.start = positions;
  ap.table = t->pages; ap.table_stride = t->stride; ap.width = t->width;
  ap.B = ap.T = B;
  ap.G = m.Hq / m.Hkv;
  ap.clear = status->parts;
  ap.n_clear = PA_PART_WORDS;
  ap.status = status;
  HY_TRY(launch_paged_append(d.kv, ap, cfg->rope_base, dev.sms, st));
  if (d.top_pages > 0) {
    PagedSelectParams sp{};
    sp.q = ws + L.q; sp.q_stride = m.qw;
    sp.table = t->pages; sp.table_stride = t->stride; sp.width = t->width;
    sp.lens = positions;
    sp.len_add = 1;
    sp.B = B; sp.G = ap.G;
    sp.n_first = paged_meta_pages(d.kv, m.M); sp.n_last = 1; sp.top = d.top_pages;
    sp.page_idx = reinterpret_cast<int*>(ws + L.idx);
    sp.status = status;
    HY_TRY(launch_paged_select(d.kv, sp, st));
  }
  PagedAttnParams p{};
  p.q = ws + L.q; p.q_stride = m.qw;
  p.out = o; p.out_dt = PDT_F32; p.out_stride = m.qw;
  p.table = t->pages; p.table_stride = t->stride; p.width = t->width;
  p.lens = positions;
  p.len_add = 1;
  p.page_idx = d.top_pages > 0 ? reinterpret_cast<const int*>(ws + L.idx) : nullptr;
  p.top = d.top_pages;
  p.B = B; p.Hq = m.Hq; p.G = ap.G;
  p.M = cfg->is_global ? 0 : m.M;
  p.W = cfg->is_global ? 0 : m.W;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)m.D));
  p.status = status;
  PagedWs aw;
  aw.part = L.part;
  aw.total = L.total;
  return launch_paged_attn(d.kv, p, ws, aw, dev.sms, st);
}

}  // namespace

extern "C" {

int hymba_paged_workspace_size(const hymba_paged_kv* kv, int batch, int n_q_heads, int max_pages, size_t* bytes) {
  HY_TRY(check_paged_sizes(kv));
  int G = 0;
  HY_TRY(paged_group(kv, n_q_heads, &G));
  if (bytes == nullptr || batch < 1 || max_pages < 1) return fail(HYMBA_ERR_INVALID_ARG, "paged workspace arguments");
  *bytes = paged_layout(kv->head_dim, G).total;   // (what the calls need does not grow with the batch)
  return HYMBA_OK;
}

int hymba_paged_append(const hymba_paged_kv* kv, const hymba_page_table* table, const int* start, const int* cu_new,
                       int n_tokens, int src_dtype, const void* k, long long k_stride, const void* v,
                       long long v_stride, const void* q, long long q_stride, int n_q_heads, void* q_out,
                       float rope_base, void* ws, size_t ws_bytes, hymba_stream stream) {
  const bool has_kv = k != nullptr;
  HY_TRY(check_paged(kv, has_kv));
  HY_TRY(check_table(table));
  HY_TRY(check_paged_ws(ws, ws_bytes, 256));
  if (src_dtype != HYMBA_DT_F32 && src_dtype != HYMBA_DT_BF16 && src_dtype != HYMBA_DT_F16)
    return fail(HYMBA_ERR_UNSUPPORTED, "source type %d", src_dtype);
  if (start == nullptr || !aligned4(start) || !aligned4(cu_new)) return fail(HYMBA_ERR_INVALID_ARG, "start / cu_new");
  if (n_tokens < 0 || (cu_new == nullptr && n_tokens != table->batch))
    return fail(HYMBA_ERR_INVALID_ARG, "n_tokens %d for a batch of %d", n_tokens, table->batch);
  if (has_kv != (v != nullptr)) return fail(HYMBA_ERR_INVALID_ARG, "k and v: both or neither");
  if ((q == nullptr) != (q_out == nullptr)) return fail(HYMBA_ERR_INVALID_ARG, "q and q_out: both or neither");
  if (!has_kv && q == nullptr) return fail(HYMBA_ERR_INVALID_ARG, "neither keys nor queries");
  if (!(rope_base >= 0.f) || std::isinf(rope_base)) return fail(HYMBA_ERR_INVALID_ARG, "rope_base %g", rope_base);
  const int vec = src_dtype == HYMBA_DT_F32 ? 4 : 8;   // 16 bytes
  int G = 1;
  if (q != nullptr) HY_TRY(paged_group(kv, n_q_heads, &G));
  struct { const void* p; long long s; long long w; const char* n; } rows[3] = {
      {k, k_stride, (long long)kv->n_kv_heads * kv->head_dim, "k"},
      {v, v_stride, (long long)kv->n_kv_heads * kv->head_dim, "v"},
      {q, q_stride, (long long)G * kv->n_kv_heads * kv->head_dim, "q"}};
  for (const auto& r : rows)
    if (r.p != nullptr && (!aligned16(r.p) || r.s < r.w || r.s % vec))
      return fail(HYMBA_ERR_INVALID_ARG, "%s rows: not 16-byte aligned, or stride %lld", r.n, r.s);
  if (!aligned16(q_out)) return fail(HYMBA_ERR_INVALID_ARG, "q_out not 16-byte aligned");
  if (q != nullptr && q == q_out &&
      (src_dtype != kv->dtype || (n_tokens > 1 && q_stride != (long long)n_q_heads * kv->head_dim)))
    return fail(HYMBA_ERR_INVALID_ARG, "queries in place: of another type than the pool, or rows not contiguous");
  DeviceInfo* dev = nullptr;
  HY_TRY(device_info(&dev));
  if (n_tokens == 0) return HYMBA_OK;
  PagedAppendParams p{};
  p.q = q; p.k = k; p.v = v;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.src = src_dtype;
  p.n_slices = 1;
  p.q_out = q_out;
  p.start = start;
  p.cu_new = cu_new;
  p.table = table->pages; p.table_stride = table->stride; p.width = table->width;
  p.B = table->batch; p.T = n_tokens; p.G = G;
  p.status = reinterpret_cast<DevStatus*>(ws);
  return launch_paged_append(kv, p, rope_base, dev->sms, (cudaStream_t)stream);
}

int hymba_paged_select(const hymba_paged_kv* kv, const hymba_page_table* table, const int* seq_lens, const void* q,
                       long long q_stride, int n_q_heads, int n_first, int n_last, int top_pages, int* page_idx,
                       void* ws, size_t ws_bytes, hymba_stream stream) {
  HY_TRY(check_paged(kv, false));
  HY_TRY(check_table(table));
  int G = 0;
  HY_TRY(paged_group(kv, n_q_heads, &G));
  HY_TRY(check_select(kv, table, n_first, n_last, top_pages));
  if (seq_lens == nullptr || !aligned4(seq_lens) || page_idx == nullptr || !aligned4(page_idx) || q == nullptr ||
      !aligned16(q) || q_stride < (long long)n_q_heads * kv->head_dim || q_stride % 8)
    return fail(HYMBA_ERR_INVALID_ARG, "seq_lens / page_idx / q");
  HY_TRY(check_paged_ws(ws, ws_bytes, 256));
  DeviceInfo* dev = nullptr;
  HY_TRY(device_info(&dev));
  PagedSelectParams p{};
  p.q = q; p.q_stride = q_stride;
  p.table = table->pages; p.table_stride = table->stride; p.width = table->width;
  p.lens = seq_lens;
  p.B = table->batch; p.G = G;
  p.n_first = n_first; p.n_last = n_last; p.top = top_pages;
  p.page_idx = page_idx;
  p.status = reinterpret_cast<DevStatus*>(ws);
  return launch_paged_select(kv, p, (cudaStream_t)stream);
}

int hymba_paged_attention(const hymba_paged_kv* kv, const hymba_page_table* table, const int* seq_lens, const void* q,
                          long long q_stride, int n_q_heads, float scale, int n_meta, int window, const int* page_idx,
                          int top_pages, void* out, int out_dtype, long long out_stride, float* lse, void* ws,
                          size_t ws_bytes, hymba_stream stream) {
  HY_TRY(check_paged(kv, true));
  HY_TRY(check_table(table));
  int G = 0;
  HY_TRY(paged_group(kv, n_q_heads, &G));
  const long long width = (long long)n_q_heads * kv->head_dim;
  if (seq_lens == nullptr || !aligned4(seq_lens) || q == nullptr || !aligned16(q) || q_stride < width || q_stride % 8)
    return fail(HYMBA_ERR_INVALID_ARG, "seq_lens / q");
  if (out_dtype != HYMBA_DT_F32 && out_dtype != HYMBA_DT_BF16 && out_dtype != HYMBA_DT_F16)
    return fail(HYMBA_ERR_UNSUPPORTED, "output type %d", out_dtype);
  if (out == nullptr || out == q || !aligned16(out) || out_stride < width || out_stride % 8 || !aligned4(lse))
    return fail(HYMBA_ERR_INVALID_ARG, "out (NULL, q itself, misaligned, or its stride) / lse");
  if (!std::isfinite(scale)) return fail(HYMBA_ERR_INVALID_ARG, "scale %g", scale);
  if (n_meta < 0 || window < 0 || (window == 0 && n_meta > 0))
    return fail(HYMBA_ERR_INVALID_ARG, "n_meta %d, window %d (meta tokens go with a window)", n_meta, window);
  if (page_idx != nullptr && (window > 0 || top_pages < 1 || !aligned4(page_idx)))
    return fail(HYMBA_ERR_INVALID_ARG, "a page list goes without a window, with top_pages >= 1");
  const PagedWs L = paged_layout(kv->head_dim, G);
  HY_TRY(check_paged_ws(ws, ws_bytes, L.total));
  DeviceInfo* dev = nullptr;
  HY_TRY(device_info(&dev));
  PagedAttnParams p{};
  p.q = q; p.q_stride = q_stride;
  p.out = out; p.out_dt = out_dtype; p.out_stride = out_stride;
  p.lse = lse;
  p.table = table->pages; p.table_stride = table->stride; p.width = table->width;
  p.lens = seq_lens;
  p.page_idx = page_idx; p.top = top_pages;
  p.B = table->batch; p.Hq = n_q_heads; p.G = G;
  p.M = n_meta; p.W = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.status = reinterpret_cast<DevStatus*>(ws);
  return launch_paged_attn(kv, p, static_cast<uint8_t*>(ws), L, dev->sms, (cudaStream_t)stream);
}

}  // extern "C"
