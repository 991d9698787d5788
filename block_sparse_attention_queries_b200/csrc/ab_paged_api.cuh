// C ABI of the norm and rotation and of the paged cache (declared in
// include/ab.h): argument checks, workspace layout, launches.  Included by
// ab_api.cu, whose helpers it uses.
#pragma once

namespace {

int log2_of(int x) {
  int k = 0;
  while ((1 << k) < x) ++k;
  return k;
}

// SMs of the current device (0: unknown), read from the driver once per device.
int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kMaxDevices && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 0;
  if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Launch of a kernel that begins with pdl_wait: it may be started while the
// kernel before it in the stream still runs.
template <typename... Params, typename... Args>
ab_status launch_after(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, Params(args)...) != cudaSuccess) {
    cudaGetLastError();
    return AB_ERR_CUDA;
  }
  return AB_OK;
}

// ------------------------------------------------------ norm and rotation
constexpr int64_t kRopeSplit = int64_t(1) << 22;     // values of q
constexpr int64_t kRopeMaxUnits = int64_t(1) << 29;  // positions in the list of units stay in 32 bits

ab_status check_norm_rope(const ab_norm_rope* nr) {
  if (!nr) return AB_ERR_INVALID_ARG;
  if (nr->norm < 0 || nr->norm > 2 || (nr->interleaved != 0 && nr->interleaved != 1)) return AB_ERR_INVALID_ARG;
  if (!(nr->eps >= 0.f) || nr->n_pos < 0) return AB_ERR_INVALID_ARG;
  if ((nr->cos_table == nullptr) != (nr->sin_table == nullptr)) return AB_ERR_INVALID_ARG;
  // a position out of range is reported by a token that has copied row 0
  if (nr->cos_table && nr->n_pos < 1) return AB_ERR_INVALID_ARG;
  const void* ptrs[] = {nr->wq, nr->wk, nr->cos_table, nr->sin_table};
  for (const void* q : ptrs)
    if (!aligned16(q)) return AB_ERR_INVALID_ARG;
  return AB_OK;
}

// Strides keep every head row 16-byte aligned; a stride of a dimension of
// size 1 is never used.
ab_status check_tokens(const ab_tokens* x, int64_t nb, int64_t nt, int64_t nh) {
  if (!x || !x->ptr || !aligned16(x->ptr)) return AB_ERR_INVALID_ARG;
  if ((nb > 1 && x->batch % 8 != 0) || (nt > 1 && x->token % 8 != 0) || (nh > 1 && x->head % 8 != 0))
    return AB_ERR_INVALID_ARG;
  return AB_OK;
}

TokenView view_of(const ab_tokens* x) {
  return TokenView{static_cast<const __nv_bfloat16*>(x->ptr), x->batch, x->token, x->head};
}

// Heads that one CTA can take for norm 2: 16 warps of 32 / (d/8) rows, 8 rows a lane.
int rope_max_heads(int d) { return 16 * (256 / d) * kRopeRowsMany; }

// tokens[k] = 0 where the k-th of q, k, v is not wanted.
ab_status launch_norm_rope(NormRopeArgs a, int d, const ab_norm_rope* nr, cudaStream_t st) {
  const int sms = sm_count();
  if (!sms) return AB_ERR_CUDA;
  int heads = 0, tokens = 0;
  int64_t all = 0;
  a.merged = true;
  for (int k = 0; k < 3; ++k) {
    if (!a.tokens[k]) continue;
    heads = a.heads[k] > heads ? a.heads[k] : heads;
    if (tokens && a.tokens[k] != tokens) a.merged = false;
    tokens = a.tokens[k];
    all += a.tokens[k];
  }
  if (all > kRopeMaxUnits) return AB_ERR_UNSUPPORTED;
  const int rows = 256 / d;  // head rows a warp covers at once
  auto go = [&](auto kern, int64_t blocks, int threads, int smem) -> ab_status {
    if (smem > 48 * 1024 && set_smem(kern, smem) != cudaSuccess) return AB_ERR_CUDA;
    return launch_after(kern, dim3(unsigned(blocks)), threads, smem, st, a);
  };
  using T128 = std::integral_constant<int, 128>;
  using T64 = std::integral_constant<int, 64>;
  auto by_type = [&](auto f) -> ab_status {
    if (d == 128) return nr->interleaved ? f(T128{}, std::true_type{}) : f(T128{}, std::false_type{});
    return nr->interleaved ? f(T64{}, std::true_type{}) : f(T64{}, std::false_type{});
  };
  if (nr->norm == kNormToken) {
    a.merged = false;
    const bool many = heads > 16 * rows * kRopeRows;
    const int nv = many ? kRopeRowsMany : kRopeRows, stages = many ? kRopeStagesMany : kRopeStages;
    const int threads = 32 * ((heads + rows * nv - 1) / (rows * nv));
    // Key heads a third of the queries' or fewer: launches of their own, with as many
    // warps as each needs (with their page means: 44 thousand tokens of 32 + 8 + 8
    // heads 240 us against 315 in one launch, of 40 + 4 + 4 235 against 373, of 32 + 4
    // + 4 heads of 64 136 against 155; of 16 + 8 + 8 178 against 180, of 24 + 12 + 12
    // 286 against 279), once the queries fill the GPU a few times (1500 tokens of 32 +
    // 8 + 8 heads 13.5 against 15.6, but 600 10.2 against 8.7, and 1500 with heads of
    // 64 11.1 against 10.4).
    const int per_warp = rows * nv, warps_kv = (a.heads[1] + per_warp - 1) / per_warp;
    if (a.tokens[0] && all > a.tokens[0] && 32 * warps_kv < threads && 3 * a.heads[1] <= a.heads[0] &&
        int64_t(a.tokens[0]) * a.heads[0] * d >= kRopeSplit) {
      NormRopeArgs q = a, kv = a;
      q.tokens[1] = q.tokens[2] = kv.tokens[0] = 0;
      const ab_status s = launch_norm_rope(q, d, nr, st);
      return s == AB_OK ? launch_norm_rope(kv, d, nr, st) : s;
    }
    const int smem = rope_smem_bytes(nv, stages, threads);
    // resident CTAs: as many as shared memory and the registers (96 a thread) allow
    int per_sm = 640 / threads;
    if (per_sm > 220 * 1024 / smem) per_sm = 220 * 1024 / smem;
    if (per_sm < 1) per_sm = 1;
    int units = 0;
    for (int k = 0; k < 3; ++k) a.units[k] = units += a.tokens[k];
    a.n_units = units;
    const int64_t blocks = units < int64_t(sms) * per_sm ? units : int64_t(sms) * per_sm;
    return by_type([&](auto dd, auto il) -> ab_status {
      constexpr int D = decltype(dd)::value;
      constexpr bool I = decltype(il)::value;
      return many ? go(token_norm_rope_kernel<D, I, kRopeRowsMany, kRopeStagesMany>, blocks, threads, smem)
                  : go(token_norm_rope_kernel<D, I, kRopeRows, kRopeStages>, blocks, threads, smem);
    });
  }
  constexpr int threads = kRopeThreads, warps = threads / 32;
  constexpr int smem = rope_smem_bytes(kRopeRows, kRopeStages, threads);
  const int64_t resident = int64_t(sms) * 5;  // CTAs: 41 KB, 96 registers a thread
  // A unit takes all heads of its token where that leaves every warp four units,
  // else one step of them: 32760 tokens of 40 heads, rotation alone, 346 us
  // against 376 in single steps; 233 tokens of 32 + 8 + 8 heads with their plan
  // 12.1 us in single steps against 13.4.
  const bool whole = all >= 4 * resident * warps;
  int64_t units = 0;
  for (int k = 0; k < 3; ++k) {
    const int steps = (a.heads[k] + rows * kRopeRows - 1) / (rows * kRopeRows);
    a.steps[k] = whole ? steps : 1;
    const int groups = a.tokens[k] ? (whole ? 1 : steps) : 0;
    units += a.merged ? groups : int64_t(a.tokens[k]) * groups;
    if (units > kRopeMaxUnits) return AB_ERR_UNSUPPORTED;
    a.units[k] = int(units);
  }
  if (a.merged) units *= tokens;
  if (units > kRopeMaxUnits) return AB_ERR_UNSUPPORTED;
  a.n_units = int(units);
  int64_t blocks = (units + warps - 1) / warps;
  blocks = blocks < resident ? blocks : resident;
  return by_type([&](auto dd, auto il) -> ab_status {
    constexpr int D = decltype(dd)::value;
    constexpr bool I = decltype(il)::value;
    return nr->norm == kNormHead ? go(norm_rope_kernel<D, true, I>, blocks, threads, smem)
                                 : go(norm_rope_kernel<D, false, I>, blocks, threads, smem);
  });
}

// Bytes [first, last) that tokens reach over.
struct Span {
  uintptr_t lo, hi;
};
Span span_of(const ab_tokens* x, int64_t nb, int64_t nt, int64_t nh, int d) {
  const int64_t n[3] = {nb, nt, nh}, s[3] = {x->batch, x->token, x->head};
  int64_t lo = 0, hi = d;
  for (int k = 0; k < 3; ++k)
    if (n[k] > 1) (s[k] < 0 ? lo : hi) += (n[k] - 1) * s[k];
  const uintptr_t p = reinterpret_cast<uintptr_t>(x->ptr);
  return {p + uintptr_t(lo * 2), p + uintptr_t(hi * 2)};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
Span span_of(const void* p, int64_t elements) {
  const uintptr_t q = reinterpret_cast<uintptr_t>(p);
  return {q, q + uintptr_t(elements) * 2};
}

void set_norm_rope(NormRopeArgs* a, const ab_norm_rope* nr) {
  a->w[0] = nr->norm ? nr->wq : nullptr;
  a->w[1] = nr->norm ? nr->wk : nullptr;
  a->cos_t = nr->cos_table;
  a->sin_t = nr->sin_table;
  a->n_pos = nr->n_pos;
  a->eps = nr->eps;
}

// Arguments of the dense call.
ab_status prepare_norm_rope(const ab_params& p, const ab_norm_rope* nr, const ab_tokens* q, const ab_tokens* k,
                            const ab_tokens* v, const int32_t* pos_q, const int32_t* pos_k, void* Q, void* K, void* V,
                            NormRopeArgs* a) {
  const ab_status s = check_norm_rope(nr);
  if (s != AB_OK) return s;
  if (!q && !k && !v) return AB_ERR_INVALID_ARG;
  const int Lk = p.L_kv > 0 ? p.L_kv : p.L;
  const ab_tokens* in[3] = {q, k, v};
  void* out[3] = {Q, K, V};
  const int32_t* pos[2] = {pos_q, pos_k};
  *a = NormRopeArgs{};
  for (int x = 0; x < 3; ++x) {
    const int len = x == 0 ? p.L : Lk;
    if (!in[x]) continue;
    if (check_tokens(in[x], p.B, len, p.H) != AB_OK || !out[x] || !aligned16(out[x])) return AB_ERR_INVALID_ARG;
    if (x < 2) {
      if (pos[x] && !aligned16(pos[x])) return AB_ERR_INVALID_ARG;
      if (nr->cos_table && !pos[x] && len > nr->n_pos) return AB_ERR_INVALID_ARG;
      a->pos[x] = pos[x];
    }
    if (int64_t(p.B) * len > kRopeMaxUnits) return AB_ERR_UNSUPPORTED;
    a->heads[x] = p.H;
    a->len[x] = len;
    a->tokens[x] = p.B * len;
    a->in[x] = view_of(in[x]);
    a->out[x] = static_cast<__nv_bfloat16*>(out[x]);
  }
  if (p.H > rope_max_heads(p.d)) return AB_ERR_UNSUPPORTED;
  for (int x = 0; x < 3; ++x) {
    if (!in[x]) continue;
    const Span o = span_of(out[x], int64_t(a->tokens[x]) * p.H * p.d);
    for (int y = 0; y < 3; ++y) {
      if (in[y] && overlap(o, span_of(in[y], p.B, a->len[y], p.H, p.d))) return AB_ERR_INVALID_ARG;
      if (in[y] && y < x && overlap(o, span_of(out[y], int64_t(a->tokens[y]) * p.H * p.d))) return AB_ERR_INVALID_ARG;
    }
  }
  set_norm_rope(a, nr);
  return AB_OK;
}

// ---------------------------------------------------------- the paged cache
ab_status check_paged(const ab_paged_params* p) {
  if (!p) return AB_ERR_INVALID_ARG;
  if (p->S < 1 || p->Hq < 1 || p->Hkv < 1 || p->num_pages < 1 || p->max_pages < 1 || p->recent < 0)
    return AB_ERR_INVALID_ARG;
  if (p->Hq % p->Hkv != 0) return AB_ERR_INVALID_ARG;
  if (!(p->keep_ratio > 0.f) || !(p->keep_ratio <= 1.f)) return AB_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return p->d > 0 ? AB_ERR_UNSUPPORTED : AB_ERR_INVALID_ARG;
  if (p->page != 16 && p->page != 32 && p->page != 64) return p->page > 0 ? AB_ERR_UNSUPPORTED : AB_ERR_INVALID_ARG;
  if (int64_t(p->max_pages) * p->page > (int64_t(1) << 24)) return AB_ERR_INVALID_ARG;
  if (int64_t(p->num_pages) * p->page > INT_MAX || int64_t(p->num_pages) * p->Hkv > INT_MAX) return AB_ERR_INVALID_ARG;
  if (p->S > kMaxSeqs || p->Hkv > 65535 || p->Hq / p->Hkv > kMaxGroup || int64_t(p->S) * p->Hkv > kShareMaxUnits)
    return AB_ERR_UNSUPPORTED;
  // positions in the list of all tiles of 64 keys, and their cost, stay in 32 bits
  if (int64_t(p->S) * p->Hkv * ((int64_t(p->max_pages) * p->page + 63) / 64) > INT_MAX / 4)
    return AB_ERR_UNSUPPORTED;
  return AB_OK;
}

bool any_bad(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (!q || !aligned16(q)) return true;
  return false;
}

PagedView paged_view(const ab_paged_params* p, const int32_t* table, const int32_t* lens, const int32_t* cu_new, int T) {
  PagedView v{};
  v.table = table; v.lens = lens; v.cu_new = cu_new; v.T = T;
  v.S = p->S; v.Hkv = p->Hkv; v.G = p->Hq / p->Hkv;
  v.page = p->page; v.page_shift = log2_of(p->page); v.num_pages = p->num_pages; v.max_pages = p->max_pages;
  return v;
}

struct PagedWorkspace {
  size_t off_scores, off_part;                     // select
  size_t off_part_o, off_ml;            // attention (its first bytes: DecMeta)
  size_t select, attend;                // bytes of each
};

PagedWorkspace paged_workspace(const ab_paged_params* p) {
  PagedWorkspace w{};
  const size_t rows = size_t(p->S) * p->Hq;
  const size_t chunks = (size_t(p->max_pages) + kSelPages - 1) / kSelPages;
  w.off_part = align256(w.off_scores + rows * ((size_t(p->max_pages) + 3) / 4 * 16));
  w.select = align256(w.off_part + rows * chunks * 8);
  const size_t heads = p->Hq / p->Hkv > 8 ? 16 : 8;
  w.off_part_o = align256(kDecMaxParts * sizeof(DecMeta));
  w.off_ml = align256(w.off_part_o + size_t(kDecMaxParts) * 2 * heads * p->d * 4);
  w.attend = align256(w.off_ml + size_t(kDecMaxParts) * 2 * heads * 8);
  return w;
}

// Rows of Q: with cu_new the tokens' rows, else one row per sequence.
ab_status check_rows(const ab_paged_params* p, const int32_t* cu_new, int32_t T) {
  if (cu_new ? (!aligned16(cu_new) || T < 1) : T != p->S) return AB_ERR_INVALID_ARG;
  return AB_OK;
}

// O is written while other CTAs still read queries, keys and values.
bool output_overlaps(const ab_paged_params* p, int32_t T, const void* Q, const void* K, const void* V, const void* O) {
  const int64_t cache = int64_t(p->num_pages) * p->Hkv * p->page * p->d;
  const Span o = span_of(O, int64_t(p->S) * p->Hq * p->d);
  return overlap(o, span_of(Q, int64_t(T) * p->Hq * p->d)) || overlap(o, span_of(K, cache)) || overlap(o, span_of(V, cache));
}

ab_status prepare_append(const ab_paged_params* p, const ab_norm_rope* nr, int32_t T, const ab_tokens* q,
                         const ab_tokens* k, const ab_tokens* v, const int32_t* slots, const int32_t* positions,
                         void* Q, void* Kc, void* Vc, void* ksum, NormRopeArgs* a) {
  ab_status s = check_norm_rope(nr);
  if (s != AB_OK) return s;
  if (T < 1) return AB_ERR_INVALID_ARG;
  if (any_bad({slots, positions, Q, Kc, Vc}) || !aligned16(ksum)) return AB_ERR_INVALID_ARG;
  if (T > kRopeMaxUnits || p->Hq > rope_max_heads(p->d)) return AB_ERR_UNSUPPORTED;
  const ab_tokens* in[3] = {q, k, v};
  void* out[3] = {Q, Kc, Vc};
  *a = NormRopeArgs{};
  for (int x = 0; x < 3; ++x) {
    a->heads[x] = x == 0 ? p->Hq : p->Hkv;
    if (check_tokens(in[x], 1, T, a->heads[x]) != AB_OK) return AB_ERR_INVALID_ARG;
    a->len[x] = a->tokens[x] = T;
    a->in[x] = view_of(in[x]);
    a->out[x] = static_cast<__nv_bfloat16*>(out[x]);
  }
  const int64_t cache = int64_t(p->num_pages) * p->Hkv * p->page * p->d;
  const Span o[3] = {span_of(Q, int64_t(T) * p->Hq * p->d), span_of(Kc, cache), span_of(Vc, cache)};
  for (int x = 0; x < 3; ++x)
    for (const Span& y : o)
      if (overlap(y, span_of(in[x], 1, T, a->heads[x], p->d))) return AB_ERR_INVALID_ARG;
  a->pos[0] = a->pos[1] = a->pos[2] = positions;
  a->slots = slots;
  a->page_shift = log2_of(p->page);
  a->num_pages = p->num_pages;
  set_norm_rope(a, nr);
  return AB_OK;
}

ab_status run_append(const ab_paged_params* p, const ab_norm_rope* nr, int32_t T, const NormRopeArgs& a, void* Kc,
                     void* ksum, cudaStream_t st) {
  ab_status s = launch_norm_rope(a, p->d, nr, st);
  if (s != AB_OK || !ksum) return s;
  // a CTA looks at 1 to 32 slots: one each up to 1184 (8 CTAs an SM), so that the
  // pages of single tokens spread over the SMs; 32 are a ballot
  int per_cta = (T + 1183) / 1184;
  per_cta = per_cta > 32 ? 32 : per_cta;
  const dim3 grid(unsigned((T + per_cta - 1) / per_cta), unsigned((p->Hkv + 7) / 8));
  const auto* kc = static_cast<const __nv_bfloat16*>(Kc);
  auto* ks = static_cast<__nv_bfloat16*>(ksum);
  return launch_after(p->d == 128 ? page_sum_kernel<128> : page_sum_kernel<64>, grid, 256, 0, st, a.slots,
                      a.cos_t ? a.pos[1] : nullptr, a.n_pos, T, per_cta, kc, ks, p->Hkv, a.page_shift, a.num_pages);
}

ab_status run_paged_select(const ab_paged_params* p, const PagedView& v, const void* Q, const void* ksum, float* P,
                           uint8_t* ws, cudaStream_t st) {
  const PagedWorkspace w = paged_workspace(p);
  SelectArgs a{};
  a.v = v;
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.ksum = static_cast<const __nv_bfloat16*>(ksum);
  a.scores = reinterpret_cast<float*>(ws + w.off_scores);
  a.part = reinterpret_cast<float2*>(ws + w.off_part);
  a.P = P;
  a.chunks = (p->max_pages + kSelPages - 1) / kSelPages;
  a.scale_log2 = float(1.4426950408889634 / std::sqrt(double(p->d)));
  const int sms = sm_count();
  if (!sms) return AB_ERR_CUDA;
  a.pitch = (p->max_pages + 3) / 4 * 4;
  // One launch with a CTA per row, for tables of few pages whose summaries fit in
  // L2: 3 x 12 rows of 47 pages 2.6 us (two launches 5.9), 64 x 8 rows of 256 7.6
  // (13.3), of 1000 31 (33); but 512 x 40 rows of 256 pages (1.3 GB) 350 (269: there
  // the warps of a CTA read neighbouring heads together), one row of 1000 7.2 (5.8).
  const int64_t rows = int64_t(p->S) * p->Hkv, bytes_all = rows * p->max_pages * p->d * 2;
  if (p->max_pages <= kRowPages && bytes_all <= kRowBytes && (p->max_pages <= 512 || rows >= 64)) {
    auto row = p->d == 128 ? (v.G > 8 ? page_row_kernel<128, true> : page_row_kernel<128, false>)
                           : (v.G > 8 ? page_row_kernel<64, true> : page_row_kernel<64, false>);
    const int bytes = v.G * a.pitch * 4;
    if (bytes > 46 * 1024 && set_smem(row, bytes) != cudaSuccess) return AB_ERR_CUDA;
    return launch_after(row, dim3(unsigned(p->S * p->Hkv)), kRowThreads, bytes, st, a);
  }
  const int64_t most = (int64_t(p->S) * p->Hkv * a.chunks + kSelWarps - 1) / kSelWarps;
  const unsigned grid = unsigned(most < sms ? most : sms);
  const bool wide = v.G > 8;
  auto score = p->d == 128 ? (wide ? page_score_kernel<128, true> : page_score_kernel<128, false>)
                           : (wide ? page_score_kernel<64, true> : page_score_kernel<64, false>);
  const int smem = kSelWarps * sel_stages(p->d) * 32 * p->d * 2;
  if (set_smem(score, smem) != cudaSuccess) return AB_ERR_CUDA;
  if (launch_after(score, dim3(grid), kSelWarps * 32, smem, st, a) != AB_OK) return AB_ERR_CUDA;
  int steps = (p->max_pages + 4 * kNormThreads - 1) / (4 * kNormThreads);
  steps = steps > 8 ? 8 : steps;
  return launch_after(page_mass_kernel, dim3(unsigned(steps), unsigned(p->Hkv), unsigned(p->S)), kNormThreads, 0, st, a);
}

ab_status run_paged_topk(const ab_paged_params* p, const float* P, const int32_t* lens, int32_t* idx, int32_t* count,
                         cudaStream_t st) {
  TopkArgs a{};
  a.P = P; a.lens = lens; a.idx = idx; a.count = count;
  a.Hkv = p->Hkv; a.page = p->page; a.page_shift = log2_of(p->page); a.max_pages = p->max_pages;
  a.recent = p->recent; a.keep = double(p->keep_ratio);
  a.cap = p->max_pages < kTopkMaxKeys ? p->max_pages : kTopkMaxKeys;
  const int smem = (a.cap > kTopkCount ? a.cap : kTopkCount) * 4;
  auto go = [&](auto kern, int threads) -> ab_status {
    if (smem > 36 * 1024 && set_smem(kern, smem) != cudaSuccess) return AB_ERR_CUDA;
    return launch_after(kern, dim3(unsigned(p->S * p->Hkv)), threads, smem, st, a);
  };
  if (p->max_pages <= 2560) return go(page_topk_kernel<256>, 256);
  return p->max_pages <= 8192 ? go(page_topk_kernel<512>, 512) : go(page_topk_kernel<1024>, 1024);
}

template <int D, bool kLists>
ab_status launch_paged_attention(const DecArgs& a, int grid, cudaStream_t st) {
  auto kern = paged_attention_kernel<D, kLists>;
  constexpr int smem = DecSmem<D>::kAlloc;
  if (set_smem(kern, smem) != cudaSuccess) return AB_ERR_CUDA;
  if (launch_after(kern, dim3(unsigned(grid)), kDecThreads, smem, st, a) != AB_OK) return AB_ERR_CUDA;
  if (grid == 1 || a.whole) return AB_OK;
  return launch_after(paged_join_kernel<D>, dim3(unsigned(grid - 1), unsigned(a.v.G)), 32 * kJoinWarps, 0, st, a, grid,
                      a.v.G > 8 ? 16 : 8);
}

ab_status run_paged_attention(const ab_paged_params* p, const PagedView& v, const void* Q, const void* Kc,
                              const void* Vc, const int32_t* idx, const int32_t* count, void* O, uint8_t* ws,
                              cudaStream_t st) {
  const PagedWorkspace w = paged_workspace(p);
  const int sms = sm_count();
  if (!sms) return AB_ERR_CUDA;
  DecArgs a{};
  a.v = v;
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.K = static_cast<const __nv_bfloat16*>(Kc);
  a.V = static_cast<const __nv_bfloat16*>(Vc);
  a.idx = idx;
  a.count = count;
  a.O = static_cast<__nv_bfloat16*>(O);
  a.scale_log2 = float(1.4426950408889634 / std::sqrt(double(p->d)));
  a.meta = reinterpret_cast<DecMeta*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + w.off_part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + w.off_ml);
  const int grid = sms < kDecMaxParts ? sms : kDecMaxParts;
  a.whole = (int64_t(p->max_pages) * p->page + dec_tile(p->d) - 1) / dec_tile(p->d) <= kWholeTiles;
  if (p->d == 128)
    return idx ? launch_paged_attention<128, true>(a, grid, st) : launch_paged_attention<128, false>(a, grid, st);
  return idx ? launch_paged_attention<64, true>(a, grid, st) : launch_paged_attention<64, false>(a, grid, st);
}

}  // namespace

extern "C" {

ab_status ab_qk_norm_rope(const ab_params* p, const ab_norm_rope* nr, const ab_tokens* q, const ab_tokens* k,
                          const ab_tokens* v, const int32_t* pos_q, const int32_t* pos_k, void* Q, void* K, void* V,
                          void* stream) {
  NvtxRange nvtx("ab_qk_norm_rope");
  ab_status s = check_sizes(p);
  if (s != AB_OK) return s;
  NormRopeArgs a;
  s = prepare_norm_rope(*p, nr, q, k, v, pos_q, pos_k, Q, K, V, &a);
  if (s != AB_OK) return s;
  return launch_norm_rope(a, p->d, nr, static_cast<cudaStream_t>(stream));
}

ab_status ab_forward_qkv(const ab_params* p, const ab_norm_rope* nr, const ab_tokens* q, const ab_tokens* k,
                         const ab_tokens* v, const int32_t* pos_q, const int32_t* pos_k, void* Q, void* K, void* V,
                         float* P, int32_t* idx, uint32_t* pi_q32, int32_t* count, void* O, void* workspace,
                         size_t ws_bytes, void* stream) {
  Dims d;
  NvtxRange nvtx("ab_forward_qkv");
  ab_status s = check_params(p, true, &d);
  if (s != AB_OK) return s;
  if (!q || !k || !v) return AB_ERR_INVALID_ARG;
  s = check_path_args(Q, K, V, P, idx, pi_q32, count, O, workspace, ws_bytes, workspace_layout(d).total);
  if (s != AB_OK) return s;
  NormRopeArgs a;
  s = prepare_norm_rope(*p, nr, q, k, v, pos_q, pos_k, Q, K, V, &a);
  if (s != AB_OK) return s;
  s = launch_norm_rope(a, d.d, nr, static_cast<cudaStream_t>(stream));
  if (s != AB_OK) return s;
  return ab_forward(p, Q, K, V, P, idx, pi_q32, count, O, workspace, ws_bytes, stream);
}

ab_status ab_paged_workspace_size(const ab_paged_params* p, int32_t with_select, size_t* bytes) {
  const ab_status s = check_paged(p);
  if (s != AB_OK) return s;
  if (!bytes) return AB_ERR_INVALID_ARG;
  const PagedWorkspace w = paged_workspace(p);
  *bytes = with_select && w.select > w.attend ? w.select : w.attend;
  return AB_OK;
}

ab_status ab_paged_plan(const ab_paged_params* p, int32_t T, const int32_t* n_new, const int32_t* lens,
                        int32_t* lens_out, int32_t* table, int32_t* free_pages, const int32_t* free_count,
                        int32_t* free_count_out, int32_t* cu_new, int32_t* slots, int32_t* positions, void* stream) {
  NvtxRange nvtx("ab_paged_plan");
  const ab_status s = check_paged(p);
  if (s != AB_OK) return s;
  if (T < 0) return AB_ERR_INVALID_ARG;
  if (any_bad({n_new, lens, lens_out, table, free_pages, free_count, free_count_out, cu_new})) return AB_ERR_INVALID_ARG;
  if (T > 0 && any_bad({slots, positions})) return AB_ERR_INVALID_ARG;
  PlanArgs a{};
  a.S = p->S; a.T = T; a.page = p->page; a.page_shift = log2_of(p->page);
  a.num_pages = p->num_pages; a.max_pages = p->max_pages;
  a.n_new = n_new; a.lens = lens; a.lens_out = lens_out; a.table = table; a.free_pages = free_pages;
  a.free_count = free_count; a.free_count_out = free_count_out;
  a.cu_new = cu_new; a.slots = slots; a.positions = positions;
  const int smem = (4 * p->S + 3) * 4;
  if (smem > 40 * 1024 && set_smem(plan_kernel, smem) != cudaSuccess) return AB_ERR_CUDA;
  return launch_after(plan_kernel, dim3(kPlanCtas), kPlanThreads, smem, static_cast<cudaStream_t>(stream), a);
}

ab_status ab_paged_append(const ab_paged_params* p, const ab_norm_rope* nr, int32_t T, const ab_tokens* q,
                          const ab_tokens* k, const ab_tokens* v, const int32_t* slots, const int32_t* positions,
                          void* Q, void* K, void* V, void* ksum, void* stream) {
  NvtxRange nvtx("ab_paged_append");
  ab_status s = check_paged(p);
  if (s != AB_OK) return s;
  if (T == 0) return check_norm_rope(nr);  // nothing to write
  NormRopeArgs a;
  s = prepare_append(p, nr, T, q, k, v, slots, positions, Q, K, V, ksum, &a);
  if (s != AB_OK) return s;
  return run_append(p, nr, T, a, K, ksum, static_cast<cudaStream_t>(stream));
}

ab_status ab_paged_select(const ab_paged_params* p, int32_t T, const void* Q, const void* ksum, const int32_t* table,
                          const int32_t* lens, const int32_t* cu_new, float* P, void* workspace, size_t ws_bytes,
                          void* stream) {
  NvtxRange nvtx("ab_paged_select");
  ab_status s = check_paged(p);
  if (s != AB_OK) return s;
  if (any_bad({Q, ksum, table, lens, P, workspace})) return AB_ERR_INVALID_ARG;
  s = check_rows(p, cu_new, T);
  if (s != AB_OK) return s;
  if (ws_bytes < paged_workspace(p).select) return AB_ERR_WORKSPACE;
  return run_paged_select(p, paged_view(p, table, lens, cu_new, T), Q, ksum, P, static_cast<uint8_t*>(workspace),
                          static_cast<cudaStream_t>(stream));
}

ab_status ab_paged_topk(const ab_paged_params* p, const float* P, const int32_t* lens, int32_t* idx, int32_t* count,
                        void* stream) {
  NvtxRange nvtx("ab_paged_topk");
  const ab_status s = check_paged(p);
  if (s != AB_OK) return s;
  if (any_bad({P, lens, idx, count})) return AB_ERR_INVALID_ARG;
  return run_paged_topk(p, P, lens, idx, count, static_cast<cudaStream_t>(stream));
}

ab_status ab_attention_paged(const ab_paged_params* p, int32_t T, const void* Q, const void* K, const void* V,
                             const int32_t* table, const int32_t* lens, const int32_t* cu_new, const int32_t* idx,
                             const int32_t* count, void* O, void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("ab_attention_paged");
  ab_status s = check_paged(p);
  if (s != AB_OK) return s;
  if (any_bad({Q, K, V, table, lens, O, workspace})) return AB_ERR_INVALID_ARG;
  if ((idx == nullptr) != (count == nullptr) || !aligned16(idx) || !aligned16(count)) return AB_ERR_INVALID_ARG;
  s = check_rows(p, cu_new, T);
  if (s != AB_OK) return s;
  if (ws_bytes < paged_workspace(p).attend) return AB_ERR_WORKSPACE;
  if (output_overlaps(p, T, Q, K, V, O)) return AB_ERR_INVALID_ARG;
  return run_paged_attention(p, paged_view(p, table, lens, cu_new, T), Q, K, V, idx, count, O,
                             static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream));
}

ab_status ab_paged_forward(const ab_paged_params* p, const ab_norm_rope* nr, int32_t T, const ab_tokens* q,
                           const ab_tokens* k, const ab_tokens* v, const int32_t* slots, const int32_t* positions,
                           const int32_t* table, const int32_t* lens, const int32_t* cu_new, void* Q, void* K, void* V,
                           void* ksum, float* P, int32_t* idx, int32_t* count, void* O, void* workspace,
                           size_t ws_bytes, void* stream) {
  NvtxRange nvtx("ab_paged_forward");
  ab_status s = check_paged(p);
  if (s != AB_OK) return s;
  if (any_bad({table, lens, cu_new, ksum, P, idx, count, O, workspace})) return AB_ERR_INVALID_ARG;
  NormRopeArgs a;
  s = prepare_append(p, nr, T, q, k, v, slots, positions, Q, K, V, ksum, &a);
  if (s != AB_OK) return s;
  s = check_rows(p, cu_new, T);
  if (s != AB_OK) return s;
  const PagedWorkspace w = paged_workspace(p);
  if (ws_bytes < w.select || ws_bytes < w.attend) return AB_ERR_WORKSPACE;
  if (output_overlaps(p, T, Q, K, V, O)) return AB_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const PagedView view = paged_view(p, table, lens, cu_new, T);
  s = run_append(p, nr, T, a, K, ksum, st);
  if (s != AB_OK) return s;
  s = run_paged_select(p, view, Q, ksum, P, ws, st);
  if (s != AB_OK) return s;
  s = run_paged_topk(p, P, lens, idx, count, st);
  if (s != AB_OK) return s;
  return run_paged_attention(p, view, Q, K, V, idx, count, O, ws, st);
}

}  // extern "C"
