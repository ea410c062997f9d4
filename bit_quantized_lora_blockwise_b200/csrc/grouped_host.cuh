// Host side of the expert-grouped linear and of dropout: plans, workspace,
// tensor maps and launch order. Included by qlora.cu inside its unnamed
// namespace (it uses that file's launchers and map helpers).
//
// The host knows E and T but not the offsets, so it sizes grids and
// workspaces for the worst split of T tokens over E experts, and picks
// the tile from the average tokens per expert; either is right for every
// split.

// An expert of c tokens has ceil(c / tile) token tiles: the most there can be
// is when each of the experts has one token and the rest fills whole tiles.
inline int64_t token_tiles_bound(int64_t T, int64_t E, int64_t tile) {
  const int64_t experts = std::min(E, T);
  return experts + (T - experts) / tile;
}

struct GroupedShape {
  int64_t E, T, N, K;
  int r;
  bool drop;
};

// Two 256-token sub-tiles per tile from this average of tokens per expert
// (T / E) on; one below it. (8 experts, 4096 columns: at 256 tokens an expert
// 11008 rows take 200 us with one and 214 with two, at 375 276 and 262. The
// same 256-token tiles serve a single token: the dequantization, not the
// tokens, sets their time. A stream over the codes with register decode, as
// the dense call's few-token path, took 131 us against 126 for 32 rows over 8
// experts and lost from 5 rows an expert on; 128-token tiles with a deeper
// ring were within 1 %.)
constexpr int64_t kGroupedTwoSubtile = 320;

using GroupedFwd1 = GemmCfg<256, A_DEQ_K, L2_A_MN, kPairBkb, kPairSb, kPairSa, kPairSp, kPairNpw, true, 1, true>;
using GroupedFwd2 = GemmCfg<256, A_DEQ_K, L2_A_MN, kPair2Bkb, kPair2Sb, kPair2Sa, kPair2Sp, kPair2Npw, true, 2, true>;
using GroupedBwd1 = GemmCfg<256, A_DEQ_MN, L2_A_K, kPairBkb, kPairSb, kPairSa, kPairSp, kPairNpw, true, 1, true>;
using GroupedBwd2 = GemmCfg<256, A_DEQ_MN, L2_A_K, kPair2Bkb, kPair2Sb, kPair2Sa, kPair2Sp, kPair2Npw, true, 2, true>;
// the backward with adapter dropout: low-rank step first, masked in TMEM
using GroupedBwdDrop1 =
    GemmCfg<256, A_DEQ_MN, L2_A_K, kPairBkb, kPairSb, kPairSa, kPairSp, kPairNpw, true, 1, true, true>;
using GroupedBwdDrop2 =
    GemmCfg<256, A_DEQ_MN, L2_A_K, kPair2Bkb, kPair2Sb, kPair2Sa, kPair2Sp, kPair2Npw, true, 2, true, true>;

// Resident pair slots of every grouped variant on this device (asked once;
// 0 without a device: the calls then return before any launch).
int grouped_pair_slots(int sms) {
  static std::once_flag once[kMaxDevices];
  static int cached[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::call_once(once[dev], [&] {
    cached[dev] = std::min({resident_pairs<GroupedFwd1>(), resident_pairs<GroupedFwd2>(), resident_pairs<GroupedBwd1>(),
                            resident_pairs<GroupedBwd2>(), resident_pairs<GroupedBwdDrop1>(),
                            resident_pairs<GroupedBwdDrop2>()});
  });
  return std::min(cached[dev], sms / 2);
}

// Partials of a grouped GEMM split over K: splits x tiles <= slots (plan_grouped).
size_t grouped_part_bytes(int slots, int ntt, int64_t kblocks) {
  return kblocks / 4 >= 2 ? align256(static_cast<size_t>(slots) * 256 * ntt * 256 * 4) : 0;
}

struct GroupedPlanHost {
  int ntt, slots;
  int64_t counters;
  size_t part;
};
// kblocks: K / 64 (forward) or N / 64 (backward)
GroupedPlanHost plan_grouped_host(const GroupedShape &s, int64_t kblocks, int sms) {
  GroupedPlanHost p{};
  p.ntt = s.T / s.E >= kGroupedTwoSubtile ? 2 : 1;
  p.slots = grouped_pair_slots(sms);
  p.counters = 2 * p.slots + 1;  // of split tiles, and of gradient_kernel's units
  p.part = grouped_part_bytes(p.slots, p.ntt, kblocks);
  return p;
}

// dA and dB over persistent CTAs (gradient_kernel): when there are more 128-row
// tiles than CTAs that can be resident.
bool persistent_gradients(const GroupedShape &s, int sms) {
  return s.E * (cdiv(s.K, 128) + cdiv(s.N, 128)) > (s.r <= 128 ? 2 : 1) * static_cast<int64_t>(sms);
}

// [counters][16-bit T x r: s XA, or Gs][backward: 16-bit T x r twice, Gs' second
// part and XA][fp32 partials][keep bits T x K / 8 (backward with dropout, for
// gradient_kernel)]
struct GroupedWs {
  size_t counters, tr, part, keep, total;
};
GroupedWs grouped_ws(const GroupedShape &s, int64_t ncounters, size_t part, bool backward, int sms) {
  GroupedWs w;
  w.counters = align256(static_cast<size_t>(ncounters) * 4);
  w.tr = align256(static_cast<size_t>(s.T) * s.r * 2);
  w.part = part;
  w.keep = backward && s.drop && persistent_gradients(s, sms) ? align256(static_cast<size_t>(s.T) * (s.K / 8)) : 0;
  w.total = w.counters + (backward ? 3 : 1) * w.tr + w.part + w.keep;
  return w;
}

static_assert(QLORA_MAX_EXPERTS == kMaxGroups, "the group table holds every expert");

// Shapes that every grouped kernel can index: weight rows, tile and unit
// counts stay within int32.
qlora_status check_grouped(const GroupedShape &s) {
  if (s.E < 1 || s.E > QLORA_MAX_EXPERTS || s.T < 0 || s.N < 64 || s.K < 64 || s.N % 64 || s.K % 64)
    return QLORA_ERR_SHAPE;
  const int64_t lim = int64_t(1) << 30;
  if (s.T > lim || s.N > lim || s.K > lim || s.E * s.N > lim || s.E * s.K > lim) return QLORA_ERR_SHAPE;
  if (token_tiles_bound(s.T, s.E, 256) * cdiv(std::max(s.N, s.K), 128) * 8 > lim) return QLORA_ERR_SHAPE;
  if (s.r < 1 || s.r > QLORA_MAX_RANK || s.r % 8) return QLORA_ERR_RANGE;
  return QLORA_OK;
}

// Threshold and factor of a dropout description (dropout.cuh); NULL or a
// threshold of 0 drops nothing.
qlora_status make_dropout(const qlora_dropout_desc *d, DropoutArgs *out) {
  *out = dropout_args(0, 0, 0u);
  if (d == nullptr) return QLORA_OK;
  if (!(d->p >= 0.0 && d->p < 1.0)) return QLORA_ERR_RANGE;
  const double t = std::floor(d->p * 65536.0 + 0.5);
  if (t > 65535.0) return QLORA_ERR_RANGE;
  *out = dropout_args(d->seed, d->offset, static_cast<uint32_t>(t));
  return QLORA_OK;
}

// One thread per 8 elements; up to 64 CTAs per SM, eight of them resident: CTAs
// that start at different times keep loads and stores mixed (8192 x 11008 in
// bf16: one resident wave 68.3 us, 16 CTAs per SM 65.2, 64 63.8).
qlora_status run_dropout(const void *x, void *y, int64_t n, int type, const DropoutArgs &d, int sms, cudaStream_t st) {
  const int grid = grid_for(cdiv(n, 8), 256, sms, 64);
  if (type == DROP_F32) return launch_pdl(dropout_kernel<DROP_F32>, grid, 256, 0, st, x, y, n, d);
  if (type == DROP_F16) return launch_pdl(dropout_kernel<DROP_F16>, grid, 256, 0, st, x, y, n, d);
  return launch_pdl(dropout_kernel<DROP_BF16>, grid, 256, 0, st, x, y, n, d);
}

// Expert stack of 16-bit matrices [groups][outer][inner]: box {box_inner, box_outer, 1}.
bool map_experts_3d(CUtensorMap *map, const void *p, int64_t inner, int64_t outer, int64_t groups, uint32_t box_inner,
                    uint32_t box_outer) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                              static_cast<cuuint64_t>(groups)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner) * 2, static_cast<cuuint64_t>(inner * outer) * 2};
  const cuuint32_t box[3] = {box_inner, box_outer, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// out[T, r] = scale * rows . adapter_e: X A (kind SK_XA; with dropout (M o X)
// A) or dY B^T (SK_G). out2: for X A optionally a second copy with another
// scale, for dY B^T the second part of what out rounds.
qlora_status grouped_rows(SkinnyKind kind, const void *rows, const void *adapter, const GroupedShape &s,
                          const GroupArgs &g, const DropoutArgs &drop, void *out, float scale, void *out2, float scale2,
                          unsigned int *zero_words, int64_t nzero, cudaStream_t st) {
  const int64_t kdim = kind == SK_XA ? s.K : s.N;
  const int64_t tiles = token_tiles_bound(s.T, s.E, 128);
  const bool masked = kind == SK_XA && s.drop;
  SkinnyPlan p;
  qlora_status e = masked          ? plan_skinny_v<false, true, true, true>(tiles * 128, kdim, s.r, &p)
                   : kind == SK_XA ? plan_skinny_v<false, true, true>(tiles * 128, kdim, s.r, &p)
                                   : plan_skinny_v<false, false, true>(tiles * 128, kdim, s.r, &p);
  if (e != QLORA_OK) return e;
  SkinnyArgs a;
  std::memset(&a, 0, sizeof a);
  SkinnyProblem &P = a.prob[0];
  const bool ok = map_kmajor(&P.tm_a, rows, kdim, s.T, 128) &&
                  (kind == SK_XA ? map_experts_3d(&P.tm_b, adapter, s.r, s.K, s.E, 64, 64)
                                 : map_experts_3d(&P.tm_b, adapter, s.N, s.r, s.E, 64, static_cast<uint32_t>(p.bn)));
  if (!ok) return QLORA_ERR_CUDA;
  P.out = out;
  P.out_ld = s.r;
  P.out_scale = scale;
  P.out2 = out2;
  P.out2_ld = s.r;
  P.out2_scale = scale2;
  P.rest = kind == SK_G ? 1 : 0;
  P.rows = static_cast<int>(s.T);
  P.cols = s.r;
  P.kblocks = static_cast<int>(kdim / 64);
  a.splits = p.splits;
  const int grid = static_cast<int>(tiles) * p.splits;
  a.prob0_ctas = grid;
  a.zero_words = zero_words;
  a.nzero = static_cast<int>(nzero);
  a.f16 = t_f16 ? 1 : 0;
  a.groups = g;
  P.masked = masked ? 1 : 0;
  a.drop = drop;
  a.drop_ld = s.K;
  if (masked) return run_skinny<false, true, true, true>(a, p.bn, grid, st);
  return kind == SK_XA ? run_skinny<false, true, true>(a, p.bn, grid, st)
                       : run_skinny<false, false, true>(a, p.bn, grid, st);
}

template <int BN, bool DROP>
qlora_status run_gradients_bn(const GradientArgs &a, int64_t units, int sms, cudaStream_t st) {
  using C = GradientCfg<BN, BN == 64 ? 3 : 4, DROP>;  // 96 KB of ring, two CTAs an SM; or 192 KB
  static std::once_flag once[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(once[dev], [&] {
    err[dev] = cudaFuncSetAttribute(gradient_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (err[dev] == cudaSuccess)
      err[dev] = cudaFuncSetAttribute(gradient_kernel<C>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      static_cast<int>(cudaSharedmemCarveoutMaxShared));
  });
  if (err[dev] != cudaSuccess) return QLORA_ERR_CUDA;
  const int grid = static_cast<int>(std::min<int64_t>(units, static_cast<int64_t>(C::PER_SM) * sms));
  return launch_pdl(gradient_kernel<C>, grid, C::THREADS, C::SMEM_BYTES, st, a);
}

template <bool DROP>
qlora_status run_gradients(const GradientArgs &a, int64_t units, int sms, cudaStream_t st) {
  if (a.r <= 64) return run_gradients_bn<64, DROP>(a, units, sms, st);
  return run_gradients_bn<128, DROP>(a, units * cdiv(a.r, 128), sms, st);
}

// dA_e = factor (M o X_e)^T Gs_e (gs, gs2: its two parts) and dB_e = s xa_e^T dY_e, every expert's in one
// launch: over persistent CTAs (`keep`: the mask's bits, which dX left), else
// with each tile's tokens split over a cluster.
qlora_status grouped_adapter_grads(const void *X, const void *dY, const void *gs, const void *gs2, const void *xa,
                                   const GroupedShape &s, const GroupArgs &g, const DropoutArgs &drop,
                                   const uint32_t *keep, unsigned int *unit_counter, void *dA, void *dB,
                                   float b_scale, int sms, cudaStream_t st) {
  const int64_t ta = s.E * cdiv(s.K, 128), tb = s.E * cdiv(s.N, 128);
  if (persistent_gradients(s, sms)) {
    GradientArgs a;
    std::memset(&a, 0, sizeof a);
    if (!map_mnmajor(&a.tm_x, X, s.K, s.T) || !map_mnmajor(&a.tm_gs, gs, s.r, s.T) ||
        !map_mnmajor(&a.tm_gs2, gs2, s.r, s.T) || !map_mnmajor(&a.tm_dy, dY, s.N, s.T) ||
        !map_mnmajor(&a.tm_xa, xa, s.r, s.T))
      return QLORA_ERR_CUDA;
    a.dA = dA;
    a.dB = dB;
    a.a_scale = drop.factor;
    a.b_scale = b_scale;
    a.K = static_cast<int>(s.K);
    a.N = static_cast<int>(s.N);
    a.r = s.r;
    a.f16 = t_f16 ? 1 : 0;
    a.groups = g;
    a.keep = keep;
    a.counter = unit_counter;
    return s.drop ? run_gradients<true>(a, ta + tb, sms, st) : run_gradients<false>(a, ta + tb, sms, st);
  }
  SkinnyPlan p;
  const qlora_status e = s.drop ? plan_skinny_v<true, true, true, true>((ta + tb) * 128, cdiv(s.T, s.E), s.r, &p)
                                : plan_skinny_v<true, true, true>((ta + tb) * 128, cdiv(s.T, s.E), s.r, &p);
  if (e != QLORA_OK) return e;
  SkinnyArgs a;
  std::memset(&a, 0, sizeof a);
  SkinnyProblem &A = a.prob[0], &B = a.prob[1];
  if (!map_mnmajor(&A.tm_a, X, s.K, s.T) || !map_mnmajor(&A.tm_b, gs, s.r, s.T) ||
      !map_mnmajor(&A.tm_b2, gs2, s.r, s.T) || !map_mnmajor(&B.tm_a, dY, s.N, s.T) ||
      !map_mnmajor(&B.tm_b, xa, s.r, s.T))
    return QLORA_ERR_CUDA;
  A.parts = 2;
  B.parts = 1;
  A.out = dA;
  A.out_ld = s.r;
  A.out_scale = drop.factor;
  A.rows = static_cast<int>(s.K);
  A.cols = s.r;
  B.out = dB;
  B.out_ld = s.N;
  B.out_scale = b_scale;
  B.transpose = 1;
  B.rows = static_cast<int>(s.N);
  B.cols = s.r;
  a.splits = p.splits;
  a.prob0_ctas = static_cast<int>(ta) * p.splits;
  a.late = 1;
  a.f16 = t_f16 ? 1 : 0;
  a.groups = g;
  const int grid = static_cast<int>(ta + tb) * p.splits;
  if (!s.drop) return run_skinny<true, true, true>(a, p.bn, grid, st);
  A.masked = 1;
  a.drop = drop;
  a.drop_ld = s.K;
  return run_skinny<true, true, true, true>(a, p.bn, grid, st);
}

template <class C>
qlora_status run_grouped_gemm(const GemmArgs &args, int slots, cudaStream_t stream) {
  // (resident_pairs has set the kernel's shared memory)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * slots);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, qgemm_kernel<C>, args);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return e == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

// What forward and backward share of the GEMM's arguments.
void grouped_gemm_args(GemmArgs *a, const uint8_t *q, const float *scale2, const float *nf4, const float *t8,
                       const GroupedShape &s, const GroupArgs &g, int64_t rows, int64_t kblocks, void *out, float *part,
                       unsigned int *counters) {
  a->rows = static_cast<int>(rows);
  a->cols = static_cast<int>(s.T);
  a->kblocks = static_cast<int>(kblocks);
  a->lora_kblocks = static_cast<int>(cdiv(s.r, 64));
  a->out = out;
  a->out_ld = rows;
  a->part = part;
  a->counters = counters;
  std::memcpy(a->nf4, nf4, sizeof a->nf4);
  std::memcpy(a->t8, t8, sizeof a->t8);
  a->q = q;
  a->scale2 = scale2;
  a->wkb = s.K / 64;
  a->f16 = t_f16 ? 1 : 0;
  a->groups = g;
  a->expert_rows = static_cast<int>(s.N);
}

qlora_status grouped_fwd(const uint8_t *packed, const uint8_t *q, const float *scale2, const float *nf4,
                         const float *t8, const GroupedShape &s, const int *offsets, const void *X, const void *A,
                         const void *B, float alpha, const DropoutArgs &drop, void *Y, void *XA_out, void *workspace,
                         size_t workspace_bytes, int sms, cudaStream_t cs) {
  const GroupedPlanHost p = plan_grouped_host(s, s.K / 64, sms);
  const GroupedWs w = grouped_ws(s, p.counters, p.part, false, sms);
  if (!workspace || workspace_bytes < w.total) return QLORA_ERR_WORKSPACE;
  if (p.slots < 1) return QLORA_ERR_CUDA;  // no room for a CTA pair
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  unsigned int *counters = reinterpret_cast<unsigned int *>(ws);
  void *xas = ws + w.counters;
  float *part = reinterpret_cast<float *>(ws + w.counters + w.tr);
  const GroupArgs g{offsets, static_cast<int>(s.E), static_cast<int>(s.T)};
  const float scl = alpha / static_cast<float>(s.r);
  qlora_status st = QLORA_OK;

  // 1) XA = D(X) A, and s XA for the low-rank step (the dropout factor in
  //    both scales: the product itself reads M o X); zeroes the counters
  st = grouped_rows(SK_XA, X, A, s, g, drop, xas, scl * drop.factor, XA_out, drop.factor, counters, p.counters, cs);
  if (st != QLORA_OK) return st;

  // 2) the base product, whose main loop overlaps 1)
  GemmArgs a;
  std::memset(&a, 0, sizeof a);
  const uint32_t box = static_cast<uint32_t>(128 * p.ntt);
  if (!map_tokens_3d(&a.tm_b, X, s.T, s.K, box, 1) ||
      !map_codes_fwd(&a.tm_pk, packed, s.E * s.N, s.K, p.ntt == 2 ? GroupedFwd2::KSUP : GroupedFwd1::KSUP) ||
      !map_experts_3d(&a.tm_a2, B, s.N, s.r, s.E, 64, 64) || !map_kmajor(&a.tm_b2, xas, s.r, s.T, box))
    return QLORA_ERR_CUDA;
  grouped_gemm_args(&a, q, scale2, nf4, t8, s, g, s.N, s.K / 64, Y, part, counters);
  trace_begin(cs);
  st = p.ntt == 2 ? run_grouped_gemm<GroupedFwd2>(a, p.slots, cs) : run_grouped_gemm<GroupedFwd1>(a, p.slots, cs);
  trace_end(cs);
  return st;
}

qlora_status grouped_bwd(const uint8_t *packed, const uint8_t *q, const float *scale2, const float *nf4,
                         const float *t8, const GroupedShape &s, const int *offsets, const void *X, const void *dY,
                         const void *A, const void *B, const void *XA, float alpha, const DropoutArgs &drop, void *dX,
                         void *dA, void *dB, void *workspace, size_t workspace_bytes, int sms, cudaStream_t cs) {
  const GroupedPlanHost p = plan_grouped_host(s, s.N / 64, sms);
  const GroupedWs w = grouped_ws(s, p.counters, p.part, true, sms);
  if (!workspace || workspace_bytes < w.total) return QLORA_ERR_WORKSPACE;
  if (p.slots < 1) return QLORA_ERR_CUDA;  // no room for a CTA pair
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  unsigned int *counters = reinterpret_cast<unsigned int *>(ws);
  void *gs = ws + w.counters;
  void *gs2 = ws + w.counters + w.tr;
  void *xa_ws = ws + w.counters + 2 * w.tr;
  float *part = reinterpret_cast<float *>(ws + w.counters + 3 * w.tr);
  uint32_t *keep = w.keep > 0 ? reinterpret_cast<uint32_t *>(ws + w.counters + 3 * w.tr + w.part) : nullptr;
  const GroupArgs g{offsets, static_cast<int>(s.E), static_cast<int>(s.T)};
  const float scl = alpha / static_cast<float>(s.r);
  qlora_status st = QLORA_OK;

  // 1) XA where it was not saved, and Gs = s dY B^T in two parts (dA reads
  //    both, dX the first), whose launch zeroes the counters. (The dropout
  //    factor of dX and dA multiplies their fp32 sums: in Gs it would cost fp16
  //    that much of its range.)
  if (XA == nullptr) {
    st = grouped_rows(SK_XA, X, A, s, g, drop, xa_ws, drop.factor, nullptr, 0.0f, nullptr, 0, cs);
    if (st != QLORA_OK) return st;
    XA = xa_ws;
  }
  st = grouped_rows(SK_G, dY, B, s, g, drop, gs, scl, gs2, scl, counters, p.counters, cs);
  if (st != QLORA_OK) return st;

  // 2) dX
  GemmArgs a;
  std::memset(&a, 0, sizeof a);
  const uint32_t box = static_cast<uint32_t>(128 * p.ntt);
  if (!map_tokens_3d(&a.tm_b, dY, s.T, s.N, box, 1) ||
      !map_codes_bwd(&a.tm_pk, packed, s.E * s.N, s.K, p.ntt == 2 ? GroupedBwd2::KSUP : GroupedBwd1::KSUP) ||
      !map_experts_3d(&a.tm_a2, A, s.r, s.K, s.E, 64, 128) || !map_kmajor(&a.tm_b2, gs, s.r, s.T, box))
    return QLORA_ERR_CUDA;
  grouped_gemm_args(&a, q, scale2, nf4, t8, s, g, s.K, s.N / 64, dX, part, counters);
  a.drop = drop;
  a.keep_bits = keep;
  trace_begin(cs);
  if (s.drop)
    st = p.ntt == 2 ? run_grouped_gemm<GroupedBwdDrop2>(a, p.slots, cs) : run_grouped_gemm<GroupedBwdDrop1>(a, p.slots, cs);
  else
    st = p.ntt == 2 ? run_grouped_gemm<GroupedBwd2>(a, p.slots, cs) : run_grouped_gemm<GroupedBwd1>(a, p.slots, cs);
  trace_end(cs);
  if (st != QLORA_OK) return st;

  // 3) dA and dB "late", as in the dense backward: every operand but the keep
  //    bits (whose readers wait for them) is complete when this launch starts,
  //    and dX is neither read nor written by it
  return grouped_adapter_grads(X, dY, gs, gs2, XA, s, g, drop, keep, counters + 2 * p.slots, dA, dB, scl, sms, cs);
}
