// dense_host.cuh -- host side of the norm (norm.cuh) and of the dense products
// (dense.cuh, dense_small.cuh): argument checks, tensor maps, choice of the
// kernel, launches, and the pre-norm layer.  A part of moe.cu, whose helpers it
// uses.
#pragma once

namespace {

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A call's memory: what it writes must not overlap what it reads, nor one
// another (kernels read ahead, and a block writes while others still read).
struct Span {
  const void* p;
  int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}
bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (auto other = outs.begin(); other != o; ++other)
      if (overlap(*o, *other)) return false;
    for (const Span& i : ins)
      if (overlap(*o, i)) return false;
  }
  return true;
}
// apart, or in the same place
bool apart_or_same(const Span& out, const Span& in) { return out.p == in.p || !overlap(out, in); }

// ---- norm ------------------------------------------------------------------------
bool type16(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F16; }

// Block shape of a row of H: threads and packs per thread (a power of two).
// Above 256 threads a thread has 64 registers, which the backward pass spills
// over and cannot read ahead in: 2048 x 16384 take 44 us forward and 97 backward
// (their bytes 41 each), 8189 x 4096 42 and 56 (41).  Packs of one element cost
// more instructions: 8189 x 1530 29 and 104 us (15).
struct RowShape {
  int threads, nv;
};
RowShape row_shape(int64_t nvec) {
  int nv = 1;
  while (nv < 4 && nvec > 256 * nv) nv *= 2;  // up to 256 threads as long as 4 packs do
  while (nvec > 1024 * int64_t(nv)) nv *= 2;
  const int64_t per = (nvec + nv - 1) / nv;
  return {static_cast<int>((per + 31) / 32 * 32), nv};
}

// f(std::integral_constant<int, NV>, std::integral_constant<int, MAXT>) for the
// kernel that holds rows of that shape: the largest block it is compiled for is
// 256 threads up to 4 packs a thread (so that it may use the registers), 1024 above.
template <int VEC, typename F>
int with_row_shape(const RowShape& rs, F&& f) {
  using std::integral_constant;
  if (rs.threads <= 256) {
    if (rs.nv == 1) return f(integral_constant<int, 1>{}, integral_constant<int, 256>{});
    if (rs.nv == 2) return f(integral_constant<int, 2>{}, integral_constant<int, 256>{});
    if (rs.nv == 4) return f(integral_constant<int, 4>{}, integral_constant<int, 256>{});
  }
  if (rs.nv == 4) return f(integral_constant<int, 4>{}, integral_constant<int, 1024>{});
  if constexpr (VEC == 1) {
    if (rs.nv == 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1024>{});
    if (rs.nv == 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1024>{});
    if (rs.nv == 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1024>{});
  }
  return fail(MOE_ERR_INVALID_ARG, "row of %d x %d packs", rs.threads, rs.nv);
}

template <typename E, int VEC>
int launch_norm(int fmt, int64_t T, const void* x, const void* res, const void* w, float eps, int H,
                int group, void* s_out, void* out, float* scales, cudaStream_t s) {
  const RowShape rs = row_shape(H / VEC);
  return with_row_shape<VEC>(rs, [&](auto nv, auto maxt) {
    constexpr int NV = decltype(nv)::value, MAXT = decltype(maxt)::value;
    auto k = fmt == norm::kSame   ? norm::add_rmsnorm_kernel<E, VEC, NV, norm::kSame, MAXT>
             : fmt == norm::kInt8 ? norm::add_rmsnorm_kernel<E, VEC, NV, norm::kInt8, MAXT>
                                  : norm::add_rmsnorm_kernel<E, VEC, NV, norm::kE4m3, MAXT>;
    return launch_pdl("add_rmsnorm_kernel launch", k, dim3(static_cast<unsigned>(T)), dim3(rs.threads), 0, s,
                      static_cast<const E*>(x), static_cast<const E*>(res), static_cast<const E*>(w), eps, H,
                      group, static_cast<E*>(s_out), out, scales);
  });
}

int do_add_rmsnorm(int type, int fmt, int64_t T, const void* x, const void* res, const void* w, float eps,
                   int H, int group, void* s_out, void* out, float* scales, cudaStream_t s) {
  // 16-byte accesses need every row to start on 16 bytes (8-bit rows: 8)
  if (type == MOE_TYPE_BF16)
    return H % 8 == 0 ? launch_norm<__nv_bfloat16, 8>(fmt, T, x, res, w, eps, H, group, s_out, out, scales, s)
                      : launch_norm<__nv_bfloat16, 1>(fmt, T, x, res, w, eps, H, group, s_out, out, scales, s);
  return H % 8 == 0 ? launch_norm<__half, 8>(fmt, T, x, res, w, eps, H, group, s_out, out, scales, s)
                    : launch_norm<__half, 1>(fmt, T, x, res, w, eps, H, group, s_out, out, scales, s);
}

template <typename E, int VEC>
int launch_norm_bwd(int64_t T, const void* dy, const void* sv, const void* w, float eps, int H,
                    const void* dstream, void* dx, float* parts, int blocks, cudaStream_t s) {
  const RowShape rs = row_shape(H / VEC);
  return with_row_shape<VEC>(rs, [&](auto nv, auto maxt) {
    constexpr int NV = decltype(nv)::value, MAXT = decltype(maxt)::value;
    auto k = eps > 0.f ? norm::rmsnorm_backward_kernel<E, VEC, NV, MAXT, false>
                       : norm::rmsnorm_backward_kernel<E, VEC, NV, MAXT, true>;
    return launch_pdl("rmsnorm_backward_kernel launch", k, dim3(blocks), dim3(rs.threads), 0, s,
                      static_cast<const E*>(dy), static_cast<const E*>(sv), static_cast<const E*>(w), eps, T, H,
                      static_cast<const E*>(dstream), static_cast<E*>(dx), parts);
  });
}

// Blocks of the backward pass, each with a row of dw partial sums: as many as
// run at once on a B200's 148 SMs (a constant, since the workspace's size is
// asked for without a device).
int norm_parts(int64_t T, int64_t H) {
  const int vec = H % 8 == 0 ? 8 : 1;
  const RowShape rs = row_shape(H / vec);
  const int maxt = rs.threads <= 256 && rs.nv <= 4 ? 256 : 1024;
  const int per_sm = norm::backward_blocks(vec, rs.nv, maxt) * std::max(1, maxt / rs.threads);
  return static_cast<int>(std::min<int64_t>(T, 148 * per_sm));
}

int check_norm_H(int64_t H) {
  REQUIRE(H >= 1 && H <= norm::kMaxH, "H=%lld outside [1, %d]", static_cast<long long>(H), norm::kMaxH);
  return MOE_OK;
}

// ---- dense products -----------------------------------------------------------------
constexpr int64_t kMaxDim = 65536;        // widths of the gated block
constexpr int64_t kMaxInt8N = 1 << 20;    // channels of the int8 product
constexpr int64_t kMaxInt8K = 131056;     // K * 128 * 128 < 2^31: the int32 sums cannot overflow

// Row-major matrix of `rows` rows of `cols` elements (of 1, 2 or 4 bytes), boxes
// of box_bytes x box_rows with the swizzle of that width: 128 bytes for the
// operands (outside the matrix reads zero), 64 for the outputs.
int make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int elem, int box_rows,
             int box_bytes = 128) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes / elem), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type = elem == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                               : CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const CUresult r = g_encode(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return MOE_OK;
}

// An operand: rows x cols as it lies in memory; mn: its m (or n) runs along a
// row (else k does).
struct Operand {
  const void* p;
  int64_t rows, cols;
  bool mn;
  int64_t k() const { return mn ? rows : cols; }
  int64_t outer() const { return mn ? cols : rows; }
};

// The pair kernel for a tile width and a type (of the 16-bit operands and
// outputs; of the outputs where the operands are int8).
template <int KIND, bool A_MN, bool B_MN, int EPI>
auto pair_kernel(int bn, int type) -> void (*)(const dense::Args) {
  using namespace dense;
  if constexpr (KIND == kI8Kind)
    if (type == kF32)
      return bn == 256 ? pair_gemm_kernel<KIND, A_MN, B_MN, EPI, 256, kF32>
                       : pair_gemm_kernel<KIND, A_MN, B_MN, EPI, 128, kF32>;
  if (type == kF16)
    return bn == 256 ? pair_gemm_kernel<KIND, A_MN, B_MN, EPI, 256, kF16>
                     : pair_gemm_kernel<KIND, A_MN, B_MN, EPI, 128, kF16>;
  return bn == 256 ? pair_gemm_kernel<KIND, A_MN, B_MN, EPI, 256, kBF16>
                   : pair_gemm_kernel<KIND, A_MN, B_MN, EPI, 128, kBF16>;
}

// What one launch computes, before a kernel is chosen for it.
struct Product {
  Operand a[dense::kMaxProb], b[dense::kMaxProb];
  void* out[dense::kMaxProb] = {};  // several products: NULL leaves one out (its size still counts for the shape)
  int nprob = 1, nseg = 1;
  int type = dense::kBF16;  // operand type, or kF32 outputs of int8
  const void* residual = nullptr;
  void* saved = nullptr;     // pre-activations (kGated: out, kDGate: in)
  void* out2 = nullptr;
  const float *a_scale = nullptr, *b_scale = nullptr, *bias = nullptr;
};

template <typename A>
void common_args(A* g, const Product& p) {
  g->residual = static_cast<const uint16_t*>(p.residual);
  g->saved = static_cast<uint8_t*>(p.saved);
  g->a_scale = p.a_scale;
  g->b_scale = p.b_scale;
  g->bias = p.bias;
  g->timeout_ns = g_timeout_ns.load();
}

// launch_pdl with clusters of `cluster` CTAs.
template <typename A>
int launch_cluster(const char* what, void (*kernel)(A), unsigned grid, int threads, size_t smem, int cluster,
                   cudaStream_t s, const A& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return MOE_OK;
}

// How a launch runs.  On CTA pairs: tiles of 256 rows x `tile` columns, `split`
// pairs to a tile.  For few tokens: tiles of `tile` tokens x `rows` weight rows,
// `split` CTAs to a tile.  ns: the estimated time of a launch on CTA pairs.
struct Plan {
  bool pairs;
  int tile, rows, split;
  int64_t ns;
};

// The choice with the smallest estimate.  Measured at T = 96 .. 2048 tokens and
// widths of 512 to 4096: a k-block takes a pair 300 ns (256 columns) or 290 ns
// (128; both wait for L2), everything else 6.5 or 5.0 us, and sharing a tile
// 2.2 us more, or 0.9 us and 0.6 us for each pair above two.  E.g. T = 256,
// N = K = 4096 in int8: 16 tiles of 256 columns 16.8 us, shared by two pairs
// 14.2, by four 24 (two rounds of clusters); 32 tiles of 128 columns 15.0,
// shared by two 11.6.
template <int EPI>
Plan pair_plan(const Product& p, int64_t kbs, const DeviceInfo& dev) {
  Plan best{true, 256, dense::kBM, 1, INT64_MAX};
  for (const int bn : {256, 128}) {
    int64_t tiles = 0;
    for (int i = 0; i < p.nprob; ++i)
      tiles += div_up(p.a[i].outer(), dense::kBM) * div_up(p.b[i].outer(), EPI == dense::kGated ? bn / 2 : bn);
    for (int split = 1; split <= dense::kMaxPairs; ++split) {
      // a shared tile has a cluster to itself: one round of them (33, 22 or 15 on 148 SMs)
      if (split > 1 && (tiles > dev.clusters[split] || kbs < 4 * split)) continue;
      const int64_t rounds = split > 1 ? 1 : div_up(tiles, dev.sms / 2);
      const int64_t share = split == 1 ? 0 : bn == 256 ? 2200 : 900 + 600 * (split - 2);
      const int64_t ns = rounds * div_up(kbs, split) * (bn == 256 ? 300 : 290) + (bn == 256 ? 6500 : 5000) + share;
      if (ns < best.ns) best = {true, bn, dense::kBM, split, ns};
    }
  }
  return best;
}

// k-blocks of a product, over its segments
template <int KIND>
int64_t all_kblocks(const Product& p) {
  return div_up(p.a[0].k(), KIND == dense::kI8Kind ? 128 : 64) * p.nseg;
}

template <int KIND, bool A_MN, bool B_MN, int EPI>
int launch_pair(const Product& p, const Plan& plan, const DeviceInfo& dev, cudaStream_t s) {
  const int elem = KIND == dense::kI8Kind ? 1 : 2, ke = 128 / elem;
  dense::Args g{};
  g.nseg = p.nseg;
  g.kblocks = static_cast<int>(div_up(p.a[0].k(), ke));
  const int bn = plan.tile;
  g.split = plan.split;
  int64_t tiles = 0;
  const int out_elem = p.type == dense::kF32 ? 4 : 2;
  g.tma_out = true;  // unless some product's rows are not whole 16-byte pieces
  for (int i = 0; i < p.nprob; ++i) g.tma_out = g.tma_out && p.b[i].outer() * out_elem % 16 == 0;
  g.nprob = 0;
  for (int i = 0; i < std::max(p.nprob, p.nseg); ++i) {  // products, or segments of one
    if (p.nprob > 1 && p.out[i] == nullptr) continue;
    const int j = p.nprob > 1 ? g.nprob : i;
    int rc = make_map(&g.a[j], p.a[i].p, p.a[i].rows, p.a[i].cols, elem, A_MN ? 64 : 128);
    if (!rc) rc = make_map(&g.b[j], p.b[i].p, p.b[i].rows, p.b[i].cols, elem, B_MN ? 64 : bn / 2);
    if (rc) return rc;
    if (i >= p.nprob) continue;
    dense::Problem& q = g.p[g.nprob++];
    q.M = p.a[i].outer();
    q.N = p.b[i].outer();
    q.mt = static_cast<int>(div_up(q.M, dense::kBM));
    q.nt = static_cast<int>(div_up(q.N, EPI == dense::kGated ? bn / 2 : bn));
    q.tile0 = static_cast<int>(tiles);
    q.out = p.out[i];
    tiles += int64_t(q.mt) * q.nt;
    if (g.tma_out) rc = make_map(&g.o[j], q.out, q.M, q.N, out_elem, 32, 64);
    if (!rc && EPI == dense::kDGate) rc = make_map(&g.o[1], p.out2, q.M, q.N, out_elem, 32, 64);
    if (rc) return rc;
  }
  if (EPI == dense::kGated) {  // b[1]: the up weights
    int rc = make_map(&g.b[1], p.b[1].p, p.b[1].rows, p.b[1].cols, elem, 64);
    if (rc) return rc;
  }
  g.tiles = static_cast<int>(tiles);
  common_args(&g, p);
  g.idesc = dense::make_idesc(KIND, p.type, A_MN, B_MN, dense::kBM, bn);
  const int64_t clusters = g.split > 1 ? tiles : std::min<int64_t>(tiles, dev.sms / 2);
  const size_t smem = bn == 256 ? dense::PairCfg<256>::SMEM : dense::PairCfg<128>::SMEM;
  return launch_cluster("pair_gemm_kernel launch", pair_kernel<KIND, A_MN, B_MN, EPI>(bn, p.type),
                        static_cast<unsigned>(clusters * 2 * g.split), dense::kPairThreads, smem, 2 * g.split, s, g);
}

// CTAs that share a few-token tile's k range: a power of two, as long as the
// SMs have room for all CTAs at once and each keeps 2 k-blocks (T = 16,
// H = 2048, I = 5632: 19.6 us; with half the CTAs 20.4, T = 1, H = 1536,
// I = 4096: 13.7 and 15.4).
int small_split(int64_t tiles, int64_t kbs, int64_t room) {
  int split = 1;
  while (split < dense::kMaxSplit && tiles * split * 2 <= room && kbs >= split * 4) split *= 2;
  return split;
}

template <int KIND, bool W_MN, int EPI, int NT, int ROWS>
int launch_small_rows(const Product& p, int split, cudaStream_t s) {
  const int elem = KIND == dense::kI8Kind ? 1 : 2, ke = 128 / elem;
  dense::SmallArgs g{};
  g.T = p.a[0].outer();
  g.N = p.b[0].outer();
  g.nseg = p.nseg;
  g.kblocks = static_cast<int>(div_up(p.a[0].k(), ke));
  g.wt = static_cast<int>(div_up(g.N, EPI == dense::kGated ? 64 : ROWS));
  const int64_t tiles = g.wt * div_up(g.T, NT);
  for (int i = 0; i < p.nseg; ++i) {
    int rc = make_map(&g.x[i], p.a[i].p, p.a[i].rows, p.a[i].cols, elem, NT);
    if (!rc) rc = make_map(&g.w[i], p.b[i].p, p.b[i].rows, p.b[i].cols, elem, W_MN ? 64 : ROWS);
    if (rc) return rc;
  }
  if (EPI == dense::kGated) {
    int rc = make_map(&g.w[1], p.b[1].p, p.b[1].rows, p.b[1].cols, elem, 64);
    if (rc) return rc;
  }
  g.split = split;
  g.out = p.out[0];
  common_args(&g, p);
  g.out2 = p.out2;
  g.type = p.type;
  g.idesc = dense::make_idesc(KIND, p.type, W_MN, false, 128, NT);
  return launch_cluster("small_gemm_kernel launch", dense::small_gemm_kernel<KIND, W_MN, EPI, NT, ROWS>,
                        static_cast<unsigned>(tiles * g.split), dense::kSmallThreads,
                        dense::SmallCfg<NT, ROWS>::SMEM, g.split, s, g);
}

template <int KIND, int EPI, int NT, int ROWS>
Plan small_plan_rows(const Product& p, int sms) {
  const int64_t tiles = div_up(p.b[0].outer(), EPI == dense::kGated ? 64 : ROWS) * div_up(p.a[0].outer(), NT);
  const int64_t room = int64_t(sms) * dense::SmallCfg<NT, ROWS>::PER_SM;
  return {false, NT, ROWS, small_split(tiles, all_kblocks<KIND>(p), room), 0};
}
template <int KIND, int EPI, int NT>
Plan small_plan(const Product& p, int sms) {
  if constexpr (EPI != dense::kGated) {
    // Tiles of 64 weight rows where 128-row tiles, split as far as they go, are
    // fewer than the SMs; with more than two token tiles already where they
    // would have to share SMs for it (H = 1536, I = 4096, dh and dx: T = 192
    // 28.8 us against 33.1 with 128 rows, but T = 128 26.1 against 23.8).
    const int64_t token_tiles = div_up(p.a[0].outer(), NT);
    const int64_t tiles = div_up(p.b[0].outer(), 128) * token_tiles;
    const int64_t room = token_tiles > 2 ? sms : int64_t(sms) * dense::SmallCfg<NT, 128>::PER_SM;
    if (tiles * small_split(tiles, all_kblocks<KIND>(p), room) < sms)
      return small_plan_rows<KIND, EPI, NT, 64>(p, sms);
  }
  return small_plan_rows<KIND, EPI, NT, 128>(p, sms);
}

// The kernel for one product of T tokens with weights.  Up to 32 tokens the
// weights are the MMA's rows; above, by the estimate of both ways: with the
// weights as rows 4 us, 0.38 us for each k-block (128 weight rows x 64 tokens)
// and 2 us for each tile that an SM gets, measured over the sizes that pair_plan
// names (int8, N = 4096: T = 128, K = 4096 9.4 us against 11.3 on pairs, T = 256
// 13.0 against 11.4, T = 192, K = 1536 9.4 against 8.3; N = 512, T = 256, K = 1536
// 4.2 against 7.7).
template <int KIND, int EPI>
Plan product_plan(const Product& p, const DeviceInfo& dev) {
  const int64_t T = p.a[0].outer();
  if (T <= 16) return small_plan<KIND, EPI, 16>(p, dev.sms);
  if (T <= 32) return small_plan<KIND, EPI, 32>(p, dev.sms);
  const int64_t tiles = div_up(p.b[0].outer(), EPI == dense::kGated ? 64 : 128) * div_up(T, 64);
  const int64_t kbs = all_kblocks<KIND>(p);
  const Plan pairs = pair_plan<EPI>(p, kbs, dev);
  return 4000 + tiles * (kbs * 380 + 2000) / dev.sms <= pairs.ns ? small_plan<KIND, EPI, 64>(p, dev.sms) : pairs;
}

template <int KIND, bool W_MN, int EPI, int NT>
int launch_small(const Product& p, const Plan& plan, cudaStream_t s) {
  if constexpr (EPI != dense::kGated)
    if (plan.rows == 64) return launch_small_rows<KIND, W_MN, EPI, NT, 64>(p, plan.split, s);
  return launch_small_rows<KIND, W_MN, EPI, NT, 128>(p, plan.split, s);
}

template <int KIND, bool B_MN, int EPI>
int launch_product(const Product& p, const DeviceInfo& dev, cudaStream_t s) {
  const Plan plan = product_plan<KIND, EPI>(p, dev);
  if (plan.pairs) return launch_pair<KIND, false, B_MN, EPI>(p, plan, dev, s);
  if (plan.tile == 16) return launch_small<KIND, B_MN, EPI, 16>(p, plan, s);
  if (plan.tile == 32) return launch_small<KIND, B_MN, EPI, 32>(p, plan, s);
  return launch_small<KIND, B_MN, EPI, 64>(p, plan, s);
}

template <int KIND, bool A_MN, bool B_MN, int EPI>
cudaError_t pair_attr() {
  cudaError_t e = cudaSuccess;
  for (const int bn : {256, 128})
    for (const int type : {dense::kBF16, dense::kF16, dense::kF32}) {
      if (type == dense::kF32 && KIND != dense::kI8Kind) continue;
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(pair_kernel<KIND, A_MN, B_MN, EPI>(bn, type)),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 bn == 256 ? dense::PairCfg<256>::SMEM : dense::PairCfg<128>::SMEM);
    }
  return e;
}
template <int KIND, bool W_MN, int EPI, int NT>
cudaError_t small_attr_nt() {
  cudaError_t e = cudaFuncSetAttribute(dense::small_gemm_kernel<KIND, W_MN, EPI, NT, 128>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, dense::SmallCfg<NT, 128>::SMEM);
  if constexpr (EPI != dense::kGated)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(dense::small_gemm_kernel<KIND, W_MN, EPI, NT, 64>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, dense::SmallCfg<NT, 64>::SMEM);
  return e;
}
template <int KIND, bool W_MN, int EPI>
cudaError_t small_attr() {
  cudaError_t e = small_attr_nt<KIND, W_MN, EPI, 16>();
  if (e == cudaSuccess) e = small_attr_nt<KIND, W_MN, EPI, 32>();
  if (e == cudaSuccess) e = small_attr_nt<KIND, W_MN, EPI, 64>();
  return e;
}
// Shared-memory limits of the kernels, and how many clusters of the pair
// kernel the device runs at once.
cudaError_t dense_setup(DeviceInfo* dev) {
  using namespace dense;
  cudaError_t e = pair_attr<kF16Kind, false, true, kGated>();
  if (e == cudaSuccess) e = pair_attr<kF16Kind, false, true, kPlain>();
  if (e == cudaSuccess) e = pair_attr<kF16Kind, false, false, kPlain>();
  if (e == cudaSuccess) e = pair_attr<kF16Kind, false, false, kDGate>();
  if (e == cudaSuccess) e = pair_attr<kF16Kind, true, true, kPlain>();
  if (e == cudaSuccess) e = pair_attr<kI8Kind, false, false, kScaled>();
  if (e == cudaSuccess) e = small_attr<kF16Kind, true, kGated>();
  if (e == cudaSuccess) e = small_attr<kF16Kind, true, kPlain>();
  if (e == cudaSuccess) e = small_attr<kF16Kind, false, kPlain>();
  if (e == cudaSuccess) e = small_attr<kF16Kind, false, kDGate>();
  if (e == cudaSuccess) e = small_attr<kI8Kind, false, kScaled>();
  for (int split = 2; e == cudaSuccess && split <= kMaxPairs; ++split) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * split));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = PairCfg<256>::SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(2 * split);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&dev->clusters[split],
                                       pair_gemm_kernel<kF16Kind, false, true, kPlain, 256, kBF16>, &cfg);
  }
  return e;
}

// The gated block's products, by their sizes; the entry points add the rest.
Product gate_up_product(int64_t T, int64_t H, int64_t I) {
  Product p{};
  p.a[0] = {nullptr, T, H, false};
  p.b[0] = p.b[1] = {nullptr, H, I, true};
  return p;
}
Product down_product(int64_t T, int64_t H, int64_t I) {
  Product p{};
  p.a[0] = {nullptr, T, I, false};
  p.b[0] = {nullptr, I, H, true};
  return p;
}
Product dh_product(int64_t T, int64_t H, int64_t I) {
  Product p{};
  p.a[0] = {nullptr, T, H, false};
  p.b[0] = {nullptr, I, H, false};
  return p;
}
Product dx_product(int64_t T, int64_t H, int64_t I) {
  Product p{};
  p.a[0] = p.a[1] = {nullptr, T, I, false};
  p.b[0] = p.b[1] = {nullptr, H, I, false};
  p.nseg = 2;
  return p;
}
Product dw_product(int64_t T, int64_t H, int64_t I) {
  Product p{};
  p.a[0] = p.a[1] = {nullptr, T, H, true};
  p.a[2] = {nullptr, T, I, true};
  p.b[0] = p.b[1] = {nullptr, T, I, true};
  p.b[2] = {nullptr, T, H, true};
  p.nprob = 3;
  return p;
}
Product int8_product(int64_t T, int64_t N, int64_t K) {
  Product p{};
  p.a[0] = {nullptr, T, K, false};
  p.b[0] = {nullptr, N, K, false};
  return p;
}

int check_ffn(int64_t T, int64_t H, int64_t I, int dtype) {
  int rc = check_T(T);
  if (rc) return rc;
  REQUIRE(H >= 8 && H <= kMaxDim && H % 8 == 0 && I >= 8 && I <= kMaxDim && I % 8 == 0,
          "H=%lld and I=%lld must be multiples of 8 in [8, %lld]", static_cast<long long>(H),
          static_cast<long long>(I), static_cast<long long>(kMaxDim));
  REQUIRE(type16(dtype), "dtype=%d: bf16 or fp16", dtype);
  return MOE_OK;
}

int check_int8(int64_t N, int64_t K) {
  REQUIRE(N >= 1 && N <= kMaxInt8N, "N=%lld outside [1, %lld]", static_cast<long long>(N),
          static_cast<long long>(kMaxInt8N));
  REQUIRE(K >= 16 && K <= kMaxInt8K && K % 16 == 0, "K=%lld must be a multiple of 16 in [16, %lld]",
          static_cast<long long>(K), static_cast<long long>(kMaxInt8K));
  return MOE_OK;
}

}  // namespace

// The public type codes are the kernels' own.
static_assert(int(MOE_TYPE_BF16) == dense::kBF16 && int(MOE_TYPE_F16) == dense::kF16 &&
                  int(MOE_TYPE_F32) == dense::kF32,
              "types");
static_assert(int(MOE_FORMAT_SAME) == norm::kSame && int(MOE_FORMAT_INT8) == norm::kInt8 &&
                  int(MOE_FORMAT_E4M3) == norm::kE4m3,
              "formats");

extern "C" {

int moe_add_rmsnorm(const void* x, const void* residual, const void* weight, float eps, int64_t T,
                    int64_t H, int dtype, void* stream_out, int format, int group, void* out,
                    float* scales, moe_stream_t stream) {
  int rc = check_T(T);
  if (!rc) rc = check_norm_H(H);
  if (rc) return rc;
  REQUIRE(type16(dtype), "dtype=%d: bf16 or fp16", dtype);
  REQUIRE(format >= MOE_FORMAT_SAME && format <= MOE_FORMAT_E4M3, "format=%d", format);
  REQUIRE(group == 0 || (group == norm::kGroup && format != MOE_FORMAT_SAME),
          "group=%d: 0, or %d with an 8-bit format", group, norm::kGroup);
  REQUIRE(eps >= 0.f && eps < INFINITY, "eps must be finite and not negative");
  if (T == 0) return MOE_OK;
  REQUIRE(x && out && (!residual || stream_out) && (format == MOE_FORMAT_SAME || scales), "null pointer");
  REQUIRE(aligned(x, 16) && aligned(out, 16) && aligned(residual, 16) && aligned(weight, 16) &&
              aligned(stream_out, 16) && aligned(scales, 16),
          "pointers must be 16-byte aligned");
  const int64_t row = T * H * 2;
  const Span X{x, row}, R{residual, row}, S{residual ? stream_out : nullptr, row};
  const Span O{out, format == MOE_FORMAT_SAME ? row : T * H};
  const Span C{format == MOE_FORMAT_SAME ? nullptr : scales, T * (group ? div_up(H, group) : 1) * 4};
  REQUIRE(apart({O, S, C}, {{weight, H * 2}}) && apart({C}, {X, R}) && apart_or_same(S, X) && apart_or_same(S, R) &&
              (format == MOE_FORMAT_SAME ? apart_or_same(O, X) && apart_or_same(O, R) : apart({O}, {X, R})),
          "outputs overlap inputs or one another");
  rc = device_setup(nullptr, nullptr);
  if (rc) return rc;
  return do_add_rmsnorm(dtype, format, T, x, residual, weight, eps, static_cast<int>(H), group, stream_out, out,
                        scales, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_add_rmsnorm_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T < 0 || T > kMaxTokens || H < 1 || H > norm::kMaxH) return 0;
  return static_cast<size_t>(norm_parts(T, H)) * static_cast<size_t>(H) * sizeof(float);
}

int moe_add_rmsnorm_backward(const void* dy, const void* s, const void* weight, float eps, int64_t T,
                             int64_t H, int dtype, const void* dstream, void* dx, float* dweight,
                             void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_T(T);
  if (!rc) rc = check_norm_H(H);
  if (rc) return rc;
  REQUIRE(type16(dtype), "dtype=%d: bf16 or fp16", dtype);
  REQUIRE(eps >= 0.f && eps < INFINITY, "eps must be finite and not negative");
  REQUIRE(aligned(dy, 16) && aligned(s, 16) && aligned(weight, 16) && aligned(dstream, 16) && aligned(dx, 16) &&
              aligned(dweight, 16) && aligned(workspace, 16),
          "pointers must be 16-byte aligned");
  REQUIRE(T == 0 || (dy && s && dx), "null pointer");
  const size_t need = dweight ? moe_add_rmsnorm_backward_workspace_bytes(T, H) : 0;
  if (need && (workspace == nullptr || workspace_bytes < need))
    return fail(MOE_ERR_WORKSPACE, "moe_add_rmsnorm_backward workspace needs %zu bytes, got %zu", need,
                workspace ? workspace_bytes : size_t(0));
  if (T == 0 && !dweight) return MOE_OK;
  REQUIRE(apart({{dx, T * H * 2}, {dweight, H * 4}, {dweight ? workspace : nullptr, int64_t(need)}},
                {{dy, T * H * 2}, {s, T * H * 2}, {weight, H * 2}, {dstream, T * H * 2}}),
          "outputs or the workspace overlap inputs or one another");
  rc = device_setup(nullptr, nullptr);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // the gradient of no tokens
    MOE_CUDA(cudaMemsetAsync(dweight, 0, static_cast<size_t>(H) * sizeof(float), st), "cudaMemsetAsync");
    return MOE_OK;
  }
  float* parts = dweight ? static_cast<float*>(workspace) : nullptr;
  const int blocks = norm_parts(T, H), h = static_cast<int>(H);
  if (dtype == MOE_TYPE_BF16)
    rc = h % 8 == 0 ? launch_norm_bwd<__nv_bfloat16, 8>(T, dy, s, weight, eps, h, dstream, dx, parts, blocks, st)
                    : launch_norm_bwd<__nv_bfloat16, 1>(T, dy, s, weight, eps, h, dstream, dx, parts, blocks, st);
  else
    rc = h % 8 == 0 ? launch_norm_bwd<__half, 8>(T, dy, s, weight, eps, h, dstream, dx, parts, blocks, st)
                    : launch_norm_bwd<__half, 1>(T, dy, s, weight, eps, h, dstream, dx, parts, blocks, st);
  if (rc || !dweight) return rc;
  return launch_pdl("rmsnorm_dw_kernel launch", norm::rmsnorm_dw_kernel, dim3((h + 31) / 32), dim3(1024), 0, st,
                    static_cast<const float*>(parts), blocks, h, dweight);
}

int moe_int8_matmul(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                    const float* bias, int64_t T, int64_t N, int64_t K, int out_dtype, void* out,
                    moe_stream_t stream) {
  int rc = check_T(T);
  if (rc) return rc;
  rc = check_int8(N, K);
  if (rc) return rc;
  REQUIRE(type16(out_dtype) || out_dtype == MOE_TYPE_F32, "out_dtype=%d: bf16, fp16 or fp32", out_dtype);
  if (T == 0) return MOE_OK;
  REQUIRE(a && a_scale && b && b_scale && out, "null pointer");
  REQUIRE(aligned(a, 16) && aligned(a_scale, 16) && aligned(b, 16) && aligned(b_scale, 16) && aligned(bias, 16) &&
              aligned(out, 16),
          "pointers must be 16-byte aligned");
  REQUIRE(apart({{out, T * N * (out_dtype == MOE_TYPE_F32 ? 4 : 2)}},
                {{a, T * K}, {a_scale, T * 4}, {b, N * K}, {b_scale, N * 4}, {bias, N * 4}}),
          "the output overlaps an input");
  DeviceInfo dev;
  rc = device_info(&dev);
  if (rc) return rc;
  Product p = int8_product(T, N, K);
  p.a[0].p = a;
  p.b[0].p = b;
  p.out[0] = out;
  p.type = out_dtype;
  p.a_scale = a_scale;
  p.b_scale = b_scale;
  p.bias = bias;
  return launch_product<dense::kI8Kind, false, dense::kScaled>(p, dev, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_gated_ffn_saved_bytes(int64_t T, int64_t I) {
  if (T < 0 || T > kMaxTokens || I < 0 || I > kMaxDim) return 0;
  return static_cast<size_t>(dense::saved_bytes(T, I));
}

int moe_gated_ffn(const void* x, const void* w_gate, const void* w_up, const void* w_down, int64_t T,
                  int64_t H, int64_t I, int dtype, const void* residual, void* h, void* saved, void* y,
                  moe_stream_t stream) {
  int rc = check_ffn(T, H, I, dtype);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  REQUIRE(x && w_gate && w_up && w_down && h && y, "null pointer");
  REQUIRE(aligned(x, 16) && aligned(w_gate, 16) && aligned(w_up, 16) && aligned(w_down, 16) && aligned(h, 16) &&
              aligned(saved, 16) && aligned(y, 16) && aligned(residual, 16),
          "pointers must be 16-byte aligned");
  const int64_t row = T * H * 2, w = H * I * 2;
  const Span X{x, row}, R{residual, row}, Y{y, row}, A{h, T * I * 2}, V{saved, dense::saved_bytes(T, I)};
  REQUIRE(apart({Y, A, V}, {{w_gate, w}, {w_up, w}, {w_down, w}}) && apart({A, V}, {X, R}) && apart_or_same(Y, X) &&
              apart_or_same(Y, R),
          "outputs overlap inputs or one another");
  DeviceInfo dev;
  rc = device_info(&dev);
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Product up = gate_up_product(T, H, I);
  up.a[0].p = x;
  up.b[0].p = w_gate;
  up.b[1].p = w_up;
  up.out[0] = h;
  up.type = dtype;
  up.saved = saved;
  rc = launch_product<dense::kF16Kind, true, dense::kGated>(up, dev, s);
  if (rc) return rc;
  Product down = down_product(T, H, I);
  down.a[0].p = h;
  down.b[0].p = w_down;
  down.out[0] = y;
  down.type = dtype;
  down.residual = residual;
  return launch_product<dense::kF16Kind, true, dense::kPlain>(down, dev, s);
}

size_t moe_gated_ffn_backward_workspace_bytes(int64_t T, int64_t I) {
  if (T < 0 || T > kMaxTokens || I < 0 || I > kMaxDim) return 0;
  return static_cast<size_t>(T) * static_cast<size_t>(I) * 4;
}

int moe_gated_ffn_backward(const void* dy, const void* x, const void* w_gate, const void* w_up,
                           const void* w_down, const void* h, const void* saved, int64_t T, int64_t H,
                           int64_t I, int dtype, void* dx, void* dw_gate, void* dw_up, void* dw_down,
                           void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_ffn(T, H, I, dtype);
  if (rc) return rc;
  REQUIRE(aligned(dy, 16) && aligned(x, 16) && aligned(w_gate, 16) && aligned(w_up, 16) && aligned(w_down, 16) &&
              aligned(h, 16) && aligned(saved, 16) && aligned(dx, 16) && aligned(dw_gate, 16) && aligned(dw_up, 16) &&
              aligned(dw_down, 16) && aligned(workspace, 16),
          "pointers must be 16-byte aligned");
  void* dw[3] = {dw_gate, dw_up, dw_down};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if (T == 0) {  // the gradients of no tokens
    rc = device_info(&dev);
    if (rc) return rc;
    for (void* d : dw)
      if (d) MOE_CUDA(cudaMemsetAsync(d, 0, static_cast<size_t>(H) * static_cast<size_t>(I) * 2, s), "cudaMemsetAsync");
    return MOE_OK;
  }
  const bool need_d = dx || dw_gate || dw_up;  // dg and du
  REQUIRE(dy && (!need_d || (w_down && saved)) && (!dx || (w_gate && w_up)) && (!(dw_gate || dw_up) || x) &&
              (!dw_down || h),
          "null pointer");
  const size_t need = need_d ? moe_gated_ffn_backward_workspace_bytes(T, I) : 0;
  if (need && (workspace == nullptr || workspace_bytes < need))
    return fail(MOE_ERR_WORKSPACE, "moe_gated_ffn_backward workspace needs %zu bytes, got %zu", need,
                workspace ? workspace_bytes : size_t(0));
  const int64_t row = T * H * 2, w = H * I * 2;
  REQUIRE(apart({{dx, row}, {dw_gate, w}, {dw_up, w}, {dw_down, w}, {need_d ? workspace : nullptr, int64_t(need)}},
                {{dy, row}, {x, row}, {w_gate, w}, {w_up, w}, {w_down, w}, {h, T * I * 2},
                 {saved, dense::saved_bytes(T, I)}}),
          "outputs or the workspace overlap inputs or one another");
  rc = device_info(&dev);
  if (rc) return rc;
  char* dg = static_cast<char*>(workspace);
  char* du = dg + static_cast<size_t>(T) * static_cast<size_t>(I) * 2;
  if (need_d) {
    Product p = dh_product(T, H, I);
    p.a[0].p = dy;
    p.b[0].p = w_down;
    p.out[0] = dg;
    p.out2 = du;
    p.type = dtype;
    p.saved = const_cast<void*>(saved);
    rc = launch_product<dense::kF16Kind, false, dense::kDGate>(p, dev, s);
    if (rc) return rc;
  }
  if (dx) {
    Product p = dx_product(T, H, I);
    p.a[0].p = dg;
    p.a[1].p = du;
    p.b[0].p = w_gate;
    p.b[1].p = w_up;
    p.out[0] = dx;
    p.type = dtype;
    rc = launch_product<dense::kF16Kind, false, dense::kPlain>(p, dev, s);
    if (rc) return rc;
  }
  // The weights' gradients asked for, in one launch, whose shape goes by all
  // three: a gradient's bits do not depend on which others are wanted.
  if (!dw_gate && !dw_up && !dw_down) return MOE_OK;
  Product p = dw_product(T, H, I);
  p.type = dtype;
  for (int i = 0; i < 3; ++i) {
    p.a[i].p = i < 2 ? x : h;
    p.b[i].p = i == 0 ? dg : i == 1 ? du : dy;
    p.out[i] = dw[i];
  }
  const Plan plan = pair_plan<dense::kPlain>(p, all_kblocks<dense::kF16Kind>(p), dev);
  return launch_pair<dense::kF16Kind, true, true, dense::kPlain>(p, plan, dev, s);
}

// ---- how a product runs --------------------------------------------------------------
int moe_dense_plan(int product, int64_t T, int64_t N, int64_t K, int32_t* plan) {
  const bool int8 = product == MOE_PRODUCT_INT8;
  int rc = check_T(T);
  if (!rc) rc = int8 ? check_int8(N, K) : check_ffn(T, K, N, MOE_TYPE_BF16);
  if (rc) return rc;
  REQUIRE(T > 0 && plan, "T=%lld: there is no product", static_cast<long long>(T));
  DeviceInfo dev;
  if (device_info(&dev) != MOE_OK) {  // no device here: a B200's
    dev.sms = 148;
    const int clusters[dense::kMaxPairs + 1] = {0, 0, 33, 22, 15};
    std::copy(clusters, clusters + dense::kMaxPairs + 1, dev.clusters);
  }
  using namespace dense;
  Plan r{};
  switch (product) {
    case MOE_PRODUCT_GATE_UP: r = product_plan<kF16Kind, kGated>(gate_up_product(T, K, N), dev); break;
    case MOE_PRODUCT_DOWN: r = product_plan<kF16Kind, kPlain>(down_product(T, K, N), dev); break;
    case MOE_PRODUCT_DH: r = product_plan<kF16Kind, kDGate>(dh_product(T, K, N), dev); break;
    case MOE_PRODUCT_DX: r = product_plan<kF16Kind, kPlain>(dx_product(T, K, N), dev); break;
    case MOE_PRODUCT_DW: {
      const Product p = dw_product(T, K, N);
      r = pair_plan<kPlain>(p, all_kblocks<kF16Kind>(p), dev);
      break;
    }
    case MOE_PRODUCT_INT8: r = product_plan<kI8Kind, kScaled>(int8_product(T, N, K), dev); break;
    default: return fail(MOE_ERR_INVALID_ARG, "product=%d", product);
  }
  plan[0] = r.pairs;
  plan[1] = r.tile;
  plan[2] = r.rows;
  plan[3] = r.split;
  return MOE_OK;
}

// ---- the pre-norm layer ------------------------------------------------------------
size_t moe_layer_normed_workspace_bytes(int64_t T) {
  if (T < 0 || T > kMaxTokens) return 0;
  return align_up(layer_ws(T, false, 0).total, 1024) + align_up(static_cast<size_t>(T) * kH * 2, 1024);
}

int moe_layer_normed(const moe_bf16* x, const moe_bf16* residual, const moe_bf16* norm_weight, float eps,
                     const moe_bf16* packed_router, const float* bias, const moe_bf16* packed_w, int64_t T,
                     moe_bf16* stream_out, moe_bf16* out, int32_t* topk_idx_out, float* topk_w_out,
                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = check_T(T);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  REQUIRE(packed_router && packed_w && out && workspace, "null pointer");
  REQUIRE(aligned(workspace, 1024), "workspace must be 1024-byte aligned");
  const size_t need = moe_layer_normed_workspace_bytes(T);
  if (workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "moe_layer_normed workspace needs %zu bytes, got %zu", need, workspace_bytes);
  REQUIRE(aligned(packed_w, 128) && aligned(packed_router, 128), "packed weights must be 128-byte aligned");
  REQUIRE(aligned(bias, 16) && aligned(out, 16) && aligned(topk_idx_out, 16) && aligned(topk_w_out, 16),
          "pointers must be 16-byte aligned");
  const int64_t row = T * kH * 2;
  const Span X{x, row}, R{residual, row}, S{residual ? stream_out : nullptr, row}, O{out, row};
  const Span I{topk_idx_out, T * kTopK * 4}, W{topk_w_out, T * kTopK * 4};
  const Span weights[] = {{norm_weight, kH * 2},
                          {packed_router, static_cast<int64_t>(moe_router_packed_bytes())},
                          {bias, kE * 4},
                          {packed_w, static_cast<int64_t>(moe_packed_weight_bytes())}};
  bool ok = apart({I, W, {workspace, static_cast<int64_t>(need)}}, {X, R, S, O}) && apart_or_same(S, X) &&
            apart_or_same(S, R) && apart_or_same(O, X) && apart_or_same(O, R) && apart_or_same(O, S);
  for (const Span& w : weights) ok = ok && apart({w}, {I, W, S, O, {workspace, static_cast<int64_t>(need)}});
  REQUIRE(ok, "outputs or the workspace overlap inputs or one another");
  const size_t layer = align_up(layer_ws(T, false, 0).total, 1024);
  moe_bf16* n = reinterpret_cast<moe_bf16*>(static_cast<char*>(workspace) + layer);
  rc = moe_add_rmsnorm(x, residual, norm_weight, eps, T, kH, MOE_TYPE_BF16, stream_out, MOE_FORMAT_SAME, 0, n,
                       nullptr, stream);
  if (rc) return rc;
  return layer_impl("moe_layer_normed", n, nullptr, packed_router, bias, packed_w, T, residual ? stream_out : x, out,
                    topk_idx_out, topk_w_out, workspace, layer, stream);
}

}  // extern "C"
