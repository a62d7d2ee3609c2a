// dense.cuh -- dense matrix products on tcgen05 for any sizes: the gated
// feed-forward block (forward and backward) and the 8-bit integer product.
//
// Every product is D[m][n] = sum_k A(m, k) B(n, k) with fp32 (int32 for int8)
// accumulators in tensor memory.  An operand is read as it lies in memory:
// "K-major" (k consecutive) or "MN-major" (m or n consecutive), so neither
// weights nor activations are transposed or packed beforehand:
//   gate/up   A = x [T][H]  K-major    B = W_gate, W_up [H][I]  MN-major
//   down      A = h [T][I]  K-major    B = W_down [I][H]        MN-major
//   d h       A = dy [T][H] K-major    B = W_down [I][H]        K-major
//   d x       A = dg, du [T][I] K-major  B = W_gate, W_up [H][I] K-major (two k segments)
//   d W       A = x, x, h   MN-major   B = dg, du, dy           MN-major (three products)
//   int8      A = a [T][K]  K-major    B = b [N][K]             K-major
// A k-block is 128 bytes of k (64 16-bit or 128 8-bit elements).  In shared
// memory a K-major operand is rows of 128 bytes with the 128-byte swizzle; an
// MN-major one is chunks of 64 m (or n), each 64 k-rows of 128 bytes, same
// swizzle.  TMA fills what lies outside the matrix with zeros, in both
// operands, so ragged sizes need no masks before the store.
// h, dg and du go from one product to the next rounded to 16 bits, the tensor
// cores' operands (fp32 ones would have to be split into two or three 16-bit
// products); the sums before the rounding are fp32.
//
// pair_gemm_kernel: two CTAs of a cluster work on one 256 x BN tile
// (tcgen05.mma.cta_group::2): each loads 128 rows of A and BN/2 rows of B and
// holds the accumulators of its 128 rows, so a byte of B in shared memory
// feeds twice the MMAs of a single-CTA tile.  Persistent, tiles round-robin;
// two accumulator sets, so the epilogue of one tile overlaps the next one's
// MMAs.  Where the tiles are too few for the SMs, 2 to 4 pairs of a larger
// cluster share a tile (`split`): each takes a range of k and sends its
// accumulators, by 32 columns, to the pair that owns these columns, which adds
// them up in rank order and stores them.
#pragma once
#include "common.cuh"

namespace moe {
namespace dense {

constexpr unsigned kSiteEmpty = 40, kSiteFull = 41, kSiteTmemFull = 42, kSiteTmemEmpty = 43,
                   kSiteDrain = 44, kSiteSmallFull = 45, kSiteSmallEmpty = 46, kSiteSmallDone = 47, kSiteSmallParts = 48, kSiteParts = 49;

enum Kind { kF16Kind = 0, kI8Kind = 1 };                 // operand width: 16 or 8 bits
enum Epi { kGated = 0, kPlain = 1, kDGate = 2, kScaled = 3 };
enum Type { kBF16 = 0, kF16 = 1, kF32 = 2 };             // 16-bit operand type / output type

constexpr int kKB = 128;                                  // bytes of k per k-block

// The saved pre-activations of the gated block: the upper 24 bits of the fp32
// g and u (mantissa cut to 15 bits, relative error below 2^-15).  Rounding them
// to 16 bits instead would cost the gradients a third rounding of the size of
// the operands' own.  They lie in blocks of 32 x 32, row-block-major, as three
// planes of 16-bit words: g's upper half, u's upper half, their next 8 bits
// (g's in the low byte).  Inside a plane 8 columns of a row are 16 consecutive
// bytes and the 32 rows of these follow one another, so that a warp with a row
// in each lane, as the accumulators come, reads and writes 512 bytes at a time.
constexpr int kSavedPlane = 2048, kSavedBlock = 3 * kSavedPlane;
__host__ __device__ constexpr int64_t saved_bytes(int64_t T, int64_t I) {
  return ((T + 31) / 32) * ((I + 31) / 32) * kSavedBlock;
}
__device__ __forceinline__ int64_t saved_block(int64_t row, int64_t col, int64_t I) {
  return ((row >> 5) * ((I + 31) >> 5) + (col >> 5)) * kSavedBlock;
}
// Offset of an element's word inside its block's plane.
__device__ __forceinline__ int saved_word(int64_t row, int64_t col) {
  return static_cast<int>(((col & 31) >> 3) * 512 + (row & 31) * 16 + (col & 7) * 2);
}

// The planes' words of two neighbouring columns (e, o) from the fp32 bits of g
// and u.
__device__ __forceinline__ uint32_t saved_high(uint32_t e, uint32_t o) { return __byte_perm(e, o, 0x7632); }
__device__ __forceinline__ uint32_t saved_low(uint32_t ge, uint32_t ue, uint32_t go, uint32_t uo) {
  return __byte_perm(__byte_perm(ge, ue, 0x0051), __byte_perm(go, uo, 0x0051), 0x5410);
}
// g and u of column j (0, 1) of a pair of words.  The low byte that was cut
// repeats the one above it: a byte of zeros would take a second instruction.
__device__ __forceinline__ void saved_get(uint32_t gh, uint32_t uh, uint32_t lo, int j, float& g, float& u) {
  g = __uint_as_float(__byte_perm(gh, lo, j ? 0x3266 : 0x1044));
  u = __uint_as_float(__byte_perm(uh, lo, j ? 0x3277 : 0x1055));
}

struct Problem {
  int64_t M, N;   // rows and columns of the output
  int mt, nt;     // tiles
  int tile0;      // first tile id
  void* out;      // [M][N]
};

constexpr int kMaxProb = 3;
struct Args {
  CUtensorMap a[kMaxProb], b[kMaxProb];  // kGated: b[0] gate, b[1] up; segments or problems
  CUtensorMap o[kMaxProb];               // outputs, boxes of 32 rows x 64 bytes (kDGate: dg, du)
  Problem p[kMaxProb];
  int nprob;       // products in the launch (each with a[i], b[i])
  int nseg;        // k segments of one product (a[i], b[i] summed), 1 or 2; nprob 1 then
  int kblocks;     // k-blocks of a segment
  int tiles;
  int split;       // pairs that share a tile, 1 .. 4; with more than one, a cluster per tile
  uint32_t idesc;
  const uint16_t* residual;        // kPlain: [M][N] or NULL
  uint8_t* saved;                  // pre-activations: kGated writes them (NULL: no), kDGate reads
  const float *a_scale, *b_scale, *bias;  // kScaled
  bool tma_out;                    // output rows are 16-byte aligned: stored through o[]
  uint64_t timeout_ns;
};

// ---------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A cluster barrier that orders execution alone (no wait for this thread's
// stores to global memory to be seen).
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrives on a barrier of the cluster.  It orders no stores to global memory
// for the other CTA (released at cluster scope it waited 1300 cycles for them).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Stores 16 bytes into the shared memory of a CTA of the cluster and completes
// them on a barrier there.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t bar, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(addr),
      "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d)
      : "memory");
}
// mbar_wait for a barrier that other CTAs of the cluster complete with data.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                  uint64_t timeout_ns, unsigned site) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t n = 1;; ++n) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((n & 31u) == 0 && global_timer_ns() - t0 > timeout_ns) {
      record_status(site);
      *abort_flag = 1;
      return false;
    }
  }
}
// TMA load into this CTA's shared memory that signals `bar` (a shared::cluster
// address: the barrier of either CTA of the pair).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int32_t c0,
                                                 int32_t c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
template <int KIND>
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
  if constexpr (KIND == kF16Kind)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
template <int KIND>
__device__ __forceinline__ void umma_single(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t acc) {
  if constexpr (KIND == kF16Kind)
    umma_f16(d, a, b, idesc, acc);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs of the pair, ranks lead
// and lead + 1 of the cluster.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3u << lead))
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(slot)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Instruction descriptor: accumulator type, operand types (16-bit: fp16 0,
// bf16 1; 8-bit: signed 1), operand majors, tile size.
__host__ __device__ constexpr uint32_t make_idesc(int kind, int type, bool a_mn, bool b_mn, int M,
                                                  int N) {
  const uint32_t d = kind == kI8Kind ? 2u : 1u;
  const uint32_t ab = kind == kI8Kind ? 1u : (type == kF16 ? 0u : 1u);
  return (d << 4) | (ab << 7) | (ab << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
         (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// Shared-memory operand descriptors with the 128-byte swizzle.  K-major: as
// smem_desc_k128.  MN-major: 8-k groups 1024 bytes apart (stride offset),
// 64-wide chunks 8192 bytes apart (leading offset).
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  if constexpr (!MN) return smem_desc_k128(addr);
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (uint64_t(8192 >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// What one MMA's k (32 bytes) moves the descriptor's address by (in 16 bytes):
// K-major along the swizzled row, MN-major by 16 k-rows of 128 bytes.
template <bool MN>
constexpr uint64_t kDescStep = MN ? (16 * 128) >> 4 : 32 >> 4;

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type) {
  if (type == kF16) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ float unpack_lo(uint32_t v, int type) {
  return type == kF16 ? f16_lo(v) : bf16_lo(v);
}
__device__ __forceinline__ float unpack_hi(uint32_t v, int type) {
  return type == kF16 ? f16_hi(v) : bf16_hi(v);
}
__device__ __forceinline__ uint16_t pack1(float v, int type) {
  return type == kF16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ float unpack1(uint16_t v, int type) {
  return type == kF16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(uint32_t(v) << 16);
}

// 1 / (1 + e^-g) by the approximate exponential and reciprocal.  Relative error
// below 2^-21 (exponential 2^-22, sum 2^-24, reciprocal 2^-23) and, where
// e^-g counts, 1.25 |g| 2^-24 more: g log2(e) is rounded (2^-24 of it, the
// constant 2^-26), an absolute error of the exponent.  At g = -16 that is 2^-19.2
// together, where the 16-bit rounding that follows is 2^-11 at best.  Results
// below 2^-126 are flushed: without the flush their range handling was half of the
// epilogues' instructions.  For very negative g the exponential is infinite and
// the quotient 0, the limit.
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

// Gradients of silu(g) * u: du = dh silu(g), dg = dh u silu'(g), where
// silu' = s + g s (1 - s) = s (1 + g (1 - s)).
__device__ __forceinline__ void dgate(float dh, float g, float u, float& dg, float& du) {
  const float s = sigmoid(g);
  du = dh * (g * s);
  dg = (dh * u) * (s * fmaf(g, 1.f - s, 1.f));
}

// 32 consecutive fp32 columns of the calling warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld_32(uint32_t taddr, uint32_t (&a)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]),
        "=r"(a[7]), "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]),
        "=r"(a[14]), "=r"(a[15]), "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]),
        "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]), "=r"(a[24]), "=r"(a[25]),
        "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
      : "r"(taddr)
      : "memory");
}

// ---------------------------------------------------------------- block stores

constexpr int kStageRow = 64;
constexpr int kStageBlock = 32 * kStageRow;    // a warp's block of 32 rows x 64 bytes
constexpr int kStageWarp = 2 * kStageBlock;    // two of them

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\t"
               "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}

// A warp's block (lane = row, its 16 words in pk) into shared memory, with the
// 64-byte swizzle of the output maps: 16-byte pieces of a row swapped by its
// number, which keeps the writes free of bank conflicts.
__device__ __forceinline__ void stage_block(const uint32_t* pk, uint32_t block, int lane) {
  const uint32_t mine = block + lane * kStageRow;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    st_shared_v4(mine + ((q ^ (lane >> 1 & 3)) * 16), pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
}

// Stores a warp's block at column c0 (an element index) and row c1 by TMA,
// which leaves out what lies outside the matrix; `turn` alternates between the
// warp's two blocks of shared memory.  (Read back and stored by the warp's
// lanes, a block took 600 cycles instead of 420.)
__device__ __forceinline__ void store_block(const uint32_t* pk, uint32_t stage, int& turn, const CUtensorMap* map,
                                            int64_t c0, int64_t c1, int lane) {
  const uint32_t block = stage + turn * kStageBlock;
  turn ^= 1;
  // the store before the last one, from this block, has read it
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
  __syncwarp();
  stage_block(pk, block, lane);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) tma_store_2d(map, block, static_cast<int32_t>(c0), static_cast<int32_t>(c1));
}

// The same for rows that are not 16-byte aligned, element by element (of ES
// bytes), lanes along the row; nrows rows and ncols columns of the block exist.
// (int8, T = 8189, K = 1536, bf16: 131 us with N = 8191, 90 with 8192.)
template <int ES>
__device__ __forceinline__ void store_block_ragged(const uint32_t* pk, uint32_t block, uint8_t* g0, int64_t ld_bytes,
                                                   int nrows, int64_t ncols, int lane) {
  stage_block(pk, block, lane);
  __syncwarp();
  constexpr int PER = 64 / ES;  // elements of a row: 32 or 16
  const int col = lane % PER;
  for (int r = lane / PER; r < nrows; r += 32 / PER) {
    if (col < ncols) {
      if constexpr (ES == 2) {
        uint16_t v;
        asm volatile("ld.shared.b16 %0, [%1];"
                     : "=h"(v)
                     : "r"(block + r * kStageRow + ((col / 8 ^ (r >> 1 & 3)) * 16) + col % 8 * 2)
                     : "memory");
        *reinterpret_cast<uint16_t*>(g0 + r * ld_bytes + col * 2) = v;
      } else {
        uint32_t v;
        asm volatile("ld.shared.b32 %0, [%1];"
                     : "=r"(v)
                     : "r"(block + r * kStageRow + ((col / 4 ^ (r >> 1 & 3)) * 16) + col % 4 * 4)
                     : "memory");
        *reinterpret_cast<uint32_t*>(g0 + r * ld_bytes + col * 4) = v;
      }
    }
  }
  __syncwarp();
}

// 32 consecutive 16-bit words of a row (16-byte aligned, `ncols` of them
// exist, a multiple of 8) as 16 packed pairs; what does not exist reads 0.
__device__ __forceinline__ void load_row32(const uint16_t* p, bool row_ok, int64_t ncols,
                                           uint32_t (&v)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 t = make_uint4(0u, 0u, 0u, 0u);
    if (row_ok && (q + 1) * 8 <= ncols) t = *reinterpret_cast<const uint4*>(p + q * 8);
    v[4 * q] = t.x; v[4 * q + 1] = t.y; v[4 * q + 2] = t.z; v[4 * q + 3] = t.w;
  }
}

// ---------------------------------------------------------------- the pair kernel

constexpr int kBM = 256;          // tile rows (128 per CTA)
// Two epilogue warps for each 32-lane quarter of tensor memory, taking its
// 32-column chunks in turn.  (12 warps of 128 registers a thread made the int8
// product 2% faster, but the gated one and its gradient 3 to 4% slower at
// T = 8189, where the card's power bounds them; 16 warps of 96 slowed all.)
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 32 * (kEpiWarps + 2);
constexpr int kABytes = 128 * kKB;
constexpr int kPartBytes = 8 * 128 * 16;  // 32 accumulator columns of 128 rows
constexpr int kMaxPairs = 4;               // pairs of a cluster (of 8 CTAs)
template <int BN>
struct PairCfg {
  static constexpr int B_BYTES = BN / 2 * kKB;
  static constexpr int STAGE = kABytes + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 6 : 8;
  static constexpr int SETS = 2;                          // accumulator sets of BN columns
  static constexpr int TMEM = SETS * BN;
  static constexpr int SMEM = STAGES * STAGE + kEpiWarps * kStageWarp + 1024 + 256;
};
struct PairTail {
  uint64_t full[8], empty[8], tfull[2], tempty[2], drain, parts;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PairTail) <= 256, "barriers fit their place");

// Tile t of a launch: product q and tile coordinates.  Within a product the
// tiles run over groups of 8 tile rows, row fastest, so that the clusters at
// work at one time share rows of A and columns of B through L2.
__device__ __forceinline__ void decode(const Args& g, int t, int& q, int& m, int& n) {
  q = 0;
  while (q + 1 < g.nprob && g.p[q + 1].tile0 <= t) ++q;
  const int mt = g.p[q].mt, nt = g.p[q].nt;
  t -= g.p[q].tile0;
  const int per = 8 * nt, grp = t / per, rem = t - grp * per;
  const int rows = min(8, mt - grp * 8);
  n = rem / rows;
  m = grp * 8 + (rem - n * rows);
}

template <int KIND, bool A_MN, bool B_MN, int EPI, int BN, int TYPE>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ Args g) {
  using C = PairCfg<BN>;
  constexpr int KE = KIND == kI8Kind ? 128 : 64;  // elements of a k-block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sEpi = smem + C::STAGES * C::STAGE;
  PairTail* S = reinterpret_cast<PairTail*>(sEpi + kEpiWarps * kStageWarp);
  volatile int* abort_flag = &S->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // rank in the pair, the pair in the cluster, the cluster rank of its CTA 0
  const uint32_t crank = cluster_rank(), rank = crank & 1, pair = crank >> 1, lead = crank & ~1u;
  // 32-column chunks of a tile's output, and those this pair stores
  constexpr int NCH = (EPI == kGated ? BN / 2 : BN) / 32, G = EPI == kGated ? 2 : 1;
  const int chunk0 = NCH * pair / g.split, chunk1 = NCH * (pair + 1) / g.split;
  constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&S->full[s], 1);
      mbar_init(&S->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&S->tfull[a], 1);
      mbar_init(&S->tempty[a], 2 * kEpiWarps);
    }
    mbar_init(&S->drain, 1);
    mbar_init(&S->parts, 1);
    S->abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(&S->parts, (g.split - 1) * (chunk1 - chunk0) * G * kPartBytes);
  }
  if (warp == kTmaWarp && lane == 0) {
    for (int i = 0; i < kMaxProb; ++i) {
      if (g.tma_out && i < g.nprob + (EPI == kDGate)) tma_prefetch_desc(&g.o[i]);
      if (i < max(g.nprob, g.nseg)) tma_prefetch_desc(&g.a[i]);
      if (i < max(g.nprob, g.nseg) + (EPI == kGated)) tma_prefetch_desc(&g.b[i]);
    }
  }
  __syncwarp();
  if (warp == kMmaWarp) tmem_alloc_pair(&S->tmem_base, C::TMEM);
  tc_fence_before();
  cluster_sync();  // every CTA's barriers exist before another signals them
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  griddep_wait();
  griddep_launch_dependents();

  const int cluster = blockIdx.x / (2 * g.split), nclusters = gridDim.x / (2 * g.split);
  const int kbs = g.kblocks * g.nseg, kb0 = kbs * pair / g.split, kb1 = kbs * (pair + 1) / g.split;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = cluster; ok && t < g.tiles; t += nclusters) {
        int q, m, n;
        decode(g, t, q, m, n);
        const int m0 = m * kBM + static_cast<int>(rank) * 128;
        // kGated: CTA 0 brings the gate columns, CTA 1 the up columns
        const int n0 = EPI == kGated ? n * (BN / 2) : n * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (!mbar_wait(&S->empty[s], ((it / C::STAGES) & 1) ^ 1, abort_flag, g.timeout_ns, kSiteEmpty)) {
            ok = false;
            break;
          }
          const int seg = kb >= g.kblocks ? 1 : 0;
          const int k0 = (kb - seg * g.kblocks) * KE;
          const CUtensorMap* ma = &g.a[q + seg];
          const CUtensorMap* mb = EPI == kGated ? &g.b[rank] : &g.b[q + seg];
          const uint32_t sa = smem_u32(smem + s * C::STAGE), sb = sa + kABytes;
          // both CTAs' bytes complete on the barrier of CTA 0, which issues the MMAs
          if (rank == 0) mbar_arrive_expect_tx(&S->full[s], 2 * C::STAGE);
          const uint32_t bar = map_to_rank(smem_u32(&S->full[s]), lead);
          if constexpr (A_MN) {
            tma_load_2d_pair(sa, ma, m0, k0, bar);
            tma_load_2d_pair(sa + 8192, ma, m0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(sa, ma, k0, m0, bar);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int c = 0; c < BN / 128; ++c) tma_load_2d_pair(sb + c * 8192, mb, n0 + c * 64, k0, bar);
          } else {
            tma_load_2d_pair(sb, mb, k0, n0, bar);
          }
        }
      }
      // After a wait that ran out, let the copies in flight land before either
      // CTA can exit (otherwise the MMAs have consumed them all).  CTA 1's
      // signal CTA 0's barriers, which it cannot wait on: it gives them 1 ms.
      if (!ok && rank == 0)
        for (int i = max(0, it - C::STAGES); i < it; ++i)
          mbar_wait_drain(&S->full[i % C::STAGES], (i / C::STAGES) & 1, kSiteDrain);
      if (!ok && rank == 1)
        for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 1000000ull;) __nanosleep(1000);
    }
  } else if (warp == kMmaWarp) {
    if (rank == 0 && lane == 0) {
      int it = 0, n_tile = 0;
      bool ok = true;
      for (int t = cluster; ok && t < g.tiles; t += nclusters, ++n_tile) {
        const int a = n_tile & 1;
        if (!mbar_wait(&S->tempty[a], ((n_tile >> 1) & 1) ^ 1, abort_flag, g.timeout_ns, kSiteTmemEmpty)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + a * BN;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (!mbar_wait(&S->full[s], (it / C::STAGES) & 1, abort_flag, g.timeout_ns, kSiteFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * C::STAGE);
          const uint64_t da = operand_desc<A_MN>(sa), db = operand_desc<B_MN>(sa + kABytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_pair<KIND>(d, da + k * kDescStep<A_MN>, db + k * kDescStep<B_MN>, g.idesc, kb != kb0 || k != 0);
          umma_commit_pair(&S->empty[s], lead);
        }
        if (ok) umma_commit_pair(&S->tfull[a], lead);
      }
      if (!ok) {  // wait for the MMAs already issued
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_u32(&S->drain))
            : "memory");
        mbar_wait_drain(&S->drain, 0, kSiteDrain);
      }
    }
  } else {
    // ---------------------------------------------- epilogue
    const int quarter = warp & 3, sub = warp >> 2;
    const uint32_t stage = smem_u32(sEpi + warp * kStageWarp);
    int n_tile = 0, turn = 0;
    for (int t = cluster; t < g.tiles; t += nclusters, ++n_tile) {
      int q, m, n;
      decode(g, t, q, m, n);
      const int a = n_tile & 1;
      const Problem& P = g.p[q];
      const int64_t row0 = int64_t(m) * kBM + rank * 128 + quarter * 32, row = row0 + lane;
      const int nrows = static_cast<int>(min(int64_t(32), max(int64_t(0), P.M - row0)));
      const bool row_ok = row < P.M;
      // kScaled: the row's scale, and the scale and bias of one column of the
      // warp's next chunk in each lane
      float sa = 0.f, sb = 0.f, bi = 0.f;
      auto column_scales = [&](int ch) {
        const int64_t c = int64_t(n) * BN + ch * 32 + lane;
        const bool in = ch < chunk1 && c < P.N;
        sb = in ? g.b_scale[c] : 0.f;
        bi = in && g.bias != nullptr ? g.bias[c] : 0.f;
      };
      if constexpr (EPI == kScaled) {
        if (row_ok) sa = g.a_scale[row];
        column_scales(chunk0 + sub);
      }
      const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&S->tfull[a], (n_tile >> 1) & 1, abort_flag,
                                                        g.timeout_ns, kSiteTmemFull));
      if (!ok && g.split == 1) break;
      tc_fence_after();
      const uint32_t d = tmem + a * BN + (uint32_t(quarter * 32) << 16);
      // Shared tile: once every CTA's products are done, its stages' memory
      // takes the other pairs' accumulators, slot (sending pair, chunk of the
      // owner's, gate or up), as 8 x 128 rows of 16 bytes.  After a wait that
      // ran out there is something to send all the same, for no owner to wait in vain.
      const uint32_t parts = smem_u32(smem);
      const int maxch = (NCH + g.split - 1) / g.split;
      if (g.split > 1) {
        cluster_sync();
        for (int o = 0; o < g.split; ++o) {
          if (o == static_cast<int>(pair)) continue;
          const uint32_t to_bar = map_to_rank(smem_u32(&S->parts), 2 * o + rank);
          const int o0 = NCH * o / g.split, o1 = NCH * (o + 1) / g.split;
#pragma unroll 1
          for (int i = o0 * G + sub; i < o1 * G; i += kEpiWarps / 4) {
            const int ch = i / G, gi = i % G;
            uint32_t v[32];
            tmem_ld_32(d + gi * (BN / 2) + ch * 32, v);
            const uint32_t slot = ((pair * maxch + ch - o0) * G + gi) * kPartBytes + (quarter * 32 + lane) * 16;
            const uint32_t to = map_to_rank(parts + slot, 2 * o + rank);
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4)
              st_async_v4(to + c4 * 2048, to_bar, v[4 * c4], v[4 * c4 + 1], v[4 * c4 + 2], v[4 * c4 + 3]);
          }
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&S->parts, 0, abort_flag, 4 * g.timeout_ns, kSiteParts)) || !ok)
          break;
      }
      auto add_parts = [&](int ch, int gi, uint32_t (&v)[32]) {
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          uint4 own = make_uint4(v[4 * c4], v[4 * c4 + 1], v[4 * c4 + 2], v[4 * c4 + 3]), sum = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
          for (int r = 0; r < g.split; ++r) {
            const uint4 w = r == static_cast<int>(pair)
                                ? own
                                : ld_shared_v4(parts + ((r * maxch + ch - chunk0) * G + gi) * kPartBytes + c4 * 2048 +
                                               (quarter * 32 + lane) * 16);
            if constexpr (KIND == kI8Kind) {
              sum.x += w.x; sum.y += w.y; sum.z += w.z; sum.w += w.w;
            } else {
              sum.x = __float_as_uint(__uint_as_float(sum.x) + __uint_as_float(w.x));
              sum.y = __float_as_uint(__uint_as_float(sum.y) + __uint_as_float(w.y));
              sum.z = __float_as_uint(__uint_as_float(sum.z) + __uint_as_float(w.z));
              sum.w = __float_as_uint(__uint_as_float(sum.w) + __uint_as_float(w.w));
            }
          }
          v[4 * c4] = sum.x; v[4 * c4 + 1] = sum.y; v[4 * c4 + 2] = sum.z; v[4 * c4 + 3] = sum.w;
        }
      };
      // this warp's chunks; after its last tensor memory read the accumulators
      // go back to the MMAs
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&S->tempty[a]), lead));
      };
      if (chunk0 + sub >= chunk1) release();
#pragma unroll 1
      for (int ch = chunk0 + sub; ch < chunk1; ch += kEpiWarps / 4) {
        const int lc = ch * 32;
        const int64_t col = int64_t(n) * (EPI == kGated ? BN / 2 : BN) + lc, left = P.N - col;
        const bool any = left > 0 && nrows > 0;
        uint4 now[EPI == kDGate ? 12 : 1];
        if constexpr (EPI == kDGate) {
          // read once, and not before much else has passed through L2
          if (any) {
            const uint4* from = reinterpret_cast<const uint4*>(g.saved + saved_block(row0, col, P.N)) + lane;
#pragma unroll
            for (int i = 0; i < 12; ++i) now[i] = __ldcs(from + i * 32);
          }
        }
        uint32_t x[32], x1[EPI == kGated ? 32 : 1];
        if constexpr (EPI == kGated)
          tmem_ld_2x32(d + lc, d + BN / 2 + lc, x, x1);
        else
          tmem_ld_32(d + lc, x);
        if (ch + kEpiWarps / 4 >= chunk1) release();
        if (!any) continue;
        if (g.split > 1) {
          add_parts(ch, 0, x);
          if constexpr (EPI == kGated) add_parts(ch, 1, x1);
        }
        const int64_t at = row0 * P.N + col;
        uint32_t pk[16];
        if constexpr (EPI == kGated) {
          if (g.saved != nullptr) {
            uint4* to = reinterpret_cast<uint4*>(g.saved + saved_block(row0, col, P.N)) + lane;
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const uint32_t *e = x + 8 * q4, *f = x1 + 8 * q4;
              __stcs(to + q4 * 32, make_uint4(saved_high(e[0], e[1]), saved_high(e[2], e[3]), saved_high(e[4], e[5]), saved_high(e[6], e[7])));
              __stcs(to + (4 + q4) * 32, make_uint4(saved_high(f[0], f[1]), saved_high(f[2], f[3]), saved_high(f[4], f[5]), saved_high(f[6], f[7])));
              __stcs(to + (8 + q4) * 32, make_uint4(saved_low(e[0], f[0], e[1], f[1]), saved_low(e[2], f[2], e[3], f[3]),
                                             saved_low(e[4], f[4], e[5], f[5]), saved_low(e[6], f[6], e[7], f[7])));
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack2(silu(__uint_as_float(x[2 * i])) * __uint_as_float(x1[2 * i]),
                          silu(__uint_as_float(x[2 * i + 1])) * __uint_as_float(x1[2 * i + 1]), TYPE);
          store_block(pk, stage, turn, &g.o[0], col, row0, lane);
        } else if constexpr (EPI == kPlain) {
          if (g.residual != nullptr) {
            uint32_t r[16];
            load_row32(g.residual + at + lane * P.N, row_ok, left, r);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pk[i] = pack2(__uint_as_float(x[2 * i]) + unpack_lo(r[i], TYPE),
                            __uint_as_float(x[2 * i + 1]) + unpack_hi(r[i], TYPE), TYPE);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pk[i] = pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), TYPE);
          }
          store_block(pk, stage, turn, &g.o[q], col, row0, lane);
        } else if constexpr (EPI == kDGate) {
          uint32_t pg[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t hw = (&now[i / 4].x)[i % 4], uw = (&now[4 + i / 4].x)[i % 4], lw = (&now[8 + i / 4].x)[i % 4];
            float dg[2], du[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float gg, uu;
              saved_get(hw, uw, lw, j, gg, uu);
              dgate(__uint_as_float(x[2 * i + j]), gg, uu, dg[j], du[j]);
            }
            pg[i] = pack2(dg[0], dg[1], TYPE);
            pk[i] = pack2(du[0], du[1], TYPE);
          }
          store_block(pg, stage, turn, &g.o[0], col, row0, lane);
          store_block(pk, stage, turn, &g.o[1], col, row0, lane);
        } else {
          // the 32 columns' values to every lane, through the block that is stored next
          const uint32_t scales = stage + turn * kStageBlock;
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + lane * 4), "f"(sb) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + 128 + lane * 4), "f"(bi) : "memory");
          __syncwarp();
          column_scales(ch + kEpiWarps / 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 s4 = ld_shared_v4(scales + i * 16), b4 = ld_shared_v4(scales + 128 + i * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t& v = x[4 * i + j];
              v = __float_as_uint(fmaf(static_cast<float>(static_cast<int>(v)) * sa, __uint_as_float((&s4.x)[j]),
                                       __uint_as_float((&b4.x)[j])));
            }
          }
          __syncwarp();
          constexpr int ES = TYPE == kF32 ? 4 : 2, NB = TYPE == kF32 ? 2 : 1, PER = 64 / ES;  // blocks, their columns
          if constexpr (TYPE != kF32) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              x[i] = pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), TYPE);
          }
#pragma unroll
          for (int f = 0; f < NB; ++f) {
            if (left <= f * PER) break;
            if (g.tma_out)
              store_block(x + f * 16, stage, turn, &g.o[0], col + f * PER, row0, lane);
            else
              store_block_ragged<ES>(x + f * 16, stage, static_cast<uint8_t*>(P.out) + (at + f * PER) * ES, P.N * ES,
                                     nrows, left - f * PER, lane);
          }
        }
      }
    }
    // the stores have been made before the block exits
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  if (g.split > 1 && warp >= kEpiWarps) {  // the epilogue warps' barrier after the products
    __syncwarp();
    cluster_sync();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_relaxed();  // neither CTA leaves while the other may still signal it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM);
  }
}

}  // namespace dense
}  // namespace moe
