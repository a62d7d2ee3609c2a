// dense_small.cuh -- the products of dense.cuh for few tokens, where reading
// the weights is all that counts.
//
// The weights are the 128-row operand of the MMA (their n on the accumulator's
// lanes) and up to NT tokens its columns, so no tensor-core row is spent on
// padding tokens, and 128 x K weight bytes stream through each CTA.  With few
// weight tiles the k range is split over the CTAs of a cluster.  Each CTA owns
// a share of the tile's outputs; every CTA sends the parts of its accumulators
// to their owners' shared memory (st.async, counted on the owner's barrier),
// and the owner adds them up in rank order, so the result does not depend on
// timing, and runs the epilogue.  One launch, no workspace, no atomics, and no
// cluster barrier after the products: gathering by a barrier, loads from the
// other CTAs and a second barrier took 1.5 us more of a 6 us launch.
#pragma once
#include "dense.cuh"

namespace moe {
namespace dense {

constexpr int kSmallThreads = 256;
constexpr int kMaxSplit = 8;

// ROWS weight rows of a tile: 128 (kGated: 64 gate and 64 up columns), or 64
// where tiles of 128 cannot occupy the SMs.  The MMA is 128 rows high in both
// cases; with 64 the upper accumulator rows are products of whatever lies
// behind the weights in shared memory, and are not read.
template <int NT, int ROWS>
struct SmallCfg {
  static constexpr int STAGE = ROWS * kKB + NT * kKB;
  // 50 to 70 KB in flight; two or three CTAs fit on an SM.  With 5 stages of
  // 128 rows, and two CTAs, T = 1 (H = 1536, I = 4096) took 14.7 us, not 13.7.
  static constexpr int STAGES = ROWS == 64 && NT <= 32 ? 5 : 3;
  // Parts lie as [sending rank][4 tokens][the owner's rows], 16 bytes a row, so
  // that a warp's rows are sent as whole lines (with a row's tokens together,
  // 64 tokens took 3.6 us to send).
  static constexpr int GROUPS = NT / 4;
  static constexpr int PART = ROWS * NT * 4;
  static constexpr int SMEM = STAGES * STAGE + PART + 1024 + 256 + (ROWS == 64 ? 2048 : 0);
  static constexpr int TMEM = NT < 32 ? 32 : NT;
  static constexpr int PER_SM = 232448 / (SMEM + 1024);  // CTAs an SM's shared memory holds
  static_assert((STAGES - 1) * STAGE + 128 * kKB <= SMEM - 1024, "the MMA's rows stay inside");
  // Too large to share an SM with a kernel that takes all its tensor memory
  // (those take 193 KB and more): a cluster whose CTAs wait for tensor memory
  // that such a kernel holds, while that kernel waits for some they hold,
  // cannot arise.
  static_assert(SMEM > 40 * 1024, "shares no SM with the persistent kernels");
};
struct SmallTail {
  uint64_t full[8], empty[8], done, parts;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(SmallTail) <= 256, "barriers fit their place");

struct SmallArgs {
  CUtensorMap w[2], x[2];  // weights (kGated: gate, up), tokens; a segment each
  int64_t T, N;            // tokens; weight columns (outputs per token)
  int wt;                  // weight tiles
  int nseg, kblocks;       // k segments, k-blocks of a segment
  int split;               // CTAs of a cluster, 1 .. kMaxSplit
  int type;
  uint32_t idesc;
  void* out;
  const uint16_t* residual;
  uint8_t* saved;
  void* out2;
  const float *a_scale, *b_scale, *bias;
  uint64_t timeout_ns;
};

template <int KIND, bool W_MN, int EPI, int NT, int ROWS>
__global__ void __launch_bounds__(kSmallThreads)
    small_gemm_kernel(const __grid_constant__ SmallArgs g) {
  using C = SmallCfg<NT, ROWS>;
  static_assert(EPI != kGated || ROWS == 128, "64 gate and 64 up columns");
  constexpr int KE = KIND == kI8Kind ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sPart = smem + C::STAGES * C::STAGE;
  SmallTail* S = reinterpret_cast<SmallTail*>(sPart + C::PART);
  volatile int* abort_flag = &S->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
  const int wtile = tile % g.wt, ttile = tile / g.wt;
  const int64_t t0 = int64_t(ttile) * NT;
  const int ntok = static_cast<int>(min(int64_t(NT), g.T - t0));
  const int ngrp = (ntok + 3) / 4;  // tokens are sent four at a time

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&S->full[s], 1);
      mbar_init(&S->empty[s], 1);
    }
    mbar_init(&S->done, 1);
    mbar_init(&S->parts, 1);
    S->abort_flag = 0;
    fence_barrier_init();
    mbar_arrive_expect_tx(&S->parts, ngrp * ROWS * 16);
  }
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < g.nseg; ++i) tma_prefetch_desc(&g.x[i]);
    tma_prefetch_desc(&g.w[0]);
    if (EPI == kGated || g.nseg > 1) tma_prefetch_desc(&g.w[1]);
  }
  __syncwarp();
  if (warp == 1) tmem_alloc(&S->tmem_base, C::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S->tmem_base;
  cluster_arrive();  // waited for before anything is sent: the barriers of all ranks exist then

  // this CTA's k-blocks: an even share of all segments' blocks
  const int kbs = g.kblocks * g.nseg;
  const int kb0 = static_cast<int>(int64_t(kbs) * rank / g.split);
  const int kb1 = static_cast<int>(int64_t(kbs) * (rank + 1) / g.split);

  auto load_w = [&](int kb, int s) {  // k-block kb of the weights into stage s
    const int seg = kb >= g.kblocks ? 1 : 0;
    const int k0 = (kb - seg * g.kblocks) * KE;
    const uint32_t sw = smem_u32(smem + s * C::STAGE);
    mbar_arrive_expect_tx(&S->full[s], C::STAGE);
    if constexpr (EPI == kGated) {
      tma_load_2d(sw, &g.w[0], wtile * 64, k0, &S->full[s]);
      tma_load_2d(sw + 8192, &g.w[1], wtile * 64, k0, &S->full[s]);
    } else if constexpr (W_MN) {
#pragma unroll
      for (int c = 0; c < ROWS / 64; ++c)
        tma_load_2d(sw + c * 8192, &g.w[seg], wtile * ROWS + c * 64, k0, &S->full[s]);
    } else {
      tma_load_2d(sw, &g.w[seg], k0, wtile * ROWS, &S->full[s]);
    }
  };
  griddep_wait();
  griddep_launch_dependents();

  // The outputs this CTA owns: unit e is column e % own of its share and the 4
  // tokens from e / own * 4 on.  What the epilogue reads of a thread's next
  // unit is loaded ahead, the first one's during the products (after their own
  // part by the two warps that drive them: they would start later).
  constexpr int PER = EPI == kGated ? 64 : ROWS;
  const int own = PER / g.split;                // output columns a rank owns
  const int rows = ROWS / g.split;              // rows of a part
  const uint32_t parts = smem_u32(sPart);
  const int64_t col0 = int64_t(wtile) * PER + rank * own;
  float pre[EPI == kScaled ? 6 : EPI == kDGate ? 8 : EPI == kPlain ? 4 : 1];
  auto fetch = [&](int e) {
    const int64_t col = col0 + e % own;
    const int tok = e / own * 4;
    if (e >= ngrp * own || col >= g.N) return;
    if constexpr (EPI == kScaled) {
      pre[4] = g.b_scale[col];
      pre[5] = g.bias != nullptr ? g.bias[col] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = t0 + min(tok + i, ntok - 1);
      if constexpr (EPI == kScaled) pre[i] = g.a_scale[row];
      if constexpr (EPI == kPlain)
        pre[i] = g.residual != nullptr ? unpack1(g.residual[row * g.N + col], g.type) : 0.f;
      if constexpr (EPI == kDGate) {
        const uint8_t* sv = g.saved + saved_block(row, col, g.N) + saved_word(row, col);
        saved_get(*reinterpret_cast<const uint16_t*>(sv), *reinterpret_cast<const uint16_t*>(sv + kSavedPlane),
                  *reinterpret_cast<const uint16_t*>(sv + 2 * kSavedPlane), 0, pre[i], pre[4 + i]);
      }
    }
  };
  if (warp >= 2) fetch(threadIdx.x);

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % C::STAGES;
        if (!mbar_wait(&S->empty[s], ((it / C::STAGES) & 1) ^ 1, abort_flag, g.timeout_ns, kSiteSmallEmpty)) {
          ok = false;
          break;
        }
        const int seg = kb >= g.kblocks ? 1 : 0;
        const int k0 = (kb - seg * g.kblocks) * KE;
        load_w(kb, s);
        tma_load_2d(smem_u32(smem + s * C::STAGE) + ROWS * kKB, &g.x[seg], k0, ttile * NT, &S->full[s]);
      }
      if (!ok)  // let the copies already issued land before the block can exit
        for (int i = max(0, it - C::STAGES); i < it; ++i)
          mbar_wait_drain(&S->full[i % C::STAGES], (i / C::STAGES) & 1, kSiteDrain);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % C::STAGES;
        if (!mbar_wait(&S->full[s], (it / C::STAGES) & 1, abort_flag, g.timeout_ns, kSiteSmallFull)) break;
        tc_fence_after();
        const uint32_t sw = smem_u32(smem + s * C::STAGE);
        const uint64_t dw = operand_desc<W_MN>(sw), dx = operand_desc<false>(sw + ROWS * kKB);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_single<KIND>(tmem, dw + k * kDescStep<W_MN>, dx + k * kDescStep<false>, g.idesc, (it | k) != 0);
        umma_commit(&S->empty[s]);
      }
      umma_commit(&S->done);  // after a wait that ran out too: the MMAs already issued
    }
  }
  __syncwarp();
  if (warp < 2) fetch(threadIdx.x);
  bool ok = mbar_wait(&S->done, 0, abort_flag, 2 * g.timeout_ns, kSiteSmallDone);
  ok = __syncthreads_and(ok && !*abort_flag) != 0;
  tc_fence_after();

  // accumulators -> their owners: weight row r (kGated: gate row r and up row
  // 64 + r) belongs to rank r / OWN.  A CTA without k-blocks, or whose wait ran
  // out, sends zeros, so that no owner waits for it in vain.
  cluster_wait();
  {
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const int owner = r % PER / own, local = r / PER * own + r % PER % own;
    const uint32_t to = map_to_rank(parts + (rank * C::GROUPS * rows + local) * 16, owner);
    const uint32_t bar = map_to_rank(smem_u32(&S->parts), owner);
    const bool have = ok && kb1 > kb0;
    for (int c = (warp >> 2) * 8; c < ntok && quarter * 32 < ROWS; c += 16) {
      uint32_t v[8];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
          "tcgen05.wait::ld.sync.aligned;"
          : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
          : "r"(tmem + c + (uint32_t(quarter * 32) << 16))
          : "memory");
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (c + 4 * h < ntok)
          st_async_v4(to + (c / 4 + h) * rows * 16, bar, have ? v[4 * h] : 0u, have ? v[4 * h + 1] : 0u,
                      have ? v[4 * h + 2] : 0u, have ? v[4 * h + 3] : 0u);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
  // every rank sends within its own waits' limits
  if (!mbar_wait_cluster(&S->parts, 0, abort_flag, 4 * g.timeout_ns, kSiteSmallParts)) return;

  auto total = [&](int local, int grp, float (&sum)[4]) {  // sums over the ranks, in rank order
    const uint32_t at = parts + (grp * rows + local) * 16;
    if constexpr (KIND == kI8Kind) {
      int a[4] = {0, 0, 0, 0};
#pragma unroll 4
      for (int r = 0; r < g.split; ++r) {
        const uint4 v = ld_shared_v4(at + r * C::GROUPS * rows * 16);
        a[0] += int(v.x); a[1] += int(v.y); a[2] += int(v.z); a[3] += int(v.w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = static_cast<float>(a[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = 0.f;
#pragma unroll 4
      for (int r = 0; r < g.split; ++r) {
        const uint4 v = ld_shared_v4(at + r * C::GROUPS * rows * 16);
        sum[0] += __uint_as_float(v.x); sum[1] += __uint_as_float(v.y);
        sum[2] += __uint_as_float(v.z); sum[3] += __uint_as_float(v.w);
      }
    }
  };
  for (int e = threadIdx.x; e < ngrp * own; e += kSmallThreads) {
    const int local = e % own, grp = e / own;
    const int64_t col = col0 + local;
    if (col < g.N) {
      float y[4], z[4];
      total(local, grp, y);
      if constexpr (EPI == kGated) total(own + local, grp, z);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = t0 + grp * 4 + i, at = row * g.N + col;
        if (grp * 4 + i >= ntok) break;
        if constexpr (EPI == kGated) {
          if (g.saved != nullptr) {
            uint8_t* sv = g.saved + saved_block(row, col, g.N) + saved_word(row, col);
            const uint32_t gb = __float_as_uint(y[i]), ub = __float_as_uint(z[i]);
            *reinterpret_cast<uint16_t*>(sv) = static_cast<uint16_t>(gb >> 16);
            *reinterpret_cast<uint16_t*>(sv + kSavedPlane) = static_cast<uint16_t>(ub >> 16);
            *reinterpret_cast<uint16_t*>(sv + 2 * kSavedPlane) = static_cast<uint16_t>(saved_low(gb, ub, 0u, 0u));
          }
          y[i] = silu(y[i]) * z[i];
        } else if constexpr (EPI == kPlain) {
          y[i] += pre[i];
        } else if constexpr (EPI == kDGate) {
          float du;
          dgate(y[i], pre[i], pre[4 + i], y[i], du);
          static_cast<uint16_t*>(g.out2)[at] = pack1(du, g.type);
        } else {
          y[i] = fmaf(y[i] * pre[i], pre[4], pre[5]);
          if (g.type == kF32) {
            static_cast<float*>(g.out)[at] = y[i];
            continue;
          }
        }
        static_cast<uint16_t*>(g.out)[at] = pack1(y[i], g.type);
      }
    }
    fetch(e + kSmallThreads);
  }
}

}  // namespace dense
}  // namespace moe
