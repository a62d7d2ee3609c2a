// dense_small.cuh -- the products of dense.cuh for few tokens, where reading
// the weights is all that counts.
//
// The weights are the 128-row operand of the MMA (their n on the accumulator's
// lanes) and up to NT tokens its columns, so no tensor-core row is spent on
// padding tokens, and 128 x K weight bytes stream through each CTA.  With few
// weight tiles the k range is split over the CTAs of a cluster: each leaves its
// partial accumulators in its shared memory, and after a cluster barrier every
// CTA adds up its share of the outputs from all of them, in rank order (so the
// result does not depend on timing), and runs the epilogue on it.  One launch,
// no workspace, no atomics.
#pragma once
#include "dense.cuh"

namespace moe {
namespace dense {

constexpr int kSmallThreads = 256;
constexpr int kMaxSplit = 8;
constexpr int kSmallRows = 128;  // weight rows of a tile (kGated: 64 gate and 64 up columns)

template <int NT>
struct SmallCfg {
  static constexpr int STAGE = kSmallRows * kKB + NT * kKB;
  // up to 110 KB a CTA, so that two share an SM (and the next launch's CTAs
  // can start reading while the last ones of this one finish)
  static constexpr int STAGES = NT <= 32 ? 5 : NT == 64 ? 4 : 3;
  static constexpr int PART = NT * kSmallRows * 4;  // reuses the stages' memory
  static constexpr int SMEM = STAGES * STAGE + 1024 + 256;
  static constexpr int TMEM = NT < 32 ? 32 : NT;
  static_assert(PART <= STAGES * STAGE, "partial sums fit the stages");
};
struct SmallTail {
  uint64_t full[8], empty[8], done;
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
  bool early;              // the weights may be read before the preceding launch has finished
  int type;
  uint32_t idesc;
  void* out;
  const uint16_t* residual;
  uint8_t* saved;
  void* out2;
  const float *a_scale, *b_scale, *bias;
  uint64_t timeout_ns;
};

template <int KIND, bool W_MN, int EPI, int NT>
__global__ void __launch_bounds__(kSmallThreads)
    small_gemm_kernel(const __grid_constant__ SmallArgs g) {
  using C = SmallCfg<NT>;
  constexpr int KE = KIND == kI8Kind ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  SmallTail* S = reinterpret_cast<SmallTail*>(smem + C::STAGES * C::STAGE);
  volatile int* abort_flag = &S->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
  const int wtile = tile % g.wt, ttile = tile / g.wt;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&S->full[s], 1);
      mbar_init(&S->empty[s], 1);
    }
    mbar_init(&S->done, 1);
    S->abort_flag = 0;
    fence_barrier_init();
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
      tma_load_2d(sw, &g.w[seg], wtile * 128, k0, &S->full[s]);
      tma_load_2d(sw + 8192, &g.w[seg], wtile * 128 + 64, k0, &S->full[s]);
    } else {
      tma_load_2d(sw, &g.w[seg], k0, wtile * 128, &S->full[s]);
    }
  };
  // Where the launch before this one is a step of the same call (which waited
  // for everything before it), the weights are no output of it: their first
  // stages are read while it still runs.
  int ahead = 0;
  if (g.early && warp == 0 && lane == 0)
    for (; ahead < C::STAGES && kb0 + ahead < kb1; ++ahead) load_w(kb0 + ahead, ahead);
  griddep_wait();
  griddep_launch_dependents();

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
        if (it >= ahead) load_w(kb, s);
        tma_load_2d(smem_u32(smem + s * C::STAGE) + kSmallRows * kKB, &g.x[seg], k0, ttile * NT, &S->full[s]);
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
        const uint64_t dw = operand_desc<W_MN>(sw), dx = operand_desc<false>(sw + kSmallRows * kKB);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_single<KIND>(tmem, dw + k * kDescStep<W_MN>, dx + k * kDescStep<false>, g.idesc, (it | k) != 0);
        umma_commit(&S->empty[s]);
      }
      umma_commit(&S->done);  // after a wait that ran out too: the MMAs already issued
    }
  }
  __syncwarp();
  bool ok = mbar_wait(&S->done, 0, abort_flag, 2 * g.timeout_ns, kSiteSmallDone);
  ok = __syncthreads_and(ok && !*abort_flag) != 0;
  tc_fence_after();

  // accumulators -> this CTA's partial sums [token][weight row], fp32 (or int32)
  uint32_t* part = reinterpret_cast<uint32_t*>(smem);
  if (ok && kb1 > kb0) {
    const int quarter = warp & 3;
#pragma unroll
    for (int c = (warp >> 2) * 8; c < NT; c += 16) {
      uint32_t v[8];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
          "tcgen05.wait::ld.sync.aligned;"
          : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
          : "r"(tmem + c + (uint32_t(quarter * 32) << 16))
          : "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i) part[(c + i) * kSmallRows + quarter * 32 + lane] = v[i];
    }
  } else {  // no k-blocks (or a wait that ran out): zeros
    for (int i = threadIdx.x; i < NT * kSmallRows; i += kSmallThreads) part[i] = 0u;
  }
  tc_fence_before();
  if (g.split > 1) cluster_sync(); else __syncthreads();

  // A share of the outputs: unit e is 4 consecutive weight rows of a token.  All
  // ranks' parts of a unit are loaded before they are added up (one after the
  // other, each load from another SM's memory would cost its full latency).
  constexpr int PER = EPI == kGated ? 64 : kSmallRows, UNITS = PER / 4;
  const int64_t t0 = int64_t(ttile) * NT;
  const int ntok = static_cast<int>(min(int64_t(NT), g.T - t0));
  const uint32_t mine = smem_u32(part);
  auto total = [&](int index, float (&sum)[4]) {  // sums over the ranks, in rank order
    uint4 v[kMaxSplit];
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r)
      if (r < g.split) v[r] = ld_cluster_v4(map_to_rank(mine + index * 4, r));
    if constexpr (KIND == kI8Kind) {
      int a[4] = {0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < g.split) {
          a[0] += int(v[r].x); a[1] += int(v[r].y); a[2] += int(v[r].z); a[3] += int(v[r].w);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = static_cast<float>(a[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < g.split) {
          sum[0] += __uint_as_float(v[r].x); sum[1] += __uint_as_float(v[r].y);
          sum[2] += __uint_as_float(v[r].z); sum[3] += __uint_as_float(v[r].w);
        }
    }
  };
  for (int e = rank * kSmallThreads + threadIdx.x; e < ntok * UNITS; e += g.split * kSmallThreads) {
    const int tok = e / UNITS, r = e % UNITS * 4;
    const int64_t col = int64_t(wtile) * PER + r, row = t0 + tok;
    if (col >= g.N) continue;
    const int64_t at = row * g.N + col;
    float y[4], z[4];
    total(tok * kSmallRows + r, y);
    if constexpr (EPI == kScaled) {
      const float sa = g.a_scale[row];
      // rows of any length: element by element
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (col + i >= g.N) break;
        const float v = fmaf(y[i] * sa, g.b_scale[col + i], g.bias != nullptr ? g.bias[col + i] : 0.f);
        if (g.type == kF32)
          static_cast<float*>(g.out)[at + i] = v;
        else
          static_cast<uint16_t*>(g.out)[at + i] = pack1(v, g.type);
      }
    } else {  // N is a multiple of 8
      uint8_t* sv = nullptr;
      if constexpr (EPI != kPlain)
        if (g.saved != nullptr) sv = g.saved + saved_block(row, col, g.N) + saved_word(row, col);
      if constexpr (EPI == kGated) {
        total(tok * kSmallRows + 64 + r, z);
        if (sv != nullptr) {
          uint32_t w[4], l[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = __float_as_uint(y[i]);
            l[i] = __float_as_uint(z[i]);
          }
          *reinterpret_cast<uint2*>(sv) = make_uint2((w[0] >> 16) | (w[1] & 0xFFFF0000u), (w[2] >> 16) | (w[3] & 0xFFFF0000u));
          *reinterpret_cast<uint2*>(sv + kSavedPlane) =
              make_uint2((l[0] >> 16) | (l[1] & 0xFFFF0000u), (l[2] >> 16) | (l[3] & 0xFFFF0000u));
          *reinterpret_cast<uint2*>(sv + 2 * kSavedPlane) = make_uint2(saved_low(w[0], l[0], w[1], l[1]), saved_low(w[2], l[2], w[3], l[3]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = silu(y[i]) * z[i];
      } else if constexpr (EPI == kPlain) {
        if (g.residual != nullptr) {
          const uint2 q = *reinterpret_cast<const uint2*>(g.residual + at);
          y[0] += unpack_lo(q.x, g.type); y[1] += unpack_hi(q.x, g.type);
          y[2] += unpack_lo(q.y, g.type); y[3] += unpack_hi(q.y, g.type);
        }
      } else {
        const uint2 gh = *reinterpret_cast<const uint2*>(sv), uh = *reinterpret_cast<const uint2*>(sv + kSavedPlane),
                    lo = *reinterpret_cast<const uint2*>(sv + 2 * kSavedPlane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float gg, uu;
          saved_get((&gh.x)[i / 2], (&uh.x)[i / 2], (&lo.x)[i / 2], i % 2, gg, uu);
          dgate(y[i], gg, uu, y[i], z[i]);
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out2) + at) =
            make_uint2(pack2(z[0], z[1], g.type), pack2(z[2], z[3], g.type));
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + at) =
          make_uint2(pack2(y[0], y[1], g.type), pack2(y[2], y[3], g.type));
    }
  }
  // a peer may still read this CTA's partial sums
  __syncwarp();
  if (g.split > 1) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

}  // namespace dense
}  // namespace moe
