// norm.cuh -- residual addition and root-mean-square norm, with a 16-bit or an
// 8-bit (int8, FP8 E4M3) output, and its backward pass.
//
//   s[t] = round(x[t] + residual[t])                    the new residual stream
//   y[t][c] = s[t][c] * rstd[t] * w[c],  rstd[t] = 1 / sqrt(mean_c s[t][c]^2 + eps)
// The norm is taken of the rounded stream, the one that is stored: the
// backward pass and every later layer see the same values.
//   8-bit: scale = max(amax |y| / top, 2^-126) over a token's row or over each
//   128 columns of it, code = round(y / scale), top = 127 (int8) or 448 (E4M3).
//   backward, with n = s * rstd and dn = dy * w:
//   dx[t] = rstd (dn - n mean_c(dn n)) + dstream[t],   dw = sum_t dy n
//
// Rows whose sum of squares leaves fp32's range are summed again, scaled by a
// power of two (a row of zeros with eps = 0 gives the formula's 0 / 0, NaN).
//
// HBM-bound: a row is read once, kept in registers (fp32 arithmetic, every sum
// in fp32), and written once.
#pragma once
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"

namespace moe {
namespace norm {

constexpr int kMaxH = 32768;       // a row lives in one block's registers
constexpr int kGroup = 128;        // columns per scale in the grouped form

enum Format { kSame = 0, kInt8 = 1, kE4m3 = 2 };

// VEC consecutive 16-bit elements as they lie in memory, in whole registers:
// 8 (16 bytes) or 1.  (An array of 16-bit members would take a register each.)
template <typename E, int VEC>
struct alignas(2 * VEC) Pack {
  uint32_t w[VEC / 2];
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (std::is_same<E, __nv_bfloat16>::value) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      if constexpr (std::is_same<E, __nv_bfloat16>::value) {
        w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      } else {
        const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
  }
};
template <typename E>
struct alignas(2) Pack<E, 1> {
  uint16_t w;
  __device__ __forceinline__ void get(float (&f)[1]) const {
    if constexpr (std::is_same<E, __nv_bfloat16>::value)
      f[0] = __uint_as_float(uint32_t(w) << 16);
    else
      f[0] = __half2float(__ushort_as_half(w));
  }
  __device__ __forceinline__ void set(const float (&f)[1]) {
    if constexpr (std::is_same<E, __nv_bfloat16>::value)
      w = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    else
      w = __half_as_ushort(__float2half_rn(f[0]));
  }
};
// VEC 8-bit codes.
template <int VEC>
struct alignas(VEC) Codes {
  uint8_t e[VEC];
};

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool MAX>
__device__ __forceinline__ float combine(float a, float b) {
  return MAX ? max_nan(a, b) : a + b;
}

// Sum (or maximum, of values that are not negative) of v over the block, in a
// fixed order, returned to every thread.  `red` holds one word per warp; two
// calls in a row need different ones.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = combine<MAX>(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = combine<MAX>(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Two sums at once: the lower 16 lanes add up a's, the upper ones b's.
__device__ __forceinline__ void block_sum2(float& a, float& b, float (&red)[2][32]) {
  const int lane = threadIdx.x & 31, l = lane & 15, which = lane >> 4;
  float v = (which ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, which ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (blockDim.x > 32) {
    const int warps = blockDim.x >> 5;
    if (l == 0) red[which][threadIdx.x >> 5] = v;
    __syncthreads();
    v = l < warps ? red[which][l] : 0.f;
    if (l + 16 < warps) v += red[which][l + 16];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  a = __shfl_sync(0xFFFFFFFFu, v, 0);
  b = __shfl_sync(0xFFFFFFFFu, v, 16);
}

__device__ __forceinline__ float scale_of(float amax, float top) {
  return max_nan(__fdiv_rn(amax, top), 1.17549435e-38f);
}

// The codes of values that share a scale: round(y / scale).  The quotient is
// that by the reciprocal, corrected once by its exact remainder, which makes it
// the correctly rounded one (Markstein 1990).  Without it values beside a tie
// (half a group's largest, for one) took the other code.  int8 at T = 8189,
// H = 4096: 43.9 us, 42.0 without the correction, 49.1 with a division for each
// value.
template <int FMT>
struct Coder {
  float scale, inv;  // an infinite scale, whose reciprocal is 0, is kept as 0: finite values give 0
  __device__ __forceinline__ explicit Coder(float s) : scale(s == INFINITY ? 0.f : s), inv(1.f / s) {}
  __device__ __forceinline__ uint8_t operator()(float y) const {
    float z = y * inv;
    z = fmaf(fmaf(-z, scale, y), inv, z);
    if constexpr (FMT == kInt8) {
      const int q = __float2int_rn(z);
      return static_cast<uint8_t>(max(-127, min(127, q)));
    } else {
      return __nv_cvt_float_to_fp8(z, __NV_SATFINITE, __NV_E4M3);
    }
  }
};

template <typename E, int VEC>
__device__ __forceinline__ void load_weight(const E* w, int p, float (&f)[VEC]) {
  if (w != nullptr) {
    reinterpret_cast<const Pack<E, VEC>*>(w)[p].get(f);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = 1.f;
  }
}

// Whether a row's sum of squares left the range in which fp32 holds it well:
// then the row is scaled by a power of two (row_scale) and summed again.  A sum
// of 0 is that of zeros or of squares that underflowed; these are below 2^-149
// each, so beside an eps of 1e-30 they are nothing, and the row (a padded one, as
// a rule) need not be scaled.
__device__ __forceinline__ bool out_of_range(float ss, float eps) {
  return !(ss >= 1e-30f && ss <= 1e38f) && !(ss == 0.f && eps >= 1e-30f);
}
// The power of two that brings the larger of amax and sqrt(eps) to [1, 2); 1
// where that is zero, infinite or NaN.
__device__ __forceinline__ float row_scale(float amax, float eps) {
  const float c = max_nan(amax, sqrtf(eps));
  if (!(c > 0.f && c < INFINITY)) return 1.f;
  return ldexpf(1.f, -max(-126, min(127, ilogbf(c))));
}

// One row per block; a thread holds NV packs of VEC elements, pack i at column
// (i * blockDim.x + threadIdx.x) * VEC.  group: 0 (a scale per row) or kGroup.
template <typename E, int VEC, int NV, int FMT, int MAXT>
__global__ void __launch_bounds__(MAXT)
    add_rmsnorm_kernel(const E* x, const E* res, const E* __restrict__ w, float eps, int H,
                       int group, E* s_out, void* out, float* __restrict__ scales) {
  __shared__ float red[3][32];
  __shared__ unsigned gmax[VEC == 1 ? kMaxH / kGroup : 1];
  using P = Pack<E, VEC>;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x, base = row * H;
  const int nvec = H / VEC;
  float v[NV][VEC];
  float ss = 0.f;
  // every load of the row before its first store (s_out or out may be x or res)
  P xa[NV], ra[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = i * blockDim.x + threadIdx.x;
    if (p < nvec) {
      xa[i] = *reinterpret_cast<const P*>(x + base + static_cast<int64_t>(p) * VEC);
      if (res != nullptr) ra[i] = *reinterpret_cast<const P*>(res + base + static_cast<int64_t>(p) * VEC);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = i * blockDim.x + threadIdx.x;
    if (p < nvec) {
      xa[i].get(v[i]);
      if (res != nullptr) {
        float r[VEC];
        ra[i].get(r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] += r[j];
        xa[i].set(v[i]);
        *reinterpret_cast<P*>(s_out + base + static_cast<int64_t>(p) * VEC) = xa[i];
        xa[i].get(v[i]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += v[i][j] * v[i][j];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
    }
  }
  if (FMT != kSame && VEC == 1 && group) {
    for (int g = threadIdx.x; g < (H + kGroup - 1) / kGroup; g += blockDim.x) gmax[g] = 0u;
  }
  ss = block_reduce<false>(ss, red[0]);
  float amax = 0.f;
  if (out_of_range(ss, eps)) {  // the whole block
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) amax = max_nan(amax, fabsf(v[i][j]));
    const float mult = row_scale(block_reduce<true>(amax, red[1]), eps);
    if (mult != 1.f) {
      eps = eps * mult * mult;
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] *= mult;
          ss += v[i][j] * v[i][j];
        }
      ss = block_reduce<false>(ss, red[2]);
    }
    __syncthreads();  // red[1] is used again below
    amax = 0.f;
  }
  const float rstd = rsqrtf(ss / static_cast<float>(H) + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = i * blockDim.x + threadIdx.x;
    if (p < nvec) {
      float wf[VEC];
      load_weight<E, VEC>(w, p, wf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] = v[i][j] * rstd * wf[j];
        amax = max_nan(amax, fabsf(v[i][j]));
      }
    }
  }
  if constexpr (FMT == kSame) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < nvec) {
        P o;
        o.set(v[i]);
        *reinterpret_cast<P*>(static_cast<E*>(out) + base + static_cast<int64_t>(p) * VEC) = o;
      }
    }
  } else {
    const float top = FMT == kInt8 ? 127.f : 448.f;
    float scale = 0.f;
    if (!group) {
      scale = scale_of(block_reduce<true>(amax, red[1]), top);
      if (threadIdx.x == 0) scales[row] = scale;
    } else if constexpr (VEC == 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int p = i * blockDim.x + threadIdx.x;
        // non-negative floats (and NaN above them) order like their bits
        if (p < nvec) atomicMax(&gmax[p / kGroup], __float_as_uint(fabsf(v[i][0])));
      }
      __syncthreads();
    }
    const int ngroups = (H + kGroup - 1) / kGroup;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (group) {
        if constexpr (VEC == 1) {
          if (p < nvec) scale = scale_of(__uint_as_float(gmax[p / kGroup]), top);
        } else {  // 16 consecutive lanes hold a group's 128 columns
          float m = 0.f;
#pragma unroll
          for (int j = 0; j < VEC; ++j) m = max_nan(m, fabsf(v[i][j]));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          scale = scale_of(m, top);
        }
        if (p < nvec && (p * VEC) % kGroup == 0) scales[row * ngroups + p * VEC / kGroup] = scale;
      }
      if (p < nvec) {
        const Coder<FMT> code(scale);
        Codes<VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.e[j] = code(v[i][j]);
        *reinterpret_cast<Codes<VEC>*>(static_cast<uint8_t*>(out) + base +
                                               static_cast<int64_t>(p) * VEC) = o;
      }
    }
  }
}

// Blocks of the backward kernel that an SM runs at once, by the registers of a
// thread's packs.
__host__ __device__ constexpr int backward_blocks(int vec, int nv, int maxt) {
  return maxt > 256 || vec * nv > 16 ? 1 : vec * nv > 8 ? 2 : 3;
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; the next row's loads are under
// way while a row is summed and written (unless a block of 1024 threads has no
// registers for it), since a block waits for its slowest warp in every row.
// dw partial sums of a block's rows stay in registers and go to
// parts[blockIdx.x].
// EPS0: the kernel for eps = 0.  Only there can 1 / rms pass fp32's range (rows
// of subnormal values) where n and dx do not, so a scaled row's two factors are
// applied one after the other.  In every call, that took 2% longer at H = 4096
// and 5% at 16384.
template <typename E, int VEC, int NV, int MAXT, bool EPS0>
__global__ void __launch_bounds__(MAXT, backward_blocks(VEC, NV, MAXT))
    rmsnorm_backward_kernel(const E* __restrict__ dy, const E* __restrict__ s,
                            const E* __restrict__ w, float eps, int64_t T, int H,
                            const E* __restrict__ dstream, E* __restrict__ dx,
                            float* __restrict__ parts) {
  __shared__ float red[3][2][32];
  using P = Pack<E, VEC>;
  griddep_wait();
  griddep_launch_dependents();
  const int nvec = H / VEC;
  float dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = 0.f;
  constexpr bool AHEAD = MAXT <= 256;
  P sn[NV], dn[NV], tn[NV];  // the next row of s, dy, dstream
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < nvec) {
        const int64_t at = row * H + static_cast<int64_t>(p) * VEC;
        sn[i] = *reinterpret_cast<const P*>(s + at);
        dn[i] = *reinterpret_cast<const P*>(dy + at);
        if (AHEAD && dstream != nullptr) tn[i] = *reinterpret_cast<const P*>(dstream + at);
      }
    }
  };
  if (AHEAD && blockIdx.x < T) fetch(blockIdx.x);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, flip ^= 1) {
    const int64_t base = row * H;
    P sv[NV], dv[NV], tv[NV];
    if (!AHEAD) fetch(row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      sv[i] = sn[i];
      dv[i] = dn[i];
      tv[i] = tn[i];
    }
    if (AHEAD && row + gridDim.x < T) fetch(row + gridDim.x);
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < nvec) {
        float a[VEC], d[VEC], wf[VEC];
        sv[i].get(a);
        dv[i].get(d);
        load_weight<E, VEC>(w, p, wf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          ss += a[j] * a[j];
          sd += a[j] * (d[j] * wf[j]);
        }
      }
    }
    // the two sums use other words in every second row, so that a fast warp's
    // next row does not overwrite what a slow one still reads
    block_sum2(ss, sd, red[flip]);
    float mult = 1.f;
    if (out_of_range(ss, eps)) {  // the whole block: as in the forward pass
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x) < nvec) {
          float a[VEC];
          sv[i].get(a);
#pragma unroll
          for (int j = 0; j < VEC; ++j) amax = max_nan(amax, fabsf(a[j]));
        }
      mult = row_scale(block_reduce<true>(amax, red[2][0]), eps);
      ss = sd = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int p = i * blockDim.x + threadIdx.x;
        if (p < nvec) {
          float a[VEC], d[VEC], wf[VEC];
          sv[i].get(a);
          dv[i].get(d);
          load_weight<E, VEC>(w, p, wf);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            a[j] *= mult;
            ss += a[j] * a[j];
            sd += a[j] * (d[j] * wf[j]);
          }
        }
      }
      __syncthreads();  // every thread has read the first sums
      block_sum2(ss, sd, red[flip]);
    }
    const float rstd = rsqrtf(ss / static_cast<float>(H) + eps * mult * mult);  // of s * mult
    const float m = sd * rstd / static_cast<float>(H);                          // mean(dn n)
    const float scale = rstd * mult;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < nvec) {
        if (!AHEAD && dstream != nullptr)
          tv[i] = *reinterpret_cast<const P*>(dstream + base + static_cast<int64_t>(p) * VEC);
        float a[VEC], d[VEC], wf[VEC], t[VEC];
        sv[i].get(a);
        dv[i].get(d);
        load_weight<E, VEC>(w, p, wf);
        if (dstream != nullptr) {
          tv[i].get(t);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) t[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          if constexpr (EPS0) {
            const float n = a[j] * mult * rstd;
            dw[i][j] += d[j] * n;
            t[j] += mult * (rstd * (d[j] * wf[j] - n * m));
          } else {
            const float n = a[j] * scale;
            dw[i][j] += d[j] * n;
            t[j] += scale * (d[j] * wf[j] - n * m);
          }
        }
        P o;
        o.set(t);
        *reinterpret_cast<P*>(dx + base + static_cast<int64_t>(p) * VEC) = o;
      }
    }
  }
  if (parts != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * blockDim.x + threadIdx.x;
      if (p < nvec) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          parts[static_cast<int64_t>(blockIdx.x) * H + static_cast<int64_t>(p) * VEC + j] = dw[i][j];
      }
    }
  }
}

// dw[c] = sum of parts[0..n)[c], in a fixed order: 32 columns per block, each
// of 32 warps adds every 32nd row, then the warps' sums are added.
__global__ void __launch_bounds__(1024)
    rmsnorm_dw_kernel(const float* __restrict__ parts, int n, int H, float* __restrict__ dw) {
  __shared__ float sum[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int r = warp; r < n; r += 32) a += parts[static_cast<int64_t>(r) * H + c];
  }
  sum[warp][lane] = a;
  __syncthreads();
  a = sum[lane][warp];  // column `warp` of the block, row sums across the lanes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  if (lane == 0 && blockIdx.x * 32 + warp < H) dw[blockIdx.x * 32 + warp] = a;
}

}  // namespace norm
}  // namespace moe
