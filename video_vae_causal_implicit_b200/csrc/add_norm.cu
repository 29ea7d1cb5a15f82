// add_norm.cu -- the residual's addition, RMS norm (+ SiLU) and an output in
// 16 or 8 bits, one pass over HBM (cc3d_add_rms_norm).
//
//   h = bf16(x + r);  a = h * sqrt(c) / max(sqrt(sum h^2 + c eps), 1e-12) * gamma (+ beta)
//   a = SiLU(a) where asked;  y = bf16(a);
//   q = E4M3(a / s), s = max|a| / 448 of the row, or a given s.
//
// Bound: HBM.  A row is read once and stays in registers as bf16 between the
// sum of squares, the row's largest magnitude and the stores, so the bytes
// moved are the inputs and outputs alone: 32760 rows of 4096 channels with a
// residual 155 us (6.1 TB/s, 93 % of a copy's rate), 7800 rows of 384 4.8 us
// and five rows of 2048 2.4 us, where a launch and its latencies count.  (With
// SiLU the exponential and the division bound: 32760 x 4096 to 16 bits 121 us
// where the bytes want 82.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ops.h"
#include "ptx.cuh"

namespace cc3d {

namespace {

constexpr float kE4m3Max = 448.f;
// The smallest row scale: its reciprocal is finite, so a row of tiny values
// cannot turn into infinities.
constexpr float kMinScale = 1e-36f;

// TPR threads share a row (a part of a warp, a warp, or a whole CTA), each
// holding CPT chunks of 8 channels: chunk sub + k * TPR.
template <int TPR, int CPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) add_norm_kernel(const AddNormArgs p) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  constexpr int kRows = kThreads / TPR;  // rows per CTA pass
  constexpr int kWarps = TPR / 32;       // (TPR > 32) warps per row
  __shared__ float red[2][kWarps > 1 ? kWarps : 1];
  const int sub = threadIdx.x % TPR;
  const int groups = p.c / 8;
  const float fc = static_cast<float>(p.c), root_c = sqrtf(fc);
  griddep_launch_dependents();
  griddep_wait();
  for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < p.rows;
       r0 += static_cast<long long>(gridDim.x) * kRows) {
    const long long row = r0 + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const long long base = row * groups;  // in chunks
    uint4 raw[CPT];
    uint4 res[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const int g = sub + k * TPR;
      raw[k] = res[k] = make_uint4(0, 0, 0, 0);
      if (live && g < groups) {
        raw[k] = __ldcs(reinterpret_cast<const uint4 *>(p.x) + base + g);
        if (p.residual) res[k] = __ldcs(reinterpret_cast<const uint4 *>(p.residual) + base + g);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      uint32_t *w = reinterpret_cast<uint32_t *>(&raw[k]);
      const uint32_t *wr = reinterpret_cast<const uint32_t *>(&res[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xffff0000u);
        if (p.residual) {
          // the stream is held in bf16: the norm reads what the next layer adds to
          w[e] = pack_bf16x2(lo + __uint_as_float(wr[e] << 16),
                             hi + __uint_as_float(wr[e] & 0xffff0000u));
          lo = __uint_as_float(w[e] << 16);
          hi = __uint_as_float(w[e] & 0xffff0000u);
        }
        ss = fmaf(lo, lo, fmaf(hi, hi, ss));
      }
      const int g = sub + k * TPR;
      if (p.h && live && g < groups) reinterpret_cast<uint4 *>(p.h)[base + g] = raw[k];
    }
    // fixed-order reductions: the result does not depend on scheduling
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if constexpr (TPR > 32) {
      if (threadIdx.x % 32 == 0) red[0][threadIdx.x / 32] = ss;
      __syncthreads();
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) ss += red[0][i];
    }
    // (not fmaxf, which would put 1e-12 in the place of a NaN and leave the
    // row's other elements finite)
    const float norm = sqrtf(fmaf(fc, p.eps, ss));
    const float inv = root_c / (norm < 1e-12f ? 1e-12f : norm);
    float a[CPT][8];
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const int g = sub + k * TPR;
      const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[k][e] = 0.f;
      if (g < groups) {
        const float4 g0 = reinterpret_cast<const float4 *>(p.gamma)[2 * g];
        const float4 g1 = reinterpret_cast<const float4 *>(p.gamma)[2 * g + 1];
        const float gm[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
          a[k][e] = v * inv * gm[e];
        }
        if (p.beta) {
          const float4 b0 = reinterpret_cast<const float4 *>(p.beta)[2 * g];
          const float4 b1 = reinterpret_cast<const float4 *>(p.beta)[2 * g + 1];
          const float bt[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) a[k][e] += bt[e];
        }
        if (p.silu) {
          // (0 from a = -87.3 down, where the divisor is out of the fast
          // division's range: the value is under 1e-36.  A form that keeps
          // those, as the product's, took 5 to 9 % longer.)
#pragma unroll
          for (int e = 0; e < 8; ++e) a[k][e] = __fdividef(a[k][e], 1.f + __expf(-a[k][e]));
        }
        if (p.y && live) {
          uint4 o;
          o.x = pack_bf16x2(a[k][0], a[k][1]);
          o.y = pack_bf16x2(a[k][2], a[k][3]);
          o.z = pack_bf16x2(a[k][4], a[k][5]);
          o.w = pack_bf16x2(a[k][6], a[k][7]);
          __stcs(reinterpret_cast<uint4 *>(p.y) + base + g, o);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(a[k][e]));
      }
    }
    if (!p.q) {
      if constexpr (TPR > 32) __syncthreads();  // red is rewritten by the next pass
      continue;
    }
    float mul;
    if (p.scales) {
#pragma unroll
      for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if constexpr (TPR > 32) {
        if (threadIdx.x % 32 == 0) red[1][threadIdx.x / 32] = top;
        __syncthreads();
        top = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, red[1][i]);
      }
      const float scale = top > 0.f ? fmaxf(top / kE4m3Max, kMinScale) : 1.f;
      if (sub == 0 && live) p.scales[row] = scale;
      mul = 1.f / scale;
    } else {
      if constexpr (TPR > 32) __syncthreads();
      mul = 1.f / p.q_scale;
    }
    // one reciprocal and a product an element in place of a division: the
    // quotient moves by at most 2 ulp of fp32, a code only next to a tie
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const int g = sub + k * TPR;
      if (live && g < groups) {
        uint2 o;
        o.x = pack_e4m3x2(a[k][0] * mul, a[k][1] * mul) |
              static_cast<uint32_t>(pack_e4m3x2(a[k][2] * mul, a[k][3] * mul)) << 16;
        o.y = pack_e4m3x2(a[k][4] * mul, a[k][5] * mul) |
              static_cast<uint32_t>(pack_e4m3x2(a[k][6] * mul, a[k][7] * mul)) << 16;
        __stcs(reinterpret_cast<uint2 *>(p.q) + base + g, o);
      }
    }
  }
}

template <int TPR, int CPT>
cudaError_t launch_one(const AddNormArgs &a, int sm_count, cudaStream_t stream) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  constexpr int kRows = kThreads / TPR;
  const long long need = (a.rows + kRows - 1) / kRows;
  const long long most = static_cast<long long>(sm_count) * (2048 / kThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(need < most ? need : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, add_norm_kernel<TPR, CPT>, a);
  count_launch();
  return e;
}

template <int TPR>
cudaError_t launch_cpt(const AddNormArgs &a, int sm_count, cudaStream_t stream) {
  switch ((a.c / 8 + TPR - 1) / TPR) {
    case 1: return launch_one<TPR, 1>(a, sm_count, stream);
    case 2: return launch_one<TPR, 2>(a, sm_count, stream);
    case 3: return launch_one<TPR, 3>(a, sm_count, stream);
    case 4: return launch_one<TPR, 4>(a, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_add_rms_norm(const AddNormArgs &a, int sm_count, cudaStream_t stream) {
  const int groups = a.c / 8;
  if (groups <= 64) return launch_cpt<16>(a, sm_count, stream);
  if (groups <= 128) return launch_cpt<32>(a, sm_count, stream);
  if (groups <= 512) return launch_cpt<128>(a, sm_count, stream);
  if (groups <= 1024) return launch_cpt<256>(a, sm_count, stream);
  return launch_cpt<512>(a, sm_count, stream);
}

}  // namespace cc3d
