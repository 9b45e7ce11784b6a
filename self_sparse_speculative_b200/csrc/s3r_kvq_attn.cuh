// Pieces shared by the quantised attention kernels: parameters, output
// addressing, empty outputs and the log-sum-exp merge of split partials.
#pragma once

#include <cuda_bf16.h>

#include <cmath>

#include "s3r_attn_common.cuh"
#include "s3r_device.cuh"
#include "s3r_kvq.cuh"

namespace s3r {

// Whether sequence b's context length is usable for the call's R rows.
__device__ __forceinline__ bool kvq_bad_context(const KvqAttnParams& p, int L) {
  return L < p.R || L < 1 || L > p.max_pages * p.P;
}

// Packed row i of unit (b, h) is query head h*G + i % G of row r0 + i / G; its
// row in the [S, R, Hq] layout.
__device__ __forceinline__ size_t kvq_out_row(const KvqAttnParams& p, int b, int h, int i) {
  const int r = p.r0 + i / p.G, g = i - (i / p.G) * p.G;
  return (size_t)(b * p.R + r) * p.Hq + (size_t)h * p.G + g;
}

// Outputs of a unit with nothing to attend over: zeros and lse = -inf.
template <typename OutT>
__device__ void kvq_write_empty(const KvqAttnParams& p, int b, int h, int tid0, int nthreads) {
  const int D4 = p.D / 4;
  for (int idx = tid0; idx < p.rows * D4; idx += nthreads) {
    const int i = idx / D4, d4 = idx - (idx / D4) * D4;
    const size_t orow = kvq_out_row(p, b, h, i);
    store_out4<OutT>(static_cast<OutT*>(p.out) + orow * p.D + d4 * 4, 0.f, 0.f, 0.f, 0.f);
    if (d4 == 0 && p.lse) p.lse[orow] = -INFINITY;
  }
}

// Merge partial states slots [slot0, slot0 + nparts) of unit (b, h): M = max
// m_s, L = sum l_s 2^(m_s - M), out = sum O_s 2^(m_s - M) / L, lse = (M + log2 L) ln 2
// (m in log2 units of the scaled score). A part with l = 0 saw nothing; a NaN
// l reaches the output.
template <typename OutT>
__device__ void kvq_combine(const KvqAttnParams& p, int b, int h, int slot0, int nparts, int nthreads) {
  const int D4 = p.D / 4;
  for (int idx = threadIdx.x; idx < p.rows * D4; idx += nthreads) {
    const int i = idx / D4, d4 = idx - (idx / D4) * D4;
    float M = -INFINITY;
    for (int s = 0; s < nparts; ++s) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)(slot0 + s) * p.rows + i);
      if (ml.y != 0.f) M = fmaxf(M, ml.x);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float Ls = 0.f;
    for (int s = 0; s < nparts; ++s) {
      const size_t pi = (size_t)(slot0 + s) * p.rows + i;
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + pi);
      if (ml.y == 0.f) continue;
      const float w = exp2f(ml.x - M);
      Ls += ml.y * w;
      const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part_o + pi * p.D) + d4);
      acc.x += w * o.x; acc.y += w * o.y; acc.z += w * o.z; acc.w += w * o.w;
    }
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
    const size_t orow = kvq_out_row(p, b, h, i);
    store_out4<OutT>(static_cast<OutT*>(p.out) + orow * p.D + d4 * 4, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (d4 == 0 && p.lse) p.lse[orow] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
  }
}

}  // namespace s3r
