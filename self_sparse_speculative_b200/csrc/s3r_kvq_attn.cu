// Attention over the quantised paged KV cache (layout and arithmetic of a held
// row: s3r_kvq.cuh): the dispatch, and the float32 kernel on CUDA cores (bf16
// goes to the tensor-core kernel, s3r_kvq_attn_tok.cuh).
//
//   score[i, t] = scale (s_k[t] q_i . n_k[t] + z_k[t] sum q_i)      (= scale q_i . k^_t)
//   out[i, d]   = sum_t p[i, t] (s_v[t] n_v[t, d] + z_v[t]) / sum_t p[i, t]
//
// with p the softmax over the positions that row i sees: those at or before
// its own (row r of R sits at L - R + r), of every page or of the listed ones.
//
// kvq_attn_f32_kernel: split-KV. A CTA owns one (sequence, KV head, split) and
// walks its pages in 16-token sub-tiles, unpacked into float32 rows in shared
// memory; running maximum and sum per row, partial states merged by
// log-sum-exp in the last CTA of the unit to finish (ticket, no waiting). A
// row that sees nothing gives zeros and lse = -inf.
#include <cuda_bf16.h>

#include <cmath>

#include "s3r_attn_common.cuh"
#include "s3r_device.cuh"
#include "s3r_internal.h"
#include "s3r_kvq.cuh"
#include "s3r_kvq_attn.cuh"

namespace s3r {
namespace {

constexpr int kF32Threads = 128;
constexpr int kF32Tok = 16;

template <int D, int P, int BITS>
__global__ void __launch_bounds__(kF32Threads) kvq_attn_f32_kernel(const KvqAttnParams p) {
  constexpr KvqLayout Y = kvq_layout(D, P, BITS);
  constexpr int kKStride = D + 4;                        // 16 tokens of one channel on 8 banks apart
  constexpr int kPer = 32 / BITS;                        // numbers per word
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(16) float f32_smem[];
  __shared__ int s_ticket;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x;
  const int L = p.context_lens[b];
  if (kvq_bad_context(p, L)) {
    if (split == 0) {
      if (tid == 0) flag_status(p.status, S3R_DEV_BAD_CONTEXT_LEN);
      kvq_write_empty<float>(p, b, h, tid, kF32Threads);
    }
    return;
  }
  const int n_b = (L + P - 1) / P;
  const int total_pages = p.page_list ? p.budget : n_b;
  const int nsplit_u = (total_pages + p.chunk_pages - 1) / p.chunk_pages;
  if (split >= nsplit_u) return;
  const int pg0 = split * p.chunk_pages, npg = min(p.chunk_pages, total_pages - pg0);
  const int rows = p.rows;
  float* sQ = f32_smem;                       // [rows, D]
  float* sO = sQ + rows * D;                  // [rows, D]
  float* sK = sO + rows * D;                  // [16, D + 4]
  float* sV = sK + kF32Tok * kKStride;        // [16, D]
  float* sS = sV + kF32Tok * D;               // [rows, 16]
  float* sM = sS + rows * kF32Tok;            // [rows]
  float* sL = sM + rows;                      // [rows]
  float* sA = sL + rows;                      // [rows]
  const float* q = static_cast<const float*>(p.q);
  for (int idx = tid; idx < rows * D; idx += kF32Threads) {
    const int i = idx / D, d = idx - (idx / D) * D;
    // an infinite channel as NaN: scores of -inf alone would look like hidden ones
    const float x = q[kvq_out_row(p, b, h, i) * D + d];
    sQ[idx] = fabsf(x) < INFINITY ? x : __int_as_float(0x7fc00000);
    sO[idx] = 0.f;
  }
  for (int i = tid; i < rows; i += kF32Threads) {
    sM[i] = -INFINITY;
    sL[i] = 0.f;
  }
  __syncthreads();
  for (int k = 0; k < npg; ++k) {
    const int lp = p.page_list ? p.page_list[((size_t)b * p.Hkv + h) * p.budget + pg0 + k] : pg0 + k;
    if (lp == -1) continue;                              // an unused list entry
    const int phys = lp >= 0 && lp < n_b ? p.block_table[(size_t)b * p.max_pages + lp] : -1;
    if (phys < 0 || phys >= p.num_pages_total) {
      if (tid == 0) flag_status(p.status, S3R_DEV_BAD_PAGE_ID);
      continue;
    }
    const uint8_t* pg = p.pages + ((size_t)phys * p.Hkv + h) * Y.page_bytes;
    const int valid = min(P, L - lp * P);
    for (int t0 = 0; t0 < valid; t0 += kF32Tok) {
      const int ntok = min(kF32Tok, valid - t0);
      for (int idx = tid; idx < kF32Tok * D / kPer; idx += kF32Threads) {
        const int t = idx % kF32Tok, w = idx / kF32Tok;  // token of the sub-tile, word of its row
        const uint32_t par = *reinterpret_cast<const uint32_t*>(pg + Y.off_kp + (t0 + t) * 4);
        const uint32_t c = *reinterpret_cast<const uint32_t*>(pg + ((w >> 2) * P + t0 + t) * 16 + (w & 3) * 4);
        const float s = __uint_as_float(par << 16), z = __uint_as_float(par & 0xffff0000u);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          sK[t * kKStride + w * kPer + i] = fmaf(s, (float)((c >> (BITS * i)) & ((1u << BITS) - 1u)), z);
      }
      for (int idx = tid; idx < kF32Tok / kPer * D; idx += kF32Threads) {
        const int d = idx % D, t = (idx / D) * kPer;     // channel, first token of the word
        const int at = t0 + t;
        const uint32_t c = *reinterpret_cast<const uint32_t*>(pg + Y.off_v + ((at / Y.ut) * D + d) * Y.unit +
                                                              (at % Y.ut) * BITS / 8);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t par = *reinterpret_cast<const uint32_t*>(pg + Y.off_vp + (at + i) * 4);
          const float s = __uint_as_float(par << 16), z = __uint_as_float(par & 0xffff0000u);
          sV[(t + i) * D + d] = t + i < ntok ? fmaf(s, (float)((c >> (BITS * i)) & ((1u << BITS) - 1u)), z) : 0.f;
        }
      }
      __syncthreads();
      for (int idx = tid; idx < rows * kF32Tok; idx += kF32Threads) {
        const int i = idx / kF32Tok, t = idx - (idx / kF32Tok) * kF32Tok;
        const int pos = lp * P + t0 + t;
        float sc = -INFINITY;
        if (t < ntok && pos <= L - p.R + p.r0 + i / p.G) {
          const float4* a = reinterpret_cast<const float4*>(sQ + i * D);
          const float4* kk = reinterpret_cast<const float4*>(sK + t * kKStride);
          float acc = 0.f;
#pragma unroll 8
          for (int d = 0; d < D / 4; ++d) {
            const float4 x = a[d], y = kk[d];
            acc = fmaf(x.x, y.x, acc); acc = fmaf(x.y, y.y, acc);
            acc = fmaf(x.z, y.z, acc); acc = fmaf(x.w, y.w, acc);
          }
          sc = acc * p.scale_log2;
        }
        sS[idx] = sc;
      }
      __syncthreads();
      for (int i = tid; i < rows; i += kF32Threads) {
        float mx = -INFINITY;
        for (int t = 0; t < kF32Tok; ++t) mx = fmaxf(mx, sS[i * kF32Tok + t]);
        const float m_old = sM[i];
        const float m_new = fmaxf(m_old, mx);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m_old == -INFINITY ? 1.f : exp2f(m_old - m_use);
        float sum = 0.f;
        for (int t = 0; t < kF32Tok; ++t) {
          const float sc = sS[i * kF32Tok + t];
          // hidden tokens are marked -0: their values are left out below, whatever they are
          const float e = sc == -INFINITY ? -0.f : exp2f(sc - m_use);
          sS[i * kF32Tok + t] = e;
          sum += e;
        }
        sL[i] = sL[i] * alpha + sum;
        sM[i] = m_new;
        sA[i] = alpha;
      }
      __syncthreads();
      for (int idx = tid; idx < rows * D; idx += kF32Threads) {
        const int i = idx / D, d = idx - (idx / D) * D;
        float acc = sO[idx] * sA[i];
        for (int t = 0; t < kF32Tok; ++t) {
          const float e = sS[i * kF32Tok + t];
          if (__float_as_int(e) != (int)0x80000000) acc = fmaf(e, sV[t * D + d], acc);
        }
        sO[idx] = acc;
      }
      __syncthreads();
    }
  }
  const bool single = nsplit_u == 1;
  const int unit = b * p.Hkv + h;
  for (int idx = tid; idx < rows * D; idx += kF32Threads) {
    const int i = idx / D, d = idx - (idx / D) * D;
    if (single) {
      const float l = sL[i];
      static_cast<float*>(p.out)[kvq_out_row(p, b, h, i) * D + d] = l == 0.f ? 0.f : sO[idx] / l;
    } else {
      p.part_o[(((size_t)unit * p.nsplit + split) * rows + i) * D + d] = sO[idx];
    }
  }
  for (int i = tid; i < rows; i += kF32Threads) {
    const float l = sL[i], m = sM[i];
    if (single) {
      if (p.lse) p.lse[kvq_out_row(p, b, h, i)] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    } else {
      const size_t pi = ((size_t)unit * p.nsplit + split) * rows + i;
      p.part_ml[pi * 2] = m;
      p.part_ml[pi * 2 + 1] = l;
    }
  }
  if (!single) {
    __threadfence();
    __syncthreads();
    if (tid == 0) s_ticket = atomicAdd(p.tickets + unit, 1u);
    __syncthreads();
    if (s_ticket == nsplit_u - 1) {
      __threadfence();
      kvq_combine<float>(p, b, h, unit * p.nsplit, nsplit_u, kF32Threads);
      if (tid == 0) p.tickets[unit] = 0u;
    }
  }
}

template <int D, int P, int BITS>
cudaError_t launch_f32(const KvqAttnParams& p, cudaStream_t st) {
  const size_t smem = sizeof(float) * ((size_t)2 * p.rows * D + kF32Tok * (2 * D + 4) + (size_t)p.rows * kF32Tok + 3 * p.rows);
  cudaError_t e = cudaFuncSetAttribute(kvq_attn_f32_kernel<D, P, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kvq_attn_f32_kernel<D, P, BITS>, dim3(p.nsplit, p.Hkv, p.S), dim3(kF32Threads), smem, st, 1, p);
}
template <int D, int P>
cudaError_t launch_f32_bits(int bits, const KvqAttnParams& p, cudaStream_t st) {
  return bits == 4 ? launch_f32<D, P, 4>(p, st) : launch_f32<D, P, 8>(p, st);
}

}  // namespace

cudaError_t launch_kvq_attn(const s3r_paged_kvq& c, s3r_dtype dt, const KvqAttnParams& p, cudaStream_t st) {
  if (dt == S3R_F32) {
    if (c.head_dim == 64)
      return c.page_size == 16 ? launch_f32_bits<64, 16>(c.bits, p, st) : launch_f32_bits<64, 64>(c.bits, p, st);
    return c.page_size == 16 ? launch_f32_bits<128, 16>(c.bits, p, st) : launch_f32_bits<128, 64>(c.bits, p, st);
  }
  // more packed rows than one launch takes: equal shares of the rows, one launch each
  const int most = kKvqRows / p.G;
  const int launches = (p.R + most - 1) / most, per = (p.R + launches - 1) / launches;
  for (int r0 = 0; r0 < p.R; r0 += per) {
    KvqAttnParams q = p;
    q.r0 = r0;
    q.rows = p.G * (p.R - r0 < per ? p.R - r0 : per);
    const cudaError_t e = c.bits == 4 ? launch_kvq_attn_tok4(c.head_dim, q, st) : launch_kvq_attn_tok8(c.head_dim, q, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace s3r
