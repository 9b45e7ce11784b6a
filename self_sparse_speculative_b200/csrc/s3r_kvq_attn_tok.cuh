// Attention over the quantised paged KV cache on the tensor cores, bf16
// queries, up to 64 packed rows (G query heads x R rows) per (sequence, KV
// head). Layout and arithmetic of a held row: s3r_kvq.cuh.
//
// The held numbers themselves go through the tensor cores; scales and minima
// meet the results outside:
//   S^T[t, i] = sum_d n_k[t, d] q[i, d]
//   y         = scale log2 e (s_k[t] S^T + z_k[t] sum_d q[i, d]),    p = 2^(y - reference)
//   w[t, i]   = p s_v[t], rounded to w' (below)
//   O^T[d, i] = sum_t n_v[t, d] w'[t, i]
//   out       = (O^T - c sum_t w' + sum_t w (z_v[t] / s_v[t] + c)) / sum_t p,   c = (2^bits - 1) / 2
// The rounding of w only meets the centred numbers n - c; the rows' means are
// summed with the unrounded weight. The reference of a row bounds y + log2 s_v,
// so that w stays in the narrow type's range whatever the values' scales.
//
// A 4-bit number n in the low bits of a byte is, read as e4m3, exactly n 2^-9
// (subnormals and the first binade have one spacing): unpacking is one shift
// and two logic operations for eight numbers. A byte of an 8-bit cache is its
// two halves: for the keys side by side in the contraction, met by (q, 16 q);
// for the values two tiles that meet the same weights and accumulate apart.
// Queries and weights are two e4m3 terms each, x = hi + lo / 32, in separate
// columns: 8 significant bits down to 2^-12 of a row's largest weight, falling
// to none at 2^-21 of it (a bf16 query exactly, after a power-of-two scale per row,
// down to 2^-12 of the row's largest, and to 2^-18 of it absolutely), and the MMAs cost no more for it (with
// so few columns they are bound by reading the A operand). Every other
// token's numbers are complemented (2^bits - 1 - n) and its weights negated:
// the sums over tokens then stay near zero, where the accumulator's
// truncation would otherwise build up a bias over a long sequence.
//
// Both operands of numbers are the MMA's A operand (M = 128 tokens of S^T, M =
// 128 lanes of channels of O^T) and live in tensor memory: a thread unpacks
// one token's channels (one channel's tokens) from 16-byte shared-memory reads
// into registers and stores them to its TMEM lane, so the unpacked form never
// crosses shared memory. Q and w are the B operands in shared memory.
//
// Warps: 4 NSM softmax (thread = token; each warpgroup NR of the rows), 4 NDQ
// unpacking (NDQ = 2: keys and values apart; 1 with more than 24 rows, where
// the softmax takes two warpgroups), one producer (a bulk copy per (page,
// head) into an NS-stage ring of 128 tokens), one MMA issuer that polls its
// barriers and issues whichever product is ready. Work is split over CTAs as
// in the bf16 attention (s3r_attn_sched.cuh), units shared by several CTAs
// merge by log-sum-exp in the last one to finish.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "s3r_attn_common.cuh"
#include "s3r_attn_sched.cuh"
#include "s3r_device.cuh"
#include "s3r_internal.h"
#include "s3r_kvq.cuh"
#include "s3r_kvq_attn.cuh"

namespace s3r {
namespace kvq {

constexpr int kTok = 128;                    // tokens per stage
constexpr float kTop = 6.0f;                 // log2 of the largest weight when a row's reference is raised
constexpr float kTau = 2.0f;                 // lazy reference slack, log2 units: weights stay below 256
constexpr float kNuInit = 1e30f;             // -(reference) before the first score of a segment
constexpr int kSmemBudget = 232448 - 10240;  // beside the static arrays
constexpr int kMaxPend = 8;                  // deferred merges of units per CTA
constexpr int kThreads = 448;                // 12 worker warps, producer, MMA issuer
constexpr int kProducer = 12, kMma = 13;

// NRT rows are columns [0, NRT) (hi) and [NRT, 2 NRT) (lo) of N.
template <int NRT, int D, int BITS>
struct Lay {
  static constexpr int N = (2 * NRT + 15) / 16 * 16;
  static constexpr int kDk = D * BITS / 4;                 // contraction length of S^T (half-bytes of a row)
  static constexpr int kPlanes = BITS / 4;                 // half-bytes of a value's number, an O^T for each
  static constexpr int kKSub = kDk > 128 ? kDk / 128 : 1;  // TMEM tiles of a stage's keys: up to 128 of k, 32 columns
  static constexpr int kKCols = kDk / 4 / kKSub;
  static constexpr uint32_t kQBytes = N * (kDk < 128 ? 128 : kDk);   // [128 k][N rows][128 B]
  static constexpr uint32_t kPBytes = N * kTok;            // [N rows][128 B]
  static constexpr uint32_t kStage = 2 * (kTok * D * BITS / 8) + 8 * kTok;
  static constexpr int kNSraw = (kSmemBudget - (int)kQBytes - 2 * (int)kPBytes - 1024) / (int)kStage;
  static constexpr int kNS = kNSraw > 12 ? 12 : kNSraw;
  static constexpr uint32_t kOffP = kQBytes;
  static constexpr uint32_t kOffKV = kOffP + 2 * kPBytes;
  static constexpr uint32_t kDynBytes = kOffKV + kNS * kStage + 1024;
  // TMEM columns: NB key tiles, NB value tiles, S^T[2], O^T[planes]
  static constexpr int NB = (2 + kPlanes) * N + 256 <= 512 ? 4 : 2;
  static constexpr uint32_t kColK = 0, kColV = 32 * NB, kColS = 64 * NB, kColO = 64 * NB + 2 * N;
  static_assert(kNS >= 2, "the ring needs two stages");
  static_assert(64 * NB + (2 + kPlanes) * N <= 512, "TMEM columns");
};

// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f8f6f4 (e4m3 inputs, f32 accumulate), 32 of k.
__device__ __forceinline__ void umma_f8_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// 32 registers to this warp's TMEM lanes, 32 consecutive columns.
__device__ __forceinline__ void tmem_st32_raw(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
         "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
         "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 1-D bulk copy global -> this CTA's shared memory with an L2 policy.
__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                               uint64_t policy) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}

// 16 registers to this warp's TMEM lanes, 16 consecutive columns.
__device__ __forceinline__ void tmem_st16_raw(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Instruction descriptor, kind::f8f6f4 with e4m3 A/B and f32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The low and high half-bytes of a word's four bytes. ALT: complemented for
// every other token of the values' words (the high half-bytes at 4 bits, the
// odd bytes at 8).
template <int BITS, bool ALT>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t* r) {
  constexpr uint32_t kMask = 0x0f0f0f0fu;
  constexpr uint32_t kLo = ALT && BITS == 8 ? 0xff00ff00u : 0u, kHi = ALT ? (BITS == 4 ? ~0u : 0xff00ff00u) : 0u;
  r[0] = (w ^ kLo) & kMask;
  r[1] = ((w >> 4) ^ kHi) & kMask;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t e) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)e));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, float k) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(k));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, float k, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(k), *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Two values as e4m3 terms hi + lo / 32 (every step but the two roundings is exact in float16).
constexpr float kLo = 1.f / 32;
struct Split {
  uint32_t hi, lo;       // e4m3x2
  uint32_t hf, lf;       // their values, f16x2
};
__device__ __forceinline__ Split split2(uint32_t h2) {
  Split s;
  s.hi = e4m3x2_of(h2);
  s.hf = half2_of_e4m3x2(s.hi);
  s.lo = e4m3x2_of(fma2(s.hf, -32.f, mul2(h2, 32.f)));
  s.lf = half2_of_e4m3x2(s.lo);
  return s;
}

// Reduce C per-row values over the warp: lane l ends with row l % C.
template <int C, bool kMax>
__device__ __forceinline__ float rows_reduce(float* v, int lane) {
#pragma unroll
  for (int w = C / 2; w >= 1; w >>= 1) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float send = up ? v[k] : v[k + w];
      const float keep = up ? v[k + w] : v[k];
      const float got = __shfl_xor_sync(0xffffffffu, send, w);
      v[k] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  float r = v[0];
#pragma unroll
  for (int o = C; o < 32; o <<= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, r, o);
    r = kMax ? fmaxf(r, x) : r + x;
  }
  return r;
}
// The NR values of each of a warpgroup's threads, reduced over each warp into red[q4][row].
template <int NR, bool kMax>
__device__ __forceinline__ void warp_part(float* v, float (*red)[32], int q4, int lane) {
  if constexpr (NR == 4 || NR == 8) {
    const float r = rows_reduce<NR, kMax>(v, lane);
    if (lane < NR) red[q4][lane] = r;
  } else if constexpr (NR == 16) {
    const float r = rows_reduce<16, kMax>(v, lane);
    if (lane < 16) red[q4][lane] = r;
  } else if constexpr (NR == 24) {
    const float r = rows_reduce<16, kMax>(v, lane), r8 = rows_reduce<8, kMax>(v + 16, lane);
    if (lane < 16) red[q4][lane] = r;
    if (lane < 8) red[q4][16 + lane] = r8;
  } else {
    red[q4][lane] = rows_reduce<32, kMax>(v, lane);
  }
}

template <int T>
__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 1, %0;" ::"n"(T) : "memory"); }
// Number of the softmax threads whose predicate is true.
template <int T>
__device__ __forceinline__ int count_softmax(bool pred) {
  int r;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.popc.u32 %0, 1, %2, p;\n\t}"
               : "=r"(r) : "r"((int)pred), "n"(T) : "memory");
  return r;
}

// Listed pages are all walked, -1 entries among them.
__device__ __forceinline__ int unit_pages(const KvqAttnParams& p, int L) {
  if (kvq_bad_context(p, L)) return 0;
  return p.page_list ? p.budget : (L + p.P - 1) / p.P;
}

template <int NR, int NSM, int D, int P, int BITS>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const KvqAttnParams p) {
  constexpr int NRT = NR * NSM;
  using L = Lay<NRT, D, BITS>;
  constexpr int N = L::N, NB = L::NB;
  constexpr KvqLayout Y = kvq_layout(D, P, BITS);
  constexpr int NS = L::kNS;
  constexpr int NDQ = 3 - NSM;
  constexpr int kSoft = 128 * NSM;                       // softmax threads
  constexpr int ppt = kTok / P;                          // pages per stage
  constexpr float kMid = BITS == 4 ? 7.5f : 127.5f;
  static_assert(ppt * Y.page_bytes == (int)L::kStage, "stage bytes");
  extern __shared__ __align__(1024) uint8_t dyn_raw[];
  uint8_t* dyn = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t s_bar[2 * NS + 4 * NB + 8];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_ticket;
  __shared__ int4 s_pend[kMaxPend];                      // units this CTA merges at its end: (b, h, slot0, nseg)
  __shared__ int s_npend;
  __shared__ int s_prefix[kMaxSeqs + 1];
  __shared__ int s_stage_lp[NS][8];
  __shared__ int s_roff[64];                             // output row of packed row i relative to (b, h)
  __shared__ float s_red[4 * NSM][32];
  __shared__ float s_red2[4 * NSM][32];
  __shared__ __align__(16) float s_nu[64];               // -(reference) per row, log2 units
  __shared__ __align__(16) float s_alpha[64];            // rescale factor / row sum
  __shared__ __align__(16) float s_corr[64];             // sum of w (z / s + c) - c w' per row
  __shared__ __align__(16) float s_qs[2][64];            // sum of a query row, by segment parity
  __shared__ __align__(16) float s_qf[2][64];            // S^T's unit per row: 2^9 over the row's scale

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();

  if (warp == 0) {                                       // per-sequence prefix of unit pages
    const int per = (p.S + 31) / 32;
    const int b0 = min(p.S, lane * per), b1 = min(p.S, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += unit_pages(p, p.context_lens[b]) * p.Hkv;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int run = incl - sum;
    for (int b = b0; b < b1; ++b) {
      s_prefix[b] = run;
      run += unit_pages(p, p.context_lens[b]) * p.Hkv;
    }
    if (lane == 31) s_prefix[p.S] = incl;
  }
  if (tid < 64) s_roff[tid] = (tid / p.G) * p.Hq + (tid % p.G);
  __syncthreads();
  // inputs (cache, table, lengths, queries) may be read before the
  // grid-dependency wait; page lists, outputs and the workspace only after it
  if (blockIdx.x == 0) {
    pdl_wait();
    for (int b = 0; b < p.S; ++b) {
      if (!kvq_bad_context(p, p.context_lens[b])) continue;
      if (tid == 0) flag_status(p.status, S3R_DEV_BAD_CONTEXT_LEN);
      for (int h = 0; h < p.Hkv; ++h) kvq_write_empty<__nv_bfloat16>(p, b, h, tid, kThreads);
    }
  }
  const int total = s_prefix[p.S];
  // at least one stage of pages per CTA (shorter pieces would cost a merge
  // for less than a stage); with lists, a whole unit per CTA where the units
  // nearly fill the grid, so that none is split
  int W = max((total + (int)gridDim.x - 1) / (int)gridDim.x, ppt);
  if (p.page_list && W < p.budget && p.S * p.Hkv * 5 >= (int)gridDim.x * 4) W = p.budget;
  const int lo = blockIdx.x * W, hi = min(total, lo + W);
  if (lo >= hi) {                                        // uniform over the CTA
    pdl_wait();
    return;
  }

  const uint32_t bar0 = smem_addr(&s_bar[0]);
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  // KF / VF: an unpacked tile of keys / values is in TMEM; KE / VE: the MMAs
  // have read it; SF: S^T(g) is complete; PF: w(g) is written (and S^T(g)
  // read); OD: O^T has stage g's part; by the parity of the tile or stage
  constexpr int B_FULL = 0, B_EMPTY = NS, B_KF = 2 * NS, B_KE = B_KF + NB, B_VF = B_KE + NB, B_VE = B_VF + NB,
                B_SF = B_VE + NB, B_PF = B_SF + 2, B_OD = B_PF + 2, B_QF = B_OD + 2, B_TD = B_QF + 1;
  uint8_t* sQ = dyn;
  uint8_t* sP = dyn + L::kOffP;
  uint8_t* sKV = dyn + L::kOffKV;
  const uint32_t aQ = smem_addr(sQ), aP = smem_addr(sP), aKV = smem_addr(sKV);

  if (warp == kMma) {
    tmem_alloc(smem_addr(&s_tmem), 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(BAR(B_FULL + i), 1);
      mbar_init(BAR(B_EMPTY + i), 12);                   // every worker warp
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(BAR(B_KF + i), 4);
      mbar_init(BAR(B_KE + i), 1);
      mbar_init(BAR(B_VF + i), 4);
      mbar_init(BAR(B_VE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(B_SF + i), 1);
      mbar_init(BAR(B_PF + i), 4 * NSM);
      mbar_init(BAR(B_OD + i), 1);
    }
    mbar_init(BAR(B_QF), 4 * NSM);
    mbar_init(BAR(B_TD), 1);
    s_abort = 0;
    s_npend = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == kProducer) {
    // ======================================================= producer warp
    if (p.page_list) pdl_wait();
    const uint64_t pol = l2_policy_evict_first();
    // page-id windows of 32 flattened positions: lane k of a window holds
    // position wbase + k. w0 = in use, w1 = page ids in flight, w2 = logical pages
    // in flight.
    int w0_lp, w0_ph, w1_lp, w1_ph, w2_lp, w2_u, u;
    auto phys_load = [&](int lp, int unit) {
      if (lp == -1) return -1;
      const int b = unit / p.Hkv;
      const int n_b = (p.context_lens[b] + P - 1) / P;
      if (lp < 0 || lp >= n_b) { flag_status(p.status, S3R_DEV_BAD_PAGE_ID); return -1; }
      const int ph = p.block_table[(size_t)b * p.max_pages + lp];
      if (ph < 0 || ph >= p.num_pages_total) { flag_status(p.status, S3R_DEV_BAD_PAGE_ID); return -1; }
      return ph;
    };
    int wbase = lo;
    page_of(p, s_prefix, wbase + lane, hi, W, &w0_lp, &u);
    w0_ph = phys_load(w0_lp, u);
    page_of(p, s_prefix, wbase + 32 + lane, hi, W, &w1_lp, &u);
    w1_ph = phys_load(w1_lp, u);
    page_of(p, s_prefix, wbase + 64 + lane, hi, W, &w2_lp, &w2_u);
    bool waited = p.page_list != nullptr;
    int g = 0;
    bool ok = true;
    for (int x = lo; x < hi && ok;) {
      const Seg sg = locate(p, s_prefix, x, hi, W);
      const int nst = (sg.npg + ppt - 1) / ppt;
      for (int j = 0; j < nst; ++j, ++g) {
        const int st = g % NS;
        if (g == NS && !waited) {                        // the ring's first fill goes out before it
          pdl_wait();
          waited = true;
        }
        int my_lp = -1, my_ph = -1;
        for (int pp = 0; pp < ppt; ++pp) {
          // positions past the segment belong to the next one: the windows
          // must not move past its first page (warp-uniform)
          if (j * ppt + pp >= sg.npg) break;
          const int xp = x + j * ppt + pp;
          while (xp >= wbase + 32) {                     // advance the windows (warp-uniform)
            wbase += 32;
            w0_lp = w1_lp; w0_ph = w1_ph;
            w1_lp = w2_lp;
            w1_ph = phys_load(w1_lp, w2_u);
            page_of(p, s_prefix, wbase + 64 + lane, hi, W, &w2_lp, &w2_u);
          }
          const int src = xp - wbase;
          const int lp = __shfl_sync(0xffffffffu, w0_lp, src & 31);
          const int ph = __shfl_sync(0xffffffffu, w0_ph, src & 31);
          if (lane == pp) { my_lp = lp; my_ph = ph; }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(BAR(B_EMPTY + st), ((g / NS) & 1) ^ 1, &s_abort, p.status))) {
          ok = false;
          break;
        }
        if (lane < 8) s_stage_lp[st][lane] = my_ph >= 0 ? my_lp : -1;
        const unsigned real = __ballot_sync(0xffffffffu, my_ph >= 0);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(BAR(B_FULL + st), (uint32_t)__popc(real) * Y.page_bytes);
        __syncwarp();
        if (my_ph >= 0)
          bulk_load_hint(aKV + st * L::kStage + lane * Y.page_bytes,
                         p.pages + ((size_t)my_ph * p.Hkv + sg.h) * Y.page_bytes, Y.page_bytes, BAR(B_FULL + st), pol);
      }
      x = sg.end;
    }
    if (!waited) pdl_wait();
    // drain: wait until every issued copy has landed
    if (lane == 0)
      for (int k = max(0, g - NS); k < g; ++k) mbar_wait_drain(BAR(B_FULL + k % NS), (k / NS) & 1, p.status);
  } else if (warp == kMma) {
    // ======================================================= MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(128, N);
      Cursor qc = cursor_begin(p, s_prefix, lo, hi, W, ppt);
      Cursor pc = qc;
      int qsub = 0, psub = 0, kt = 0, vt = 0;            // tile within the stage, tiles so far
      // Q and w: K-major, 128-byte rows, 8-row groups 1024 B apart; a K32
      // step is 32 bytes inside the swizzle row, the next 128 of k (the next
      // tile) N x 128 B further. A tile's K32 step is 8 TMEM columns.
      const uint64_t dQ0 = smem_desc_sw128(aQ, 16, 1024), dP0 = smem_desc_sw128(aP, 16, 1024);
      constexpr uint64_t kBlock = (N * 128) >> 4;
      // QK(g) needs its keys (first in a segment, also the segment's Q) and
      // PV(g - 2) issued (w(g - 2) written: S^T buffer g & 1 has been read);
      // PV(g) needs w(g) and its values. Each tile is issued as soon as it is
      // ready. Bounded: no progress for the wait limit flags a timeout and stops.
      auto issue_qk = [&]() {
        tc_fence_after();
        const int buf = kt % NB;
        const uint32_t dS = tmem + L::kColS + (qc.g & 1) * N, a = tmem + L::kColK + buf * 32;
        const uint64_t qd = dQ0 + (uint64_t)qsub * kBlock;
#pragma unroll
        for (int kk = 0; kk < L::kKCols / 8; ++kk)
          umma_f8_ta(dS, a + kk * 8, qd + kk * 2, idesc, (kk > 0 || qsub > 0) ? 1u : 0u);
        umma_commit(BAR(B_KE + buf));
        ++kt;
        if (++qsub == L::kKSub) {
          qsub = 0;
          umma_commit(BAR(B_SF + (qc.g & 1)));
          cursor_next(p, s_prefix, hi, W, ppt, qc);
        }
      };
      auto issue_pv = [&]() {
        tc_fence_after();
        const int buf = vt % NB;
        const uint32_t a = tmem + L::kColV + buf * 32, dO = tmem + L::kColO + psub * N;
        const uint64_t pd = dP0 + (uint64_t)(pc.g & 1) * (L::kPBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f8_ta(dO, a + kk * 8, pd + kk * 2, idesc, (kk > 0 || pc.j > 0) ? 1u : 0u);
        umma_commit(BAR(B_VE + buf));
        ++vt;
        if (++psub == L::kPlanes) {
          psub = 0;
          umma_commit(BAR(B_OD + (pc.g & 1)));
          cursor_next(p, s_prefix, hi, W, ppt, pc);
        }
      };
      unsigned long long idle_since = 0;
      uint32_t spins = 0;
      while (pc.valid) {
        bool progress = false;
        if ((psub != 0 || mbar_test_wait(BAR(B_PF + (pc.g & 1)), (pc.g >> 1) & 1)) &&
            mbar_test_wait(BAR(B_VF + vt % NB), (vt / NB) & 1)) {
          issue_pv();
          progress = true;
        }
        if (qc.valid && qc.g <= pc.g + 1 && (qc.j != 0 || qsub != 0 || mbar_test_wait(BAR(B_QF), qc.s & 1)) &&
            mbar_test_wait(BAR(B_KF + kt % NB), (kt / NB) & 1)) {
          issue_qk();
          progress = true;
        }
        if (progress) {
          idle_since = 0;
          continue;
        }
        if ((++spins & 63u) == 0) {
          if (*(volatile int*)&s_abort) break;
          const unsigned long long now = globaltimer_ns();
          if (idle_since == 0) {
            idle_since = now;
          } else if (now - idle_since > kWaitLimitNs) {
            *(volatile int*)&s_abort = 1;
            flag_status(p.status, S3R_DEV_WAIT_TIMEOUT);
            break;
          }
        }
      }
      umma_commit(BAR(B_TD));
    }
  } else if (warp >= 4 * NSM) {
    // ======================================================= unpacking warps
    const int wg = (warp - 4 * NSM) >> 2;                // 0: keys (and values where NDQ = 1), 1: values
    const int t = tid & 127;                             // TMEM lane: token of S^T, channel of O^T
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
    Cursor c = cursor_begin(p, s_prefix, lo, hi, W, ppt);
    int kt = 0, vt = 0;
    bool ok = true;
    for (; c.valid && ok; cursor_next(p, s_prefix, hi, W, ppt, c)) {
      const int st = c.g % NS;
      ok = __all_sync(0xffffffffu, mbar_wait(BAR(B_FULL + st), (c.g / NS) & 1, &s_abort, p.status));
      if (!ok) break;
      const uint8_t* stage = sKV + st * L::kStage;
      if (wg == 0) {
        const uint8_t* row = stage + (t / P) * Y.page_bytes + (t % P) * 16;
#pragma unroll
        for (int sub = 0; sub < L::kKSub; ++sub, ++kt) {
          ok = __all_sync(0xffffffffu, mbar_wait(BAR(B_KE + kt % NB), ((kt / NB) & 1) ^ 1, &s_abort, p.status));
          if (!ok) break;
          tc_fence_after();
          uint32_t r[L::kKCols];
#pragma unroll
          for (int k = 0; k < L::kKCols / 8; ++k) {
            const uint4 w = *reinterpret_cast<const uint4*>(row + (sub * 4 + k) * (P * 16));
            unpack<BITS, false>(w.x, r + 8 * k);
            unpack<BITS, false>(w.y, r + 8 * k + 2);
            unpack<BITS, false>(w.z, r + 8 * k + 4);
            unpack<BITS, false>(w.w, r + 8 * k + 6);
          }
          const uint32_t dst = tmem + lane_base + L::kColK + (kt % NB) * 32;
          if constexpr (L::kKCols == 32) tmem_st32_raw(dst, r);
          else tmem_st16_raw(dst, r);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(B_KF + kt % NB));
        }
        if (!ok) break;
      }
      if (wg == NDQ - 1) {
        // the halves of 8-bit numbers are two tiles, taken together
#pragma unroll
        for (int i = 0; i < L::kPlanes; ++i)
          ok = ok && __all_sync(0xffffffffu, mbar_wait(BAR(B_VE + (vt + i) % NB), (((vt + i) / NB) & 1) ^ 1, &s_abort, p.status));
        if (!ok) break;
        tc_fence_after();
        if (D == 128 || t < D) {                         // whole warps; lanes past D hold anything and are never read
          const uint32_t dst = tmem + lane_base + L::kColV;
          constexpr int kWordsPage = P * BITS / 32;      // words of a channel in one page: 2, 4, 8 or 16
#pragma unroll
          for (int half = 0; half < L::kPlanes; ++half) {
            uint32_t r[32];
            // the channel's words half * 16 .. + 15 of the stage
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              uint32_t w[4];
              if constexpr (Y.unit == 16) {
                const int word = half * 16 + k, pg = word / kWordsPage, u = word % kWordsPage / 4;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + pg * Y.page_bytes + Y.off_v + (u * D + t) * 16);
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
              } else {
                const int pg = k / 2;
                const uint2 v0 = *reinterpret_cast<const uint2*>(stage + pg * Y.page_bytes + Y.off_v + t * 8);
                const uint2 v1 = *reinterpret_cast<const uint2*>(stage + (pg + 1) * Y.page_bytes + Y.off_v + t * 8);
                w[0] = v0.x; w[1] = v0.y; w[2] = v1.x; w[3] = v1.y;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t x[2];
                unpack<BITS, true>(w[i], x);
                if constexpr (BITS == 4) {
                  r[2 * (k + i)] = x[0];
                  r[2 * (k + i) + 1] = x[1];
                } else {
                  r[k + i] = x[0];
                  r[16 + k + i] = x[1];
                }
              }
            }
            if constexpr (BITS == 4) {
              tmem_st32_raw(dst + (vt % NB) * 32, r);
            } else {
              tmem_st16_raw(dst + (vt % NB) * 32 + half * 16, r);
              tmem_st16_raw(dst + ((vt + 1) % NB) * 32 + half * 16, r + 16);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < L::kPlanes; ++i, ++vt)
          if (lane == 0) mbar_arrive(BAR(B_VF + vt % NB));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_EMPTY + st));
    }
  } else {
    // ======================================================= softmax warps
    const int wg = NSM == 1 ? 0 : warp >> 2;             // rows wg * NR ..
    const int q4 = warp & 3, t = tid & 127;              // token of the stage; channel in the epilogue
    const int rb = wg * NR;
    const uint32_t lane_base = (uint32_t)q4 << 21;
    constexpr int kDc = D / 8;                           // lanes of 8 channels per Q row
    constexpr int kQC = (NRT * kDc + kSoft - 1) / kSoft;
    auto q_at = [&](const Seg& s, int ch) {
      const size_t base = (size_t)(s.b * p.R + p.r0) * p.Hq + (size_t)s.h * p.G;
      return static_cast<const __nv_bfloat16*>(p.q) + (base + s_roff[ch / kDc]) * D + (ch % kDc) * 8;
    };
    auto q_prefetch = [&](const Seg& s) {
#pragma unroll
      for (int k = 0; k < kQC; ++k) {
        const int ch = tid + kSoft * k;
        if (ch / kDc < p.rows && (ch & 3) == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(q_at(s, ch)));
      }
    };
    // A segment's Q as two e4m3 terms of q 2^e in the order of the unpacked
    // numbers, 2^e the row's power-of-two scale; the sum of each row.
    auto q_store = [&](const Seg& s, int par) {
#pragma unroll
      for (int k = 0; k < kQC; ++k) {
        const int ch = tid + kSoft * k, r = ch / kDc, c8 = ch % kDc;
        if (NRT * kDc % kSoft != 0 && r >= NRT) break;   // uniform over a warp
        const uint4 qv = r < p.rows ? __ldg(reinterpret_cast<const uint4*>(q_at(s, ch))) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {qv.x, qv.y, qv.z, qv.w};
        float x[8], sum = 0.f, big = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16);
          x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          sum += x[2 * i] + x[2 * i + 1];
          big = fmaxf(big, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
        }
#pragma unroll
        for (int o = kDc / 2; o >= 1; o >>= 1) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        }
        // largest value into [128, 256) (4 bits) or [8, 16) (8 bits: 16 q is met too)
        const int ex = min(max((int)(__float_as_uint(big) >> 23), 40), 240);
        const int top = BITS == 4 ? 7 : 3;
        const float up = __uint_as_float((uint32_t)(254 - ex + top) << 23);
        if (c8 == 0) {
          s_qs[par][r] = sum;
          s_qf[par][r] = 512.f / up;
        }
        uint32_t hi[4], lo[4];                           // e4m3 pairs: channels (0, 2) (4, 6) (1, 3) (5, 7), or in order
        uint8_t* const at = sQ + r * 128;
          constexpr int kLoRow = NRT * 128;
        if constexpr (BITS == 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c0 = (i & 1) * 4 + (i >> 1);
            const Split sp = split2(half2_of(x[c0] * up, x[c0 + 2] * up));
            hi[i] = sp.hi;
            lo[i] = sp.lo;
          }
          // 8 bytes at k = 8 c8; hi and lo rows may differ in r & 7
          const int place = ((c8 >> 1) << 4), sub = (c8 & 1) * 8;
          *reinterpret_cast<uint2*>(at + (place ^ ((r & 7) << 4)) + sub) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(at + kLoRow + (place ^ (((r + NRT) & 7) << 4)) + sub) =
              make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        } else {
          uint32_t hx[4], lx[4];                         // the same times 16 (exact)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Split sp = split2(half2_of(x[2 * i] * up, x[2 * i + 1] * up));
            hi[i] = sp.hi;
            lo[i] = sp.lo;
            hx[i] = e4m3x2_of(mul2(sp.hf, 16.f));
            lx[i] = e4m3x2_of(mul2(sp.lf, 16.f));
          }
          const int place = (c8 & 7) << 4;
          uint8_t* const blk = at + (c8 >> 3) * (N * 128);
          *reinterpret_cast<uint4*>(blk + (place ^ ((r & 7) << 4))) =
              make_uint4(hi[0] | hi[1] << 16, hx[0] | hx[1] << 16, hi[2] | hi[3] << 16, hx[2] | hx[3] << 16);
          *reinterpret_cast<uint4*>(blk + kLoRow + (place ^ (((r + NRT) & 7) << 4))) =
              make_uint4(lo[0] | lo[1] << 16, lx[0] | lx[1] << 16, lo[2] | lo[3] << 16, lx[2] | lx[3] << 16);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_QF));
    };
    // where this thread's weights go: its token's place along k
    const int kpos = BITS == 4 ? (t & ~7) + ((t & 1) << 2) + ((t & 7) >> 1) : t;
    uint8_t* const pw = sP + (kpos & 15);
    const int pck = kpos >> 4;
    const uint32_t sign = (t & 1) ? 0x80008000u : 0u;    // every other token's weights are negated

    Seg sg = locate(p, s_prefix, lo, hi, W);
    q_prefetch(sg);                                      // an input: no earlier kernel writes it
    pdl_wait();
    q_store(sg, 0);
    // C rows' columns of S^T or O^T, from column `at` of the hi ones: x[r] hi, x[C + r] lo
    constexpr int C = NR <= 8 ? NR : 8;
    auto load_rows = [&](uint32_t at, float* x) {
      if constexpr (C == 4) {                            // hi and lo side by side
        tmem_ld8(at, x);
      } else {
        tmem_ld8(at, x);
        tmem_ld8(at + NRT, x + C);
      }
      tmem_wait_ld();
    };
    auto scale_o = [&]() {
#pragma unroll
      for (int k = 0; k < L::kPlanes; ++k)
#pragma unroll
        for (int c = 0; c < NR; c += C) {
          const uint32_t at = tmem + lane_base + L::kColO + k * N + rb + c;
          float x[2 * C];
          load_rows(at, x);
#pragma unroll
          for (int r = 0; r < C; ++r) {
            x[r] *= s_alpha[rb + c + r];
            x[C + r] *= s_alpha[rb + c + r];
          }
          tmem_st8(at, x);
          if constexpr (C != 4) tmem_st8(at + NRT, x + C);
        }
      tmem_wait_st();
    };
    int g = 0;
    bool ok = true;
    int par = 0;
    for (int x = lo; x < hi; par ^= 1) {
      const bool has_next = sg.end < hi;
      Seg nx = sg;
      if (has_next) {
        nx = locate(p, s_prefix, sg.end, hi, W);
        q_prefetch(nx);
      }
      const int nst = (sg.npg + ppt - 1) / ppt;
      const int Lb = p.context_lens[sg.b];
      if (tid < NRT) s_nu[tid] = kNuInit;
      float l[NR], corr[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) l[r] = corr[r] = 0.f;
      sync_softmax<kSoft>();
      bool abort_all = false;
      for (int j = 0; j < nst; ++j, ++g) {
        const int st = g % NS, sb = g & 1;
        ok &= mbar_wait(BAR(B_FULL + st), (g / NS) & 1, &s_abort, p.status);
        // this thread's token: parameters, position, hidden rows
        const uint8_t* pg = sKV + st * L::kStage + (t / P) * Y.page_bytes;
        const uint32_t kp = *reinterpret_cast<const uint32_t*>(pg + Y.off_kp + (t % P) * 4);
        const uint32_t vp = *reinterpret_cast<const uint32_t*>(pg + Y.off_vp + (t % P) * 4);
        const int lp = s_stage_lp[st][t / P];
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_EMPTY + st));
        const int pos = lp * P + (t % P);
        const bool valid = lp >= 0 && pos < Lb;
        uint32_t hide = valid ? 0u : ~0u;
        const int excess = pos - (Lb - p.R) - p.r0;      // rows before it do not see the token
        if (valid && excess > 0) {
          const int nm = p.G * excess - rb;
          hide = nm <= 0 ? 0u : nm >= 32 ? ~0u : (1u << nm) - 1u;
        }
        const float sk = __uint_as_float(kp << 16), zk = __uint_as_float(kp & 0xffff0000u);
        float sv = __uint_as_float(vp << 16);
        float zc = __fdividef(__uint_as_float(vp & 0xffff0000u), sv) + kMid;
        const float ka = p.scale_log2 * sk, kb = p.scale_log2 * zk;
        if (!valid) {
          sv = 1.f;
          zc = 0.f;
        } else if (!(fabsf(sv) + fabsf(zc) < INFINITY)) {   // a NaN row: the rows that see it, and only they
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (!((hide >> r) & 1u)) corr[r] = __int_as_float(0x7fc00000);
          sv = 1.f;
          zc = 0.f;
        }
        const float rsv = __fdividef(1.f, sv), lgs = __log2f(sv);
        ok &= mbar_wait(BAR(B_SF + sb), (g >> 1) & 1, &s_abort, p.status);
        tc_fence_after();
        float s[NR];
        // s <- y + log2 s_v (- reference); hidden: -inf. Rows in steps of C,
        // so that few of S^T's columns are live at once.
        auto load_s = [&](bool with_ref) {
#pragma unroll
          for (int c = 0; c < NR; c += C) {
            float x[2 * C];
            load_rows(tmem + lane_base + L::kColS + sb * N + rb + c, x);
#pragma unroll
            for (int r = 0; r < C; r += 4) {
              const float4 qs = *reinterpret_cast<const float4*>(&s_qs[par][rb + c + r]);
              const float4 qf = *reinterpret_cast<const float4*>(&s_qf[par][rb + c + r]);
              float4 nu = make_float4(0.f, 0.f, 0.f, 0.f);
              if (with_ref) nu = *reinterpret_cast<const float4*>(&s_nu[rb + c + r]);
              s[c + r] = fmaf(fmaf(x[C + r], kLo, x[r]) * qf.x, ka, fmaf(qs.x, kb, nu.x + lgs));
              s[c + r + 1] = fmaf(fmaf(x[C + r + 1], kLo, x[r + 1]) * qf.y, ka, fmaf(qs.y, kb, nu.y + lgs));
              s[c + r + 2] = fmaf(fmaf(x[C + r + 2], kLo, x[r + 2]) * qf.z, ka, fmaf(qs.z, kb, nu.z + lgs));
              s[c + r + 3] = fmaf(fmaf(x[C + r + 3], kLo, x[r + 3]) * qf.w, ka, fmaf(qs.w, kb, nu.w + lgs));
            }
          }
          if (hide) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
              if ((hide >> r) & 1u) s[r] = -INFINITY;
          }
        };
        load_s(true);
        float ymax = s[0];
#pragma unroll
        for (int r = 1; r < NR; ++r) ymax = fmaxf(ymax, s[r]);
        // one barrier per stage: stop together, or raise the references together
        const int cnt = count_softmax<kSoft>(!ok || ymax > kTop + kTau);
        bool rescale_o = false;
        if (cnt > 0) {
          if (count_softmax<kSoft>(!ok) > 0) { abort_all = true; break; }
          // stage maximum per row (S^T is intact until PF), then reload
          load_s(false);
          warp_part<NR, true>(s, &s_red[4 * wg], q4, lane);
          sync_softmax<kSoft>();
          if (t < NR) {
            const float mx = fmaxf(fmaxf(s_red[4 * wg][t], s_red[4 * wg + 1][t]),
                                   fmaxf(s_red[4 * wg + 2][t], s_red[4 * wg + 3][t]));
            const float m_old = -s_nu[rb + t];
            const float m_new = fmaxf(m_old, mx - kTop);
            s_alpha[rb + t] = ex2(m_old - m_new);
            s_nu[rb + t] = -m_new;
          }
          sync_softmax<kSoft>();
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float a = s_alpha[rb + r];
            l[r] *= a;
            corr[r] *= a;
          }
          load_s(true);
          rescale_o = j > 0;
        }
        // w buffer sb was last read by PV(g - 2); a rescale of O^T also needs
        // PV(g - 1) done
        const int gw = g - (rescale_o ? 1 : 2);
        if (gw >= 0) ok &= mbar_wait(BAR(B_OD + (gw & 1)), (gw >> 1) & 1, &s_abort, p.status);
        tc_fence_after();
        if (rescale_o) {
          scale_o();
        }
        uint8_t* const pb = pw + sb * L::kPBytes;
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          const float w0 = ex2(s[r]), w1 = ex2(s[r + 1]);
          l[r] = fmaf(w0, rsv, l[r]);
          l[r + 1] = fmaf(w1, rsv, l[r + 1]);
          const Split sp = split2(half2_of(w0, w1) ^ sign);
          const uint32_t rounded = fma2(sp.lf, kLo, sp.hf);
          const float2 wr = __half22float2(*reinterpret_cast<const __half2*>(&rounded));
          corr[r] = fmaf(w0, zc, fmaf(wr.x, -kMid, corr[r]));
          corr[r + 1] = fmaf(w1, zc, fmaf(wr.y, -kMid, corr[r + 1]));
          // rows rb + r, rb + r + 1 (hi) and NRT further (lo)
          const int i0 = rb + r, i1 = i0 + 1;
          pb[i0 * 128 + ((pck ^ (i0 & 7)) << 4)] = (uint8_t)sp.hi;
          pb[i1 * 128 + ((pck ^ (i1 & 7)) << 4)] = (uint8_t)(sp.hi >> 8);
          pb[(NRT + i0) * 128 + ((pck ^ ((NRT + i0) & 7)) << 4)] = (uint8_t)sp.lo;
          pb[(NRT + i1) * 128 + ((pck ^ ((NRT + i1) & 7)) << 4)] = (uint8_t)(sp.lo >> 8);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_PF + sb));
      }
      if (abort_all) break;
      // ---- the last QK of this segment is done: stage the next segment's Q
      if (has_next) q_store(nx, par ^ 1);
      // ---- segment epilogue: row sums, then (O^T + corr) / l
      warp_part<NR, false>(l, &s_red[4 * wg], q4, lane);
      warp_part<NR, false>(corr, &s_red2[4 * wg], q4, lane);
      sync_softmax<kSoft>();
      const bool single = sg.nseg == 1;
      const int slot_idx = sg.unit + blockIdx.x;         // partial slot of (unit, this CTA)
      const size_t rowbase = (size_t)(sg.b * p.R + p.r0) * p.Hq + (size_t)sg.h * p.G;
      if (t < NR) {
        const int i = rb + t;
        const float lt = (s_red[4 * wg][t] + s_red[4 * wg + 1][t]) + (s_red[4 * wg + 2][t] + s_red[4 * wg + 3][t]);
        const float ct = (s_red2[4 * wg][t] + s_red2[4 * wg + 1][t]) + (s_red2[4 * wg + 2][t] + s_red2[4 * wg + 3][t]);
        const float m = -s_nu[i];
        if (i < p.rows) {
          if (single) {
            if (p.lse) p.lse[rowbase + s_roff[i]] = lt == 0.f ? -INFINITY : (m + log2f(lt)) * kLn2;
          } else {
            const size_t pi = (size_t)slot_idx * p.rows + i;
            p.part_ml[pi * 2] = m;
            p.part_ml[pi * 2 + 1] = lt;
          }
        }
        s_alpha[i] = lt == 0.f ? 0.f : 1.f / lt;
        s_corr[i] = ct;
      }
      ok &= mbar_wait(BAR(B_OD + ((g - 1) & 1)), ((g - 1) >> 1) & 1, &s_abort, p.status);   // PV of the last stage
      tc_fence_after();
      sync_softmax<kSoft>();
      {
#pragma unroll
        for (int c = 0; c < NR; c += C) {
          float x[L::kPlanes][2 * C];
#pragma unroll
          for (int k = 0; k < L::kPlanes; ++k) load_rows(tmem + lane_base + L::kColO + k * N + rb + c, x[k]);
          if (D == 128 || t < D) {
#pragma unroll
            for (int r = 0; r < C; ++r) {
              const int i = rb + c + r;
              if (i >= p.rows) break;
              float o = fmaf(x[0][C + r], kLo, x[0][r]);
              if constexpr (BITS == 8) o = fmaf(fmaf(x[1][C + r], kLo, x[1][r]), 16.f, o);
              o = fmaf(o, 512.f, s_corr[i]);
              if (single)
                static_cast<__nv_bfloat16*>(p.out)[(rowbase + s_roff[i]) * D + t] = __float2bfloat16_rn(o * s_alpha[i]);
              else
                p.part_o[((size_t)slot_idx * p.rows + i) * D + t] = o;
            }
          }
        }
      }
      tc_fence_before();
      if (!single) {
        __threadfence();
        sync_softmax<kSoft>();
        if (tid == 0) s_ticket = atomicAdd(p.tickets + sg.unit, 1u);
        sync_softmax<kSoft>();
        if (s_ticket == sg.nseg - 1) {
          // this CTA finished the unit last: merge its partials after the
          // CTA's own streaming is done (immediately if the list is full)
          if (s_npend < kMaxPend) {
            if (tid == 0) s_pend[s_npend] = make_int4(sg.b, sg.h, sg.first_cta + sg.unit, sg.nseg);
          } else {
            __threadfence();
            kvq_combine<__nv_bfloat16>(p, sg.b, sg.h, sg.first_cta + sg.unit, sg.nseg, kSoft);
          }
          sync_softmax<kSoft>();
          if (tid == 0) {
            if (s_npend < kMaxPend) ++s_npend;
            p.tickets[sg.unit] = 0u;
          }
        }
      }
      sync_softmax<kSoft>();                             // s_alpha / s_nu reads done
      x = sg.end;
      sg = nx;
    }
    // ---- deferred merges of the units this CTA finished last (skipped,
    // together, after a failed wait)
    if (count_softmax<kSoft>(!ok) == 0) {
      __threadfence();
      for (int k = 0; k < s_npend; ++k) {
        const int4 u = s_pend[k];
        kvq_combine<__nv_bfloat16>(p, u.x, u.y, u.z, u.w, kSoft);
      }
    }
  }

  // ---- teardown: every role is done; wait for the MMAs, free TMEM
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    if (lane == 0) mbar_wait_drain(BAR(B_TD), 0, p.status);
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int NR, int NSM, int D, int P, int BITS>
cudaError_t launch_one(const KvqAttnParams& p, cudaStream_t st) {
  const size_t smem = Lay<NR * NSM, D, BITS>::kDynBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<NR, NSM, D, P, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  int grid = device_sm_count();
  if (grid > kMaxPersistentCtas) grid = kMaxPersistentCtas;
  return launch_kernel(attn_kernel<NR, NSM, D, P, BITS>, dim3(grid), dim3(kThreads), smem, st, 1, p);
}

// Rows of the softmax: the packed rows rounded up; beyond 24, two warpgroups
// share them. TMEM holds S^T and O^T of 64 rows at 4 bits, of 48 at 8.
template <int D, int P, int BITS>
cudaError_t launch_rows(const KvqAttnParams& p, cudaStream_t st) {
  if (p.rows <= 4) return launch_one<4, 1, D, P, BITS>(p, st);
  if (p.rows <= 8) return launch_one<8, 1, D, P, BITS>(p, st);
  if (p.rows <= 16) return launch_one<16, 1, D, P, BITS>(p, st);
  if (p.rows <= 24) return launch_one<24, 1, D, P, BITS>(p, st);
  if (p.rows <= 32) return launch_one<16, 2, D, P, BITS>(p, st);
  if (p.rows <= 48) return launch_one<24, 2, D, P, BITS>(p, st);
  if constexpr (BITS == 4) return launch_one<32, 2, D, P, BITS>(p, st);
  else return cudaErrorInvalidValue;
}

}  // namespace kvq
}  // namespace s3r
