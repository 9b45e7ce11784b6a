// Attention over the quantised paged KV cache on the tensor cores, bf16
// queries, up to 64 packed rows (G query heads x R rows) per (sequence, KV
// head). Layout and arithmetic of a held row: s3r_kvq.cuh.
//
// The held numbers themselves go through the tensor cores, as n - c with a
// constant c; scales and minima meet the results outside:
//   S^T[t, i] = sum_d (n_k[t, d] - c) q[i, d]
//   y         = scale log2 e (s_k[t] S^T + (z_k[t] + c s_k[t]) sum_d q[i, d]),   p = 2^(y - reference)
//   w[t, i]   = p s_v[t], rounded to w'
//   O^T[d, i] = sum_t (n_v[t, d] - c) w'[t, i]
//   out       = (O^T + sum_t w (z_v[t] / s_v[t] + c)) / sum_t p
// The reference of a row bounds y + log2 s_v, so that w stays in a narrow
// type's range whatever the values' scales (a row of equal values has no numbers for w to meet
// and counts with a step of 2^-8 of its value); queries are met as q 2^e with a
// power of two per row. Sums over tokens stay near zero (with n itself, or 16
// + n, the accumulator's truncation built up an error of 1e-2 over 16384 tokens).
//
// Two forms of the numbers:
// - f16, c = 8 or 128 (8 bits; 4 bits beyond 16 rows): a number placed in the
//   mantissa of 1024 (or 16 times it, in place, for the odd half-bytes) by one
//   logic operation for two, centred by one fused multiply-add: 9 instructions
//   for eight 4-bit numbers, 8 for eight 8-bit ones. Queries and weights are one f16
//   term (w to 2^-12 of itself, a bf16 query exactly down to 2^-21 of its row's largest).
// - e4m3, c = 0 (4 bits, up to 16 rows): a 4-bit number in the low bits of a
//   byte is, read as e4m3, exactly n 2^-9 (subnormals and the first binade have
//   one spacing): 3 instructions for eight. Queries and weights are two terms hi +
//   lo / 32 in separate columns, w rounded to 9 bits once for both its sums.
//   Every other token's numbers are complemented (15 - n) and its weights
//   negated, which keeps the sums over tokens near zero. Below 2^-5 (the largest weight
//   lies in 2^6 to 2^8) a weight has fewer bits, down to whole steps of 2^-14, taken up or down by a
//   threshold of the token's own so that sums keep their value. The two terms cost the
//   softmax about 8 instructions a row and token: 64 x 8192 tokens with 8 KV heads
//   take 131 us a call at 4 rows against 230 in f16, 157 against 239 at 8, 218 against
//   257 at 16, but 324 against 274 at 24.
//
// Both operands of numbers are the MMA's A operand (M = 128 tokens of S^T, M =
// 128 lanes of channels of O^T) and live in tensor memory: a thread unpacks
// one token's channels (one channel's tokens) from 16-byte shared-memory reads
// into registers and stores them to its TMEM lane, so the unpacked form, 2 to 4
// times the packed bytes, never crosses shared memory. Q and w are the B
// operands in shared memory.
//
// Warps: two softmax warpgroups (thread = token), two unpacking ones, one
// producer (a bulk copy per (page, head) into a ring of 128-token stages), one
// MMA issuer per product. Up to 24 rows the softmax warpgroups take alternate
// stages (ALT): a stage's softmax is a chain of waits and latencies of about
// 1500 cycles, twice what a stage's bytes take; each keeps its own references,
// sums and O^T, merged at the end of a segment. More rows do not fit a thread's
// registers: there the warpgroups share the rows of every stage. Work is split
// over CTAs as in the bf16 attention (s3r_attn_sched.cuh), units shared by
// several CTAs merge by log-sum-exp in the last one to finish.
//
// What bounds it, measured: HBM for few rows in 8 bits (64 x 8192 tokens, 8 KV heads, 4
// packed rows: 6.2 TB/s, 0.94 of a copy's rate; 8: 0.86). Elsewhere instruction issue: five roles share
// every SM quadrant, about 590 instructions a stage at 4 rows and 4 bits, issued in 53%
// of cycles with instruction fetch among the first stalls (4.4 TB/s, 0.67;
// 16 x 16384 tokens 70 us a call, 285 MB). 45 rows: 256 x 8192 tokens 1278 us, 1.8 TB/s: a
// stage of the softmax warpgroups takes about 2300 cycles, 1300 of them scores and
// weights, the rest the latencies of three waits, parameters and a barrier.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "s3r_attn_common.cuh"
#include "s3r_attn_sched.cuh"
#include "s3r_device.cuh"
#include "s3r_internal.h"
#include "s3r_kvq.cuh"
#include "s3r_kvq_attn.cuh"

namespace s3r {
namespace kvq {

constexpr int kTok = 128;                    // tokens per stage
constexpr int kHidden = 0x7fffffff;
constexpr float kNuInit = 1e30f;             // -(reference) before the first score of a segment
constexpr int kSmemBudget = 232448 - 10240;  // beside the static arrays
constexpr int kMaxPend = 2;                  // units a CTA's range shares with others: its first and its last
constexpr int kThreads = 608;                // 8 softmax and 8 unpacking warps, producer, two MMA issuers
constexpr int kSoft = 256;                   // softmax threads
constexpr int kProducer = 16, kMmaQk = 17, kMmaPv = 18;

// ALT: NR rows, both warpgroups; else 2 NR rows, NR each. E4: e4m3 operands,
// two terms of a row in columns NRT apart.
template <int NR, bool ALT, int D, int BITS>
struct Lay {
  static constexpr bool E4 = BITS == 4 && ALT && NR <= 16;
  static constexpr int NRT = ALT ? NR : 2 * NR;
  static constexpr int N = ((E4 ? 2 * NRT : NRT) + 15) / 16 * 16;
  static constexpr int kTile = E4 ? 32 : 64;               // TMEM columns of 128 numbers a lane
  static constexpr int kKCols = kTile * D / 128;           // of a stage's keys
  static constexpr uint32_t kRowK = E4 ? 128 : 64;         // of k in one 128-byte row of Q and w
  static constexpr uint32_t kQBytes = N * 128 * ((D + kRowK - 1) / kRowK);   // [blocks of kRowK][N rows][128 B], two (segment parity)
  static constexpr uint32_t kPBytes = E4 ? N * kTok : kTok * 128;   // E4: [N rows][128 B of k], f16: [128 k][up to 64 rows], two (stage parity)
  static constexpr uint32_t kXBytes = ALT ? NR * 128 * 4 : 0;   // O^T of the second warpgroup, [row][channel]
  static constexpr uint32_t kStage = 2 * (kTok * D * BITS / 8) + 8 * kTok;
  static constexpr uint32_t kOffP = 2 * kQBytes;
  static constexpr uint32_t kOffX = kOffP + 2 * kPBytes;
  // TMEM columns: NB key tiles, NB value tiles, S^T[NSB], O^T[1 or 2]
  static constexpr int kO = ALT ? 2 : 1;
  static constexpr int NSB = 4 * kTile + (4 + kO) * N <= 512 ? 4 : 2;
  static constexpr int kFit = (512 - (NSB + kO) * N) / (2 * kTile);
  static constexpr int NB = kFit >= 4 ? 4 : 2;
  static constexpr int kNT = E4 ? NB : 4;                  // stages of tokens' parameters
  static constexpr int NKE = NB > NSB ? NB : NSB;          // products of keys whose completion may still be waited for
  static constexpr uint32_t kColK = 0, kColV = kTile * NB, kColS = 2 * kTile * NB, kColO = kColS + NSB * N;
  static constexpr uint32_t kOffT = kOffX + kXBytes;       // tokens' parameters: float4 [128], float2 [128] a stage
  static constexpr uint32_t kOffKV = kOffT + kNT * 128 * 24;
  static constexpr int kNSraw = (kSmemBudget - (int)kOffKV - 1024) / (int)kStage;
  static constexpr int kNS = kNSraw >= 8 ? 8 : kNSraw >= 4 ? 4 : 2;   // ring sizes are powers of two
  static constexpr uint32_t kDynBytes = kOffKV + kNS * kStage + 1024;
  // log2 of the largest weight when a row's reference is raised, and the
  // slack before it is raised again: weights stay below 256 or 2^15
  static constexpr float kTop = E4 ? 6.f : 8.f, kTau = E4 ? 2.f : 7.f;
  static_assert(kNSraw >= 2, "the ring needs two stages");
  static_assert(NB >= 2 && 2 * kTile * NB + (NSB + kO) * N <= 512, "TMEM columns");
  static_assert(E4 || kNT >= NB + 2, "parameters are written at most NB + 1 stages after the last product that used their place");
};

// D[tmem] (+)= A[tmem] * B[smem]^T, f32 accumulate: 32 of k of e4m3 or 16 of f16.
template <bool E4>
__device__ __forceinline__ void umma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (E4)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// 4 columns of this warp's lanes.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float* v) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
               :: "r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                  "r"(__float_as_uint(v[3])));
}
// Registers from the unpacking warpgroups to the softmax ones: with 608
// threads launched at 96 registers, 256 x 128 + 256 x 64 + 96 x 96 is the same total.
constexpr int kLaunchRegs = 96;
template <bool SOFTMAX>
__device__ __forceinline__ void split_registers() {
  if (SOFTMAX) asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// 32 (16) registers to this warp's TMEM lanes, as many consecutive columns.
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
__device__ __forceinline__ void tmem_st16_raw(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 1-D bulk copy global -> this CTA's shared memory with an L2 policy.
__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                               uint64_t policy) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}

// Instruction descriptor, f16 A/B (kind::f16) or e4m3 A/B (kind::f8f6f4), f32
// accumulator, A K-major, B K-major or N-major.
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t fma2(uint32_t a, float k, float c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(k), __float2half2_rn(c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The centred numbers of a word as f16 pairs. 4 bits: numbers (0, 4) (1, 5)
// (2, 6) (3, 7) of eight; 8 bits: (0, 1) (2, 3) of four. Every step is exact.
template <int BITS>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t* r) {
  if constexpr (BITS == 4) {
    constexpr uint32_t kBase = 0x64006400u;              // 1024: numbers land as 1024 + n, 1024 + 16 n
    const uint32_t v = w >> 8;
    r[0] = fma2((w & 0x000f000fu) | kBase, 1.f, -1032.f);
    r[1] = fma2((w & 0x00f000f0u) | kBase, 0.0625f, -72.f);
    r[2] = fma2((v & 0x000f000fu) | kBase, 1.f, -1032.f);
    r[3] = fma2((v & 0x00f000f0u) | kBase, 0.0625f, -72.f);
  } else {
    r[0] = fma2(__byte_perm(w, 0x64646464u, 0x4140), 1.f, -1152.f);
    r[1] = fma2(__byte_perm(w, 0x64646464u, 0x4342), 1.f, -1152.f);
  }
}

// The eight 4-bit numbers of a word as e4m3 (n 2^-9): the even ones, the odd
// ones. ALT: 15 - n for the odd ones (every other token of the values).
template <bool ALT>
__device__ __forceinline__ void unpack_e4(uint32_t w, uint32_t* r) {
  r[0] = w & 0x0f0f0f0fu;
  r[1] = ((w >> 4) ^ (ALT ? ~0u : 0u)) & 0x0f0f0f0fu;
}

// Two rows at once.
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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
// Two float16 values as e4m3 terms hi + kLo lo. A value of 9 significant bits
// is exact (hi: 4 bits, rounded to nearest; what is left: 16 steps at most)
// down to the spacing of lo, 2^-14.
constexpr float kLo = 1.f / 32;
struct Split { uint32_t hi, lo; };
__device__ __forceinline__ Split split2(uint32_t h2) {
  Split s;
  s.hi = e4m3x2_of(h2);
  uint32_t hf;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hf) : "h"((uint16_t)s.hi));
  const __half2 k = __float2half2_rn(32.f), m = __float2half2_rn(-32.f);
  const __half2 lo = __hfma2(*reinterpret_cast<const __half2*>(&hf), m, __hmul2(*reinterpret_cast<const __half2*>(&h2), k));
  s.lo = e4m3x2_of(*reinterpret_cast<const uint32_t*>(&lo));
  return s;
}
// Rounded to 9 significant bits.
__device__ __forceinline__ float2 round9(float2 x) {
  const float2 c = mul_pair(x, both(32769.f));
  const float2 d = fma_pair(x, both(-1.f), c);             // c - x
  return fma_pair(d, both(-1.f), c);
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

// Barrier over a softmax warpgroup (barriers 1 and 2).
__device__ __forceinline__ void sync_wg(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }
// Number of its threads whose predicate is true.
__device__ __forceinline__ int count_wg(int wg, bool pred) {
  int r;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.popc.u32 %0, %2, 128, p;\n\t}"
               : "=r"(r) : "r"((int)pred), "r"(1 + wg) : "memory");
  return r;
}

// A value that all lanes hold, as one the compiler knows to be uniform: role,
// loop and address arithmetic then run once a warp (without it the 8-bit
// case of 16 x 16384 tokens and 5 rows took 180 us instead of 140).
__device__ __forceinline__ uint32_t uni(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ Seg locate_uni(const KvqAttnParams& p, const int* s_prefix, int x, int hi, int W) {
  Seg s = locate(p, s_prefix, x, hi, W);
  s.b = (int)uni(s.b);
  s.h = (int)uni(s.h);
  s.k0 = (int)uni(s.k0);
  s.npg = (int)uni(s.npg);
  s.end = (int)uni(s.end);
  s.unit = (int)uni(s.unit);
  s.first_cta = (int)uni(s.first_cta);
  s.nseg = (int)uni(s.nseg);
  return s;
}
// Stages of a CTA's range in order: g of all, j of the nst of segment s.
struct Walk {
  Seg sg;
  int s, j, nst;
  uint32_t g;
  bool valid;
};
__device__ __forceinline__ Walk walk_begin(const KvqAttnParams& p, const int* s_prefix, int lo, int hi, int W, int ppt) {
  Walk w;
  w.s = w.j = 0;
  w.g = 0u;
  w.valid = lo < hi;
  w.sg = locate_uni(p, s_prefix, lo, hi, W);
  w.nst = (w.sg.npg + ppt - 1) / ppt;
  return w;
}
__device__ __forceinline__ void walk_next(const KvqAttnParams& p, const int* s_prefix, int hi, int W, int ppt, Walk& w) {
  ++w.g;
  if (++w.j < w.nst) return;
  w.j = 0;
  ++w.s;
  w.valid = w.sg.end < hi;
  if (w.valid) {
    w.sg = locate_uni(p, s_prefix, w.sg.end, hi, W);
    w.nst = (w.sg.npg + ppt - 1) / ppt;
  }
}

// Whether one of the D numbers of a page's token t is not 0 (v: the page's V
// pieces of `unit` bytes, in shared memory).
template <int D, int BITS>
__device__ __forceinline__ bool any_number(const uint8_t* v, int t, int unit) {
  const int at = t * BITS / 8;
  const uint8_t* const word = v + at / unit * (D * unit) + (at % unit & ~3);
  const uint32_t mask = ((1u << BITS) - 1u) << (t * BITS & 31);
  uint32_t any = 0u;
#pragma unroll 1
  for (int d = 0; d < D && (any & mask) == 0u; d += 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= *reinterpret_cast<const uint32_t*>(word + (d + i) * unit);
  }
  return (any & mask) != 0u;
}

// Listed pages are all walked, -1 entries among them.
__device__ __forceinline__ int unit_pages(const KvqAttnParams& p, int L) {
  if (kvq_bad_context(p, L)) return 0;
  return p.page_list ? p.budget : (L + p.P - 1) / p.P;
}

template <int NR, bool ALT, int D, int P, int BITS>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const KvqAttnParams p) {
  using L = Lay<NR, ALT, D, BITS>;
  constexpr KvqLayout Y = kvq_layout(D, P, BITS);
  constexpr int kUnit = Y.unit;                          // bytes of a V piece
  constexpr int NRT = L::NRT, N = L::N, NB = L::NB, NS = L::kNS, NSB = L::NSB, NKE = L::NKE, kNT = L::kNT;
  constexpr int ppt = kTok / P;                          // pages per stage
  constexpr bool E4 = L::E4;
  constexpr float kTop = L::kTop, kTau = L::kTau;
  constexpr float kMid = E4 ? 0.f : BITS == 4 ? 8.f : 128.f;   // subtracted from the numbers
  static_assert(ppt * Y.page_bytes == (int)L::kStage, "stage bytes");
  extern __shared__ __align__(1024) uint8_t dyn_raw[];
  uint8_t* dyn = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t s_bar[2 * NS + 3 * NB + NKE + kNT + NSB + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int4 s_pend[kMaxPend];                      // units this CTA merges at its end: (b, h, slot0, nseg)
  __shared__ int s_npend;
  __shared__ int s_prefix[kMaxSeqs + 1];
  __shared__ int s_stage_lp[NS][8];
  __shared__ int s_roff[64];                             // output row of packed row i relative to (b, h)
  // per warpgroup (ALT: both hold the same rows, else rows wg * NR ..)
  __shared__ float s_red[8][32];
  __shared__ float s_red2[8][32];
  __shared__ __align__(16) float s_nu[2][32];            // -(reference) per row, log2 units
  __shared__ __align__(16) float s_alpha[2][32];         // rescale factor per row
  __shared__ __align__(16) float s_sum[2][32];           // sum of p per row, then 1 / the merged sum
  // ALT, handed over by the second warpgroup: reference and sum; then both
  // parts' factors (-1: a part without tokens)
  __shared__ float s_xm[32], s_xl[32], s_f0[32], s_f1[32];
  __shared__ __align__(16) float s_corr[2][32];          // sum of w (z / s + c) per row
  __shared__ __align__(16) float s_qs[2][64];            // by segment parity: 2^-16 of the sum of a query row
  __shared__ __align__(16) float s_qf[2][64];            // 2^-16 / the query row's scale

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = (int)uni((uint32_t)tid >> 5);
  pdl_launch_dependents();
  if (tid < 64) s_roff[tid] = (tid / p.G) * p.Hq + (tid % p.G);
  const uint32_t bar0 = smem_addr(&s_bar[0]);
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  // KF / VF: a stage's keys / values are unpacked in TMEM; TF: its token
  // parameters are in shared memory; KE / VE: its product of keys / values is
  // done (S^T / O^T has its part, the tile is free); PF: w(g) is written (and
  // S^T(g) and the parameters read). Stage g uses barrier g % size of each
  // ring, and each ring is as long as the stages between a completion and its
  // last waiter, so that none is two phases ahead of a wait.
  constexpr int B_FULL = 0, B_EMPTY = NS, B_KF = 2 * NS, B_VF = B_KF + NB, B_TF = B_VF + NB, B_KE = B_TF + kNT, B_VE = B_KE + NKE,
                B_PF = B_VE + NB, B_QF = B_PF + NSB, B_TD = B_QF + 1, B_X = B_TD + 1, B_Y = B_X + 1;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(BAR(B_FULL + i), 1);
      mbar_init(BAR(B_EMPTY + i), E4 ? 4 : 8);           // the warps that unpack the stage
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(BAR(B_KF + i), 4);
      mbar_init(BAR(B_VF + i), 4);
      mbar_init(BAR(B_VE + i), 1);
    }
    for (int i = 0; i < NKE; ++i) mbar_init(BAR(B_KE + i), 1);
    for (int i = 0; i < kNT; ++i) mbar_init(BAR(B_TF + i), 4);
    for (int i = 0; i < NSB; ++i) mbar_init(BAR(B_PF + i), ALT ? 4 : 8);
    mbar_init(BAR(B_QF), 8);
    mbar_init(BAR(B_TD), 2);
    mbar_init(BAR(B_X), 4);
    mbar_init(BAR(B_Y), 4);
    s_abort = 0;
    s_npend = 0;
    fence_barrier_init();
  }
  // Everything below may have been written by the kernel before this one: a row
  // just stored, a length just moved. That a writer lets this kernel launch only
  // when it is done does not make its writes visible here; the wait does.
  pdl_wait();
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
  __syncthreads();
  // sequences without pages have an unusable length
  bool none = false;
  if (blockIdx.x == 0)
    for (int b = tid; b < p.S; b += kThreads) none |= s_prefix[b] == s_prefix[b + 1];
  if (blockIdx.x == 0 && __syncthreads_or(none)) {
    for (int b = 0; b < p.S; ++b) {
      if (s_prefix[b] != s_prefix[b + 1]) continue;
      if (tid == 0) flag_status(p.status, S3R_DEV_BAD_CONTEXT_LEN);
      for (int h = 0; h < p.Hkv; ++h) kvq_write_empty<__nv_bfloat16>(p, b, h, tid, kThreads);
    }
  }
  const int total = (int)uni((uint32_t)s_prefix[p.S]);
  // at least one stage of pages per CTA (shorter pieces would cost a merge
  // for less than a stage); with lists, a whole unit per CTA where the units
  // nearly fill the grid, so that none is split (a call of 120 units of 64 pages
  // takes 24 us against 29 split, 128 of 32 pages 17 against 22, 144 of 64 pages 25 against 31)
  int W = max((total + (int)gridDim.x - 1) / (int)gridDim.x, ppt);
  if (p.page_list && W < p.budget && p.S * p.Hkv * 5 >= (int)gridDim.x * 4) W = p.budget;
  const int lo = blockIdx.x * W, hi = min(total, lo + W);
  if (lo >= hi) return;                                  // uniform over the CTA

  uint8_t* sQ = dyn;
  uint8_t* sP = dyn + L::kOffP;
  uint8_t* sKV = dyn + L::kOffKV;
  const uint32_t aQ = smem_addr(sQ), aP = smem_addr(sP), aKV = smem_addr(sKV);

  if (warp == kMmaQk) {
    tmem_alloc(smem_addr(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uni(s_tmem);

  if (warp == kProducer) {
    // ======================================================= producer warp
    const uint64_t pol = l2_policy_evict_first();
    // Pages in batches of 32 of one segment, a lane each: the lane that looked
    // a page up copies it, and the next batch's ids are in flight meanwhile.
    auto look_up = [&](const Seg& s, int k, int* lp, int* ph) {
      *lp = *ph = -1;
      if (k + lane >= s.npg) return;
      *lp = p.page_list ? p.page_list[(size_t)s.unit * p.budget + s.k0 + k + lane] : s.k0 + k + lane;
      bool there = *lp >= 0;
      if (p.page_list) there = there && *lp < (p.context_lens[s.b] + P - 1) / P;
      if (there) *ph = p.block_table[(size_t)s.b * p.max_pages + *lp];
    };
    bool ok = true, more = true;
    uint32_t g = 0;
    int k = 0, lp, ph;
    Seg sg = locate_uni(p, s_prefix, lo, hi, W);
    look_up(sg, 0, &lp, &ph);
    while (more && ok) {
      Seg nx = sg;
      int nk = k + 32, nlp = -1, nph = -1;
      if (nk >= sg.npg) {
        nk = 0;
        more = sg.end < hi;
        if (more) nx = locate_uni(p, s_prefix, sg.end, hi, W);
      }
      if (more) look_up(nx, nk, &nlp, &nph);
      if (lp != -1 && (ph < 0 || ph >= p.num_pages_total)) {
        flag_status(p.status, S3R_DEV_BAD_PAGE_ID);
        ph = -1;
      }
      const unsigned real = __ballot_sync(0xffffffffu, ph >= 0);
      const int stages = (min(32, sg.npg - k) + ppt - 1) / ppt;
      const uint8_t* const src = p.pages + ((size_t)max(ph, 0) * p.Hkv + sg.h) * Y.page_bytes;
      for (int j = 0; j < stages; ++j, ++g) {
        const uint32_t st = g % NS;
        if (!__all_sync(0xffffffffu, mbar_wait(BAR(B_EMPTY + st), ((g / NS) & 1) ^ 1, &s_abort, p.status))) {
          ok = false;
          break;
        }
        const bool here = lane / ppt == j;
        if (here) s_stage_lp[st][lane % ppt] = ph >= 0 ? lp : -1;
        __syncwarp();
        if (lane == 0)
          mbar_arrive_expect_tx(BAR(B_FULL + st), (uint32_t)__popc((real >> (j * ppt)) & ((1u << ppt) - 1u)) * Y.page_bytes);
        __syncwarp();
        if (here && ph >= 0)
          bulk_load_hint(aKV + st * L::kStage + (lane % ppt) * Y.page_bytes, src, Y.page_bytes, BAR(B_FULL + st), pol);
      }
      sg = nx;
      k = nk;
      lp = nlp;
      ph = nph;
    }
    // drain: wait until every issued copy has landed
    if (lane == 0)
      for (uint32_t k = g > NS ? g - NS : 0; k < g; ++k) mbar_wait_drain(BAR(B_FULL + k % NS), (k / NS) & 1, p.status);
  } else if (warp >= kMmaQk) {
    // ======================================================= MMA issuers
    // One warp for each product, in stage order. The whole warp runs the loop
    // on values made uniform by shuffles and one elected lane issues: an MMA
    // then costs 10 cycles to issue instead of 46 from a lane's own branch
    // (N = 16, measured), and a commit about 80 - there is one per tile, which
    // both the unpacking warps (tile free) and the softmax (product done) wait on.
    // QK(g) needs its stage unpacked, w(g - NSB) written (S^T buffer g % NSB has been read)
    // and first in a segment the segment's Q; PV(g) needs w(g).
    constexpr uint32_t idQk = idesc_f32(128, N, false), idPv = idesc_f32(128, N, !E4);
    // Q (and w of E4): K-major, 128-byte rows, 8-row groups 1024 B apart; a
    // step of k is 32 bytes inside the swizzle row, the next row N x 128 B
    // further. w in f16: rows along the 128 bytes, a step of k 16 tokens, 2048
    // B. A tile's step is 8 TMEM columns.
    const uint64_t dB0 = smem_desc_sw128(warp == kMmaQk ? aQ : aP, 16, 1024);
    constexpr uint32_t kBlock = (N * 128) >> 4;
    for (Walk c = walk_begin(p, s_prefix, lo, hi, W, ppt); c.valid; walk_next(p, s_prefix, hi, W, ppt, c)) {
      const uint32_t buf = c.g % NB;
      if (warp == kMmaQk) {
        bool ok = mbar_wait(BAR(B_KF + buf), (c.g / NB) & 1, &s_abort, p.status);
        if (c.g >= NSB) ok = ok && mbar_wait(BAR(B_PF + c.g % NSB), (c.g / NSB - 1) & 1, &s_abort, p.status);
        if (c.j == 0) ok = ok && mbar_wait(BAR(B_QF), c.s & 1, &s_abort, p.status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t d = uni(tmem + L::kColS + c.g % NSB * N), a = uni(tmem + L::kColK + buf * L::kTile);
        const uint32_t bar = uni(BAR(B_KE + c.g % NKE)), step = uni((c.s & 1) * (L::kQBytes >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < L::kKCols / 8; ++kk)
            umma_ta<E4>(d, a + kk * 8, dB0 + step + (kk >> 2) * kBlock + (kk & 3) * 2, idQk, kk > 0 ? 1u : 0u);
          umma_commit(bar);
        }
      } else {
        bool ok = mbar_wait(BAR(B_VF + buf), (c.g / NB) & 1, &s_abort, p.status);
        ok = ok && mbar_wait(BAR(B_PF + c.g % NSB), (c.g / NSB) & 1, &s_abort, p.status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const uint32_t d = uni(tmem + L::kColO + (ALT ? (c.g & 1) * N : 0)), a = uni(tmem + L::kColV + buf * L::kTile);
        const uint32_t first = uni(c.j >= (ALT ? 2 : 1) ? 1u : 0u), bar = uni(BAR(B_VE + buf));
        const uint32_t step = uni((c.g & 1) * (L::kPBytes >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < L::kTile / 8; ++kk)
            umma_ta<E4>(d, a + kk * 8, dB0 + step + kk * (E4 ? 2 : 2048 >> 4), idPv, kk > 0 ? 1u : first);
          umma_commit(bar);
        }
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(BAR(B_TD));
    __syncwarp();
  } else if (warp >= 8) {
    // ======================================================= unpacking warps
    // E4: the warpgroups take alternate stages, keys and values, so that a
    // warpgroup's chain of waits, loads and stores spans two stages; the tiles
    // and parameters of stage g - NB are free once its product of values is
    // done. Else (two tiles in TMEM): one takes the keys, one the values and
    // parameters, so that keys run ahead of the softmax (5 rows of 16 x 16384
    // tokens in 8 bits: 146 us, alternating 160).
    split_registers<false>();
    const int uwg = (warp - 8) >> 2;
    const int t = tid & 127;                             // TMEM lane: token of S^T, channel of O^T
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
    constexpr int kWordsPage = P * BITS / 32;            // words of a channel in one page: 2, 4, 8 or 16
    int Lb = -1, of = -1;                                // length of sequence `of`
    // Words of a row (16-byte reads) to columns of this lane, 16 columns (8 bits:
    // 32) a turn of a rolled loop: five roles run on every SM quadrant at once and
    // instruction fetch, not arithmetic, bounds them (unrolled, 48 rows of 4-bit
    // tokens took 1800 ns a stage instead of 1590).
    auto unpack_columns = [&](auto values, auto cols, auto words, uint32_t dst) {
      constexpr int kCols = decltype(cols)::value, kTurn = BITS == 8 && kCols >= 32 ? 32 : 16;
      constexpr int kWords = (E4 ? 8 : BITS) * kTurn / 16;   // words of a turn
#pragma unroll 1
      for (int c = 0; c < kCols / kTurn; ++c) {
        uint32_t r[kTurn];
#pragma unroll
        for (int k = 0; k < kWords; k += 4) {
          const uint4 w = words(c * kWords + k);
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (E4) unpack_e4<decltype(values)::value>(v[i], r + 2 * (k + i));
            else unpack<BITS>(v[i], r + (k + i) * (16 / BITS));
          }
        }
        if constexpr (kTurn == 32) tmem_st32_raw(dst + c * 32, r);
        else tmem_st16_raw(dst + c * 16, r);
      }
    };
    for (Walk c = walk_begin(p, s_prefix, lo, hi, W, ppt); c.valid; walk_next(p, s_prefix, hi, W, ppt, c)) {
      const uint32_t g = c.g, st = g % NS, buf = g % NB;
      if (E4 && (g & 1u) != (uint32_t)uwg) continue;
      if (of != c.sg.b) {
        of = c.sg.b;
        Lb = p.context_lens[of];
      }
      bool ok = mbar_wait(BAR(B_FULL + st), (g / NS) & 1, &s_abort, p.status);
      const uint8_t* const stage = sKV + st * L::kStage;
      // the token's parameters for the softmax: y = ka S^T + kb sum q (scaled),
      // log2 s_v, 1 / s_v, the centre of its values over s_v, and its position
      // against the rows' (hidden from rows before `excess`; from all: kHidden)
      auto token_parameters = [&]() {
        const uint8_t* pg = stage + (t / P) * Y.page_bytes;
        const uint32_t kp = *reinterpret_cast<const uint32_t*>(pg + Y.off_kp + (t % P) * 4);
        const uint32_t vp = *reinterpret_cast<const uint32_t*>(pg + Y.off_vp + (t % P) * 4);
        const int lp = s_stage_lp[st][t / P];
        const int pos = lp * P + (t % P);
        const bool valid = lp >= 0 && pos < Lb;
        const float sk = __uint_as_float(kp << 16), zk = __uint_as_float(kp & 0xffff0000u);
        const float sv = valid ? __uint_as_float(vp << 16) : 1.f;
        const float zv = valid ? __uint_as_float(vp & 0xffff0000u) : 0.f;
        float4* const at4 = reinterpret_cast<float4*>(dyn + L::kOffT + (g % kNT) * (128 * 24));
        float2* const at2 = reinterpret_cast<float2*>(at4 + 128);
        auto put = [&](float step) {
          const float r = __fdividef(1.f, step);
          at4[t] = make_float4(p.scale_log2 * sk, p.scale_log2 * fmaf(kMid, sk, zk), __log2f(step), r);
          // 4 bits as e4m3: every other token holds 15 - n and meets -w
          at2[t] = make_float2(fmaf(zv, r, E4 ? (t & 1 ? 15.f : 0.f) : kMid),
                               __int_as_float(valid ? pos - (Lb - p.R) - p.r0 : kHidden));
        };
        put(sv);
        // A row of equal values is held with s = 1, which says nothing of its
        // size: taken as a step it would set the reference of rows a thousand
        // times smaller and leave their weights no bits. It has no numbers for a
        // weight to meet, so any step serves; one of about 2^-8 |z| keeps it
        // among its likes (2^-80: a row of zeros stays out of the way, and its
        // weights in float32's range). Its numbers tell it from a row whose step is 1.
        // The token's number is hidden from the compiler there, so that the addresses
        // stay in the rare path (hoisted, 64 x 8192 tokens of 8 bits with one row took
        // 210 us instead of 198). A cache of equal rows only pays for the search: 16 x 16384
        // tokens of zeros take 152 us back to back, others 66.
        // A key of equal values scores scale z sum q: its centred numbers, -c s sum q, would
        // cancel against c s sum q in float32 only, with s = 1 far above keys of small steps.
        if (valid && (sv == 1.f || (kMid != 0.f && sk == 1.f))) {
          uint32_t u = (uint32_t)t;
          asm volatile("" : "+r"(u));
          const uint8_t* const its = stage + u / P * Y.page_bytes;
          if (sv == 1.f && !any_number<D, BITS>(its + Y.off_v, (int)(u % P), Y.unit))
            put(__uint_as_float((uint32_t)max((int)(vp >> 23 & 0xffu) - 8, 47) << 23));
          if (kMid != 0.f && sk == 1.f) {
            uint32_t any = 0u;
#pragma unroll 1
            for (uint32_t c = 0; c < D * BITS / 128; ++c) {
              const uint4 w = *reinterpret_cast<const uint4*>(its + (c * P + u % P) * 16);
              any |= w.x | w.y | w.z | w.w;
            }
            if (any == 0u) reinterpret_cast<float2*>(at4 + t)[0] = make_float2(0.f, p.scale_log2 * zk);
          }
        }
      };
      if (!E4 && uwg == 1) {
        // ahead of the values: the softmax needs them with S^T
        token_parameters();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_TF + g % kNT));
      }
      if (g >= NB) {
        const uint32_t x = g - NB;
        ok = ok && (E4 || uwg == 1 ? mbar_wait(BAR(B_VE + buf), (x / NB) & 1, &s_abort, p.status)
                                   : mbar_wait(BAR(B_KE + x % NKE), (x / NKE) & 1, &s_abort, p.status));
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (E4 || uwg == 0) {
        const uint32_t dst = tmem + lane_base + L::kColK + buf * L::kTile;
        const uint8_t* const row = stage + (t / P) * Y.page_bytes + (t % P) * 16;
        auto words = [&](int k) { return *reinterpret_cast<const uint4*>(row + (k / 4) * (P * 16)); };
        unpack_columns(std::false_type{}, std::integral_constant<int, L::kKCols>{}, words, dst);
      }
      if ((E4 || uwg == 1) && (D == 128 || t < D)) {     // whole warps; lanes past D hold anything and are never read
        const uint32_t dst = tmem + lane_base + L::kColV + buf * L::kTile;
        auto words = [&](int k) {
          const int pg = k / kWordsPage;
          if constexpr (kUnit == 16)
            return *reinterpret_cast<const uint4*>(stage + pg * Y.page_bytes + Y.off_v + (k % kWordsPage / 4 * D + t) * 16);
          const uint2 v0 = *reinterpret_cast<const uint2*>(stage + pg * Y.page_bytes + Y.off_v + t * 8);   // two pages of two words
          const uint2 v1 = *reinterpret_cast<const uint2*>(stage + (pg + 1) * Y.page_bytes + Y.off_v + t * 8);
          return make_uint4(v0.x, v0.y, v1.x, v1.y);
        };
        unpack_columns(std::true_type{}, std::integral_constant<int, L::kTile>{}, words, dst);
      }
      if constexpr (E4) token_parameters();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (E4 || uwg == 0) mbar_arrive(BAR(B_KF + buf));
        if (E4) mbar_arrive(BAR(B_TF + g % kNT));
        if (E4 || uwg == 1) mbar_arrive(BAR(B_VF + buf));
        mbar_arrive(BAR(B_EMPTY + st));
      }
    }
  } else {
    // ======================================================= softmax warps
    split_registers<true>();
    const int wg = warp >> 2, q4 = warp & 3, t = tid & 127;   // token of the stage; channel in the epilogue
    const int rb = ALT ? 0 : wg * NR;                    // first row
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
    // A segment's Q as q 2^e in f16 (or two e4m3 terms) in the order of the unpacked numbers, 2^e
    // the row's power-of-two scale; the sum of each row. Both warpgroups.
    auto q_store = [&](const Seg& s, int par) {
      uint8_t* const dst = sQ + par * L::kQBytes;
#pragma unroll
      for (int k = 0; k < kQC; ++k) {
        const int ch = tid + kSoft * k, r = ch / kDc, c8 = ch % kDc;
        if (NRT * kDc % kSoft != 0 && r >= NRT) break;   // uniform over a warp (NRT kDc is a multiple of 32)
        const uint4 qv = r < p.rows ? __ldg(reinterpret_cast<const uint4*>(q_at(s, ch))) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {qv.x, qv.y, qv.z, qv.w};
        float x[8], sum = 0.f, big = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(w[i] << 16);
          x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          big = fmaxf(big, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
        }
#pragma unroll
        for (int o = kDc / 2; o >= 1; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        // largest value into [128, 256), for values from 2^-103 to the type's
        // largest (smaller ones keep fewer bits); 2^-16 / up and the token's 2^16
        // scale stay in float32's range
        const int ex = max((int)(__float_as_uint(big) >> 23), 24);
        const float up = __uint_as_float((uint32_t)(254 - ex + 7) << 23);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          x[i] *= up;
          x[i + 1] *= up;
          sum += x[i] + x[i + 1];
        }
#pragma unroll
        for (int o = kDc / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (c8 == 0) {
          const float back = 0x1p-16f / up;
          // an infinite channel reaches every score as NaN: e4m3 would hold it as 448
          s_qs[par][r] = big < INFINITY ? sum * back : __int_as_float(0x7fc00000);
          s_qf[par][r] = (E4 ? 512.f : 1.f) * back;
        }
        if constexpr (E4) {
          // 8 bytes at k = 8 c8: channels 0 2 4 6 1 3 5 7; hi and lo rows may differ in r & 7
          const Split a = split2(half2_of(x[0], x[2])), b = split2(half2_of(x[4], x[6]));
          const Split c = split2(half2_of(x[1], x[3])), d = split2(half2_of(x[5], x[7]));
          const int place = (c8 >> 1) << 4, sub = (c8 & 1) * 8;
          *reinterpret_cast<uint2*>(dst + r * 128 + (place ^ ((r & 7) << 4)) + sub) = make_uint2(a.hi | b.hi << 16, c.hi | d.hi << 16);
          *reinterpret_cast<uint2*>(dst + (NRT + r) * 128 + (place ^ (((NRT + r) & 7) << 4)) + sub) =
              make_uint2(a.lo | b.lo << 16, c.lo | d.lo << 16);
        } else {
          const uint4 v = BITS == 4 ? make_uint4(half2_of(x[0], x[4]), half2_of(x[1], x[5]), half2_of(x[2], x[6]), half2_of(x[3], x[7]))
                                    : make_uint4(half2_of(x[0], x[1]), half2_of(x[2], x[3]), half2_of(x[4], x[5]), half2_of(x[6], x[7]));
          *reinterpret_cast<uint4*>(dst + (c8 >> 3) * (N * 128) + r * 128 + (((c8 & 7) ^ (r & 7)) << 4)) = v;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(B_QF));
    };
    // where this thread's weights go: its token's place along k
    const int kpos = E4 ? (t & ~7) + ((t & 1) << 2) + ((t & 7) >> 1) : BITS == 4 ? (t & ~7) + ((t & 3) << 1) + ((t >> 2) & 1) : t;
    uint8_t* const pw = E4 ? sP + (kpos & 15) : sP + kpos * 128;
    const int pck = E4 ? kpos >> 4 : kpos & 7;
    const uint32_t sign = E4 && (t & 1) ? 0x80008000u : 0u;   // every other token's weights are negated
    // E4: weights below 2^-14 of the row's scale would all round to 0 (or all
    // up), and 2^19 positions of 2^-21 of the largest are a quarter of it (such a
    // row was off by 4.8%). So a weight is rounded after a token's own offset, 128 offsets
    // spread evenly over a step of 2^-14, turned with the stage; t keeps its parity
    // in them, since the numbers of odd tokens are complemented. A hidden weight of 0 stays 0.
    auto offset_at = [&](uint32_t g) { return ((float)((uint32_t)(t * 79) + g * 54u & 127u) - 63.5f) * 0x1p-21f; };

    // barriers of a stage's products: S^T(x) complete; O^T with x's part complete
    auto s_done = [&](uint32_t x) { return mbar_wait(BAR(B_KE + x % NKE), (x / NKE) & 1, &s_abort, p.status); };
    auto o_done = [&](uint32_t x) { return mbar_wait(BAR(B_VE + x % NB), (x / NB) & 1, &s_abort, p.status); };
    constexpr int C = NR <= 8 ? NR : 8;                  // rows read from TMEM at once
    auto tm_load = [&](uint32_t at, float* x) {
      if constexpr (C == 4) tmem_ld4(at, x);
      else tmem_ld8(at, x);
      tmem_wait_ld();
    };
    auto tm_store = [&](uint32_t at, const float* x) {
      if constexpr (C == 4) tmem_st4(at, x);
      else tmem_st8(at, x);
    };
    Seg sg = locate_uni(p, s_prefix, lo, hi, W);
    q_store(sg, 0);
    uint32_t g = 0;
    int seg = 0;
    bool ok = true;
    for (int x = lo; x < hi; ++seg) {
      const int par = seg & 1;
      const bool has_next = sg.end < hi;
      Seg nx = sg;
      if (has_next) {
        nx = locate_uni(p, s_prefix, sg.end, hi, W);
        q_prefetch(nx);
      }
      const int nst = (sg.npg + ppt - 1) / ppt;
      if (t < NR) s_nu[wg][t] = kNuInit;
      float l[NR], corr[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) l[r] = corr[r] = 0.f;
      // the segment's Q sums are read after this barrier and a wait on QF: both warpgroups have stored theirs
      sync_wg(wg);
      ok &= mbar_wait(BAR(B_QF), par, &s_abort, p.status);
      bool abort_all = false;
      int mine = -1;                                     // this warpgroup's last stage of the segment
      const uint32_t g0 = g;
      for (; g < g0 + nst; ++g) {
        if (ALT && (int)(g & 1) != wg) continue;
        const uint32_t sb = g & 1;
        // The products' barriers are asked early, so that the answers' latency
        // passes under other work: with shared rows both before the parameters (48
        // rows: 1575 -> 1520 ns a stage); with alternate stages only PV(g - 2)'s, and
        // later, when it is likely done (8 rows 706 -> 685, at the top 718).
        auto o_test = [&]() { return g < 2 || mbar_test_wait(BAR(B_VE + (g - 2) % NB), ((g - 2) / NB) & 1); };
        bool s_early = false, o_early = false;
        if (!ALT) {
          s_early = mbar_test_wait(BAR(B_KE + g % NKE), (g / NKE) & 1);
          o_early = o_test();
        }
        ok &= mbar_wait(BAR(B_TF + g % kNT), (g / kNT) & 1, &s_abort, p.status);
        const uint8_t* const tp = dyn + L::kOffT + (g % kNT) * (128 * 24);
        const float4 ta = reinterpret_cast<const float4*>(tp)[t];
        const float2 tb = reinterpret_cast<const float2*>(tp + 128 * 16)[t];
        const float ka = ta.x, kb = ta.y;
        float lgs = ta.z, rsv = ta.w, zc = tb.x;
        const int excess = __float_as_int(tb.y);
        uint32_t hide = 0u;
        if (excess > 0) {
          const int nm = p.G * excess - rb;
          hide = excess == kHidden || nm >= 32 ? ~0u : nm <= 0 ? 0u : (1u << nm) - 1u;
        }
        if (!(fabsf(zc) + rsv < INFINITY)) {             // a NaN row of values: the rows that see it, and only they
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (!((hide >> r) & 1u)) corr[r] = __int_as_float(0x7fc00000);
          lgs = zc = 0.f;
          rsv = 1.f;
        }
        if (ALT) o_early = o_test();
        if (!s_early) ok &= s_done(g);
        tc_fence_after();
        float s[NR];
        // s <- y + log2 s_v (- reference); hidden: -inf. The reference comes off the
        // rounded sum, which is what it was raised from: taken off inside it, scores of
        // 1e8 left weights beyond a float16 (infinite outputs) or none.
        auto load_s = [&](bool with_ref) {
          const uint32_t at = tmem + lane_base + L::kColS + g % NSB * N + rb;
          if constexpr (E4) {
            float lo[NR];
            if constexpr (NR == 4) {
              tmem_ld4(at, s);
              tmem_ld4(at + NRT, lo);
            } else {
              tmem_ld_cols<NR>(at, s);
              tmem_ld_cols<NR>(at + NRT, lo);
            }
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < NR; r += 2) {
              const float2 v = fma_pair(make_float2(lo[r], lo[r + 1]), both(kLo), make_float2(s[r], s[r + 1]));
              s[r] = v.x;
              s[r + 1] = v.y;
            }
          } else {
            if constexpr (NR == 4) tmem_ld4(at, s);
            else tmem_ld_cols<NR>(at, s);
            tmem_wait_ld();
          }
#pragma unroll
          for (int r = 0; r < NR; r += 4) {
            const float4 qs = *reinterpret_cast<const float4*>(&s_qs[par][rb + r]);
            const float4 qf = *reinterpret_cast<const float4*>(&s_qf[par][rb + r]);
            float4 nu = make_float4(0.f, 0.f, 0.f, 0.f);
            if (with_ref) nu = *reinterpret_cast<const float4*>(&s_nu[wg][r]);
            auto y = [&](float2 x, float2 f, float2 q, float2 n) {
              return fma_pair(fma_pair(mul_pair(x, f), both(ka), fma_pair(q, both(kb), both(lgs))), both(1.f), n);
            };
            const float2 a = y(make_float2(s[r], s[r + 1]), make_float2(qf.x, qf.y), make_float2(qs.x, qs.y), make_float2(nu.x, nu.y));
            const float2 b = y(make_float2(s[r + 2], s[r + 3]), make_float2(qf.z, qf.w), make_float2(qs.z, qs.w),
                               make_float2(nu.z, nu.w));
            s[r] = a.x;
            s[r + 1] = a.y;
            s[r + 2] = b.x;
            s[r + 3] = b.y;
          }
          if (hide) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
              if ((hide >> r) & 1u) s[r] = -INFINITY;
          }
        };
        load_s(true);
        float ymax = fmaxf(s[0], s[1]);
#pragma unroll
        for (int r = 2; r < NR; r += 2) ymax = max3(ymax, s[r], s[r + 1]);
        // one barrier per stage: stop together, or raise the references together
        const int cnt = count_wg(wg, !ok || ymax > kTop + kTau);
        bool rescale_o = false;
        if (cnt > 0) {
          if (count_wg(wg, !ok) > 0) { abort_all = true; break; }
          // stage maximum per row (S^T is intact until PF), then reload
          load_s(false);
          warp_part<NR, true>(s, &s_red[4 * wg], q4, lane);
          sync_wg(wg);
          if (t < NR) {
            const float mx = fmaxf(fmaxf(s_red[4 * wg][t], s_red[4 * wg + 1][t]),
                                   fmaxf(s_red[4 * wg + 2][t], s_red[4 * wg + 3][t]));
            const float m_old = -s_nu[wg][t];
            const float m_new = fmaxf(m_old, __fsub_ru(mx, kTop));   // the largest weight is at most 2^kTop
            s_alpha[wg][t] = ex2(m_old - m_new);
            s_nu[wg][t] = -m_new;
          }
          sync_wg(wg);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float a = s_alpha[wg][r];
            l[r] *= a;
            corr[r] *= a;
          }
          load_s(true);
          rescale_o = mine >= 0;
        }
        // w buffer sb was last read by PV(g - 2); a rescale of O^T also needs
        // its last PV done (ALT: the same)
        const uint32_t back = !ALT && rescale_o ? 1 : 2;
        if (back == 1 ? g >= 1 : !o_early) ok &= o_done(g - back);
        tc_fence_after();
        if (rescale_o) {
#pragma unroll
          for (int c = 0; c < (E4 ? 2 * NR : NR); c += C) {   // E4: the lo columns too
            const uint32_t at = tmem + lane_base + L::kColO + (ALT ? wg * N : rb) + c;
            float o[C];
            tm_load(at, o);
#pragma unroll
            for (int r = 0; r < C; ++r) o[r] *= s_alpha[wg][(c + r) % NR];
            tm_store(at, o);
          }
          tmem_wait_st();
        }
        uint8_t* const pb = pw + sb * L::kPBytes;
        const float offset = E4 ? offset_at(g) : 0.f;
        uint32_t h[NR / 2];
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          float2 w = make_float2(ex2(s[r]), ex2(s[r + 1]));
          const float2 ln = fma_pair(w, both(rsv), make_float2(l[r], l[r + 1]));
          l[r] = ln.x;
          l[r + 1] = ln.y;
          if constexpr (E4) w = round9(w);               // the numbers' and the minima's sums meet one rounded weight (small ones in the mean)
          const float2 cn = fma_pair(w, both(zc), make_float2(corr[r], corr[r + 1]));
          corr[r] = cn.x;
          corr[r + 1] = cn.y;
          if constexpr (E4) w = fma_pair(w, both(1.f), both(offset));
          h[r / 2] = half2_of(w.x, w.y);
          if constexpr (E4) {
            const Split sp = split2(h[r / 2] ^ sign);
            pb[r * 128 + ((pck ^ (r & 7)) << 4)] = (uint8_t)sp.hi;
            pb[(r + 1) * 128 + ((pck ^ ((r + 1) & 7)) << 4)] = (uint8_t)(sp.hi >> 8);
            pb[(NRT + r) * 128 + ((pck ^ ((NRT + r) & 7)) << 4)] = (uint8_t)sp.lo;
            pb[(NRT + r + 1) * 128 + ((pck ^ ((NRT + r + 1) & 7)) << 4)] = (uint8_t)(sp.lo >> 8);
          }
        }
        if constexpr (!E4) {
          // eight rows of this token are 16 bytes of its row of k
          if constexpr (NR == 4) {
            *reinterpret_cast<uint2*>(pb + (pck << 4)) = make_uint2(h[0], h[1]);
          } else {
#pragma unroll
            for (int r = 0; r < NR; r += 8)
              *reinterpret_cast<uint4*>(pb + (((rb + r) / 8 ^ pck) << 4)) = make_uint4(h[r / 2], h[r / 2 + 1], h[r / 2 + 2], h[r / 2 + 3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_PF + g % NSB));
        mine = (int)g;
      }
      if (abort_all) break;
      // ---- the next segment's Q goes to the other buffer: the products of
      // the segment before this one are done (this warpgroup has waited for a
      // later one, or for its last), and its sums have been read by the other
      // warpgroup (which has met this one at that segment's end, here or below)
      if (wg == 1 && seg > 0) ok &= mbar_wait(BAR(B_Y), (seg - 1) & 1, &s_abort, p.status);
      if (has_next) q_store(nx, par ^ 1);
      // ---- segment epilogue: row sums, then (O^T + corr) / l
      warp_part<NR, false>(l, &s_red[4 * wg], q4, lane);
      warp_part<NR, false>(corr, &s_red2[4 * wg], q4, lane);
      sync_wg(wg);
      if (t < NR) {
        const float (*a)[32] = &s_red[4 * wg], (*c)[32] = &s_red2[4 * wg];
        s_sum[wg][t] = (a[0][t] + a[1][t]) + (a[2][t] + a[3][t]);
        s_corr[wg][t] = (c[0][t] + c[1][t]) + (c[2][t] + c[3][t]);
      }
      if (mine >= 0) ok &= o_done((uint32_t)mine);                 // PV of the last stage
      tc_fence_after();
      sync_wg(wg);
      float* const sX = reinterpret_cast<float*>(dyn + L::kOffX);
      // rows c .. c + C of this thread's channel
      auto load_o = [&](int c, float* o) {
        const uint32_t at = tmem + lane_base + L::kColO + (ALT ? wg * N : rb) + c;
        tm_load(at, o);
        if constexpr (E4) {
          float lo[C];
          tm_load(at + NRT, lo);
#pragma unroll
          for (int r = 0; r < C; ++r) o[r] = fmaf(lo[r], kLo, o[r]) * 512.f;
        }
#pragma unroll
        for (int r = 0; r < C; ++r) o[r] += s_corr[wg][c + r];
      };
      if (ALT && wg == 1) {
        // hand over: references, sums, unnormalised rows
        if (t < NR) {
          s_xm[t] = -s_nu[1][t];
          s_xl[t] = s_sum[1][t];
        }
        if (mine >= 0) {
#pragma unroll
          for (int c = 0; c < NR; c += C) {
            float o[C];
            load_o(c, o);
#pragma unroll
            for (int r = 0; r < C; ++r) sX[(c + r) * 128 + t] = o[r];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_X));
      } else {
        const bool single = sg.nseg == 1;
        const int slot_idx = sg.unit + blockIdx.x;       // partial slot of (unit, this CTA)
        const size_t rowbase = (size_t)(sg.b * p.R + p.r0) * p.Hq + (size_t)sg.h * p.G;
        if (ALT) ok &= mbar_wait(BAR(B_X), par, &s_abort, p.status);   // the second warpgroup's part
        if (t < NR) {
          // one state from one or two: a warpgroup without tokens has sum 0
          const int i = rb + t;
          float lt = s_sum[wg][t], m = -s_nu[wg][t];
          if (ALT) {
            const float l1 = s_xl[t], m1 = s_xm[t];
            const float mm = l1 == 0.f ? m : lt == 0.f ? m1 : fmaxf(m, m1);
            const float a0 = ex2(m - mm), a1 = ex2(m1 - mm);
            s_f0[t] = lt == 0.f ? -1.f : a0;
            s_f1[t] = l1 == 0.f ? -1.f : a1;
            lt = (lt == 0.f ? 0.f : lt * a0) + (l1 == 0.f ? 0.f : l1 * a1);
            m = mm;
          }
          if (i < p.rows) {
            if (single) {
              if (p.lse) p.lse[rowbase + s_roff[i]] = lt == 0.f ? -INFINITY : (m + log2f(lt)) * kLn2;
            } else {
              const size_t pi = (size_t)slot_idx * p.rows + i;
              p.part_ml[pi * 2] = m;
              p.part_ml[pi * 2 + 1] = lt;
            }
          }
          s_sum[wg][t] = lt == 0.f ? 0.f : 1.f / lt;
        }
        sync_wg(wg);
#pragma unroll
        for (int c = 0; c < NR; c += C) {
          float o[C];
          load_o(c, o);
          if (D == 128 || t < D) {
#pragma unroll
            for (int r = 0; r < C; ++r) {
              const int i = rb + c + r;
              if (i >= p.rows) break;
              float v = o[r];
              if (ALT) {
                // a part without tokens has no O^T, whatever lies there
                const float a0 = s_f0[c + r], a1 = s_f1[c + r];
                v = a0 >= 0.f ? v * a0 : 0.f;
                if (a1 >= 0.f) v = fmaf(sX[(c + r) * 128 + t], a1, v);
              }
              if (single)
                static_cast<__nv_bfloat16*>(p.out)[(rowbase + s_roff[i]) * D + t] = __float2bfloat16_rn(v * s_sum[wg][c + r]);
              else
                p.part_o[((size_t)slot_idx * p.rows + i) * D + t] = v;
            }
          }
        }
        tc_fence_before();
        if (!single) __threadfence();
        __syncwarp();
        if (!ALT && wg == 1) {
          if (lane == 0) mbar_arrive(BAR(B_X));          // its rows are written
        } else {
          if (!ALT) ok &= mbar_wait(BAR(B_X), par, &s_abort, p.status);
          if (lane == 0) mbar_arrive(BAR(B_Y));
        }
        if (!single && wg == 0) {
          sync_wg(wg);
          if (tid == 0) {
            __threadfence();
            if (atomicAdd(p.tickets + sg.unit, 1u) == (unsigned)(sg.nseg - 1)) {
              // this CTA finished the unit last: its partials are merged after
              // the CTA's own streaming is done
              s_pend[s_npend++] = make_int4(sg.b, sg.h, sg.first_cta + sg.unit, sg.nseg);
              p.tickets[sg.unit] = 0u;
            }
          }
        }
      }
      sync_wg(wg);                             // s_alpha / s_nu / s_sum reads done
      x = sg.end;
      sg = nx;
    }
    // ---- deferred merges of the units this CTA finished last (skipped,
    // together, after a failed wait)
    if (wg == 0 && count_wg(wg, !ok) == 0) {
      __threadfence();
      for (int k = 0; k < s_npend; ++k) {
        const int4 u = s_pend[k];
        kvq_combine<__nv_bfloat16>(p, u.x, u.y, u.z, u.w, 128);
      }
    }
  }

  // ---- teardown: every role is done; wait for the MMAs, free TMEM
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaQk) {
    tc_fence_after();
    if (lane == 0) mbar_wait_drain(BAR(B_TD), 0, p.status);
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int NR, bool ALT, int D, int P, int BITS>
cudaError_t launch_one(const KvqAttnParams& p, cudaStream_t st) {
  const size_t smem = Lay<NR, ALT, D, BITS>::kDynBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<NR, ALT, D, P, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  // the register split draws on the launch's registers: never run it on others
  // (asked once; a query that fails is asked again by the next call)
  static std::atomic<int> regs{0};
  if (regs == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, attn_kernel<NR, ALT, D, P, BITS>);
    if (e != cudaSuccess) return e;
    regs = a.numRegs;
  }
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  int grid = device_sm_count();
  if (grid > kMaxPersistentCtas) grid = kMaxPersistentCtas;
  return launch_kernel(attn_kernel<NR, ALT, D, P, BITS>, dim3(grid), dim3(kThreads), smem, st, 1, p);
}

// Rows of a softmax warpgroup: the packed rows rounded up; beyond 24, half of them.
template <int D, int P, int BITS>
cudaError_t launch_rows(const KvqAttnParams& p, cudaStream_t st) {
  if (p.rows <= 4) return launch_one<4, true, D, P, BITS>(p, st);
  if (p.rows <= 8) return launch_one<8, true, D, P, BITS>(p, st);
  if (p.rows <= 16) return launch_one<16, true, D, P, BITS>(p, st);
  if (p.rows <= 24) return launch_one<24, true, D, P, BITS>(p, st);
  if (p.rows <= 32) return launch_one<16, false, D, P, BITS>(p, st);
  if (p.rows <= 48) return launch_one<24, false, D, P, BITS>(p, st);
  return launch_one<32, false, D, P, BITS>(p, st);
}

}  // namespace kvq
}  // namespace s3r
