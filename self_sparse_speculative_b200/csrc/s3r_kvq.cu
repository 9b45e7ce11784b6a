// Writing and reading the quantised paged KV cache (layout and arithmetic of a
// row: s3r_kvq.cuh). The drafter and the verifier of S3R share one cache
// ("S3R: Fast and Faithful RL Rollouts via Self-Sparse Speculative Decoding",
// weekinpapers.com, Abstract); held in 4 bits it is 3.8 times smaller than in
// bf16, in 8 bits 1.9 times (D = 128).
//
//   kvq_store_kernel     rows quantised and written: n new rows per sequence
//                        (append), or positions of a bf16 / f32 paged cache
//                        (pack)
//   kvq_read_kernel      a window of positions back to rows of bf16 / f32
//   kvq_rollback_kernel  the lengths back to the committed prefix
//
// Measured (16 x 16384 tokens, 8 KV heads, D 128, 4 bits): quantising a bf16 cache
// 330 us, 4.1 TB/s, bound by instruction issue (73% of cycles, 17 instructions a
// value); reading back 249 us, 5.5 TB/s, 0.83 of a copy's rate. Single rows are a
// chain of dependent loads (length -> page id -> rows), 3 to 4 us a kernel.
//
// A CTA of 128 threads takes tiles of T consecutive tokens of one (sequence, KV
// head), T = 32 for 64-token pages and 16 for 16-token ones: a tile then holds
// whole V pieces, so the V bytes of a tile belong to one CTA and no two CTAs of
// a call write the same byte; with small rows or pages a CTA takes two or four
// tiles. A row is D/8 lanes of 8 channels (16-byte loads of bf16); minimum and
// maximum meet by shuffles. K numbers go out as they are; V numbers turn
// channel-major through shared memory, four channels by eight tokens per
// thread with byte permutes, and leave as 16-byte pieces. A V piece of which
// only some tokens are written keeps the other tokens' bits.
//
// These kernels write inputs of later calls: they wait for the previous kernel
// before touching anything and let the next one start only when they are done.
#include <cuda_bf16.h>

#include "s3r_device.cuh"
#include "s3r_internal.h"
#include "s3r_kvq.cuh"

namespace s3r {
namespace {

constexpr int kKvqThreads = 128;

struct KvqParams {
  uint8_t* pages;             // [num_pages_total, Hkv, page_bytes]
  const int32_t* block_table;
  const int32_t* lens;
  int32_t* lens_out;          // append: lengths to update (null: leave them)
  const void* k_src;          // append: rows [S, n, Hkv, D]; pack: paged cache [src_pages, Hkv, P, D]
  const void* v_src;
  const int32_t* src_table;   // pack: the source's block table
  int32_t src_max_pages, src_pages_total;
  void* k_out;                // read: [S, n, Hkv, D]
  void* v_out;
  const int32_t* start;       // read: first position per sequence (null: 0)
  const int32_t* num_accepted;
  int32_t S, Hkv, P, max_pages, num_pages_total;
  int32_t n, overwrite, rows;
  uint32_t* status;
  uint32_t* tickets;          // [S]
};

// 8 consecutive channels of a row (of this lane), as loaded.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcg(reinterpret_cast<const float4*>(p));
    b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float2 pair(int i) const {
    return i == 0 ? make_float2(a.x, a.y) : i == 1 ? make_float2(a.z, a.w) : i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w);
  }
};

// Minimum and maximum over a row, NaN if it holds one. bf16: exact in packed
// bf16, both in one word {min, -max} across the lanes.
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ uint32_t range_of(const Raw8<__nv_bfloat16>& x) {
  const uint32_t lo = as_u32(__hmin2_nan(__hmin2_nan(as_bf2(x.w[0]), as_bf2(x.w[1])), __hmin2_nan(as_bf2(x.w[2]), as_bf2(x.w[3]))));
  const uint32_t hi = as_u32(__hmax2_nan(__hmax2_nan(as_bf2(x.w[0]), as_bf2(x.w[1])), __hmax2_nan(as_bf2(x.w[2]), as_bf2(x.w[3]))));
  return as_u32(__hmin2_nan(as_bf2(__byte_perm(lo, hi ^ 0x80008000u, 0x5410)), as_bf2(__byte_perm(lo, hi ^ 0x80008000u, 0x7632))));
}
__device__ __forceinline__ uint32_t range_join(uint32_t a, uint32_t b) { return as_u32(__hmin2_nan(as_bf2(a), as_bf2(b))); }
__device__ __forceinline__ uint32_t range_from(uint32_t a, int lanes) { return __shfl_xor_sync(0xffffffffu, a, lanes); }
__device__ __forceinline__ float2 range_ends(uint32_t m) {
  return make_float2(__uint_as_float(m << 16), __uint_as_float((m & 0xffff0000u) ^ 0x80000000u));
}
__device__ __forceinline__ float2 range_of(const Raw8<float>& x) {
  float a = x.a.x, b = x.a.x;
  const float y[7] = {x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    a = min_nan(a, y[i]);
    b = max_nan(b, y[i]);
  }
  return make_float2(a, b);
}
__device__ __forceinline__ float2 range_join(float2 a, float2 b) { return make_float2(min_nan(a.x, b.x), max_nan(a.y, b.y)); }
__device__ __forceinline__ float2 range_from(float2 a, int lanes) {
  return make_float2(__shfl_xor_sync(0xffffffffu, a.x, lanes), __shfl_xor_sync(0xffffffffu, a.y, lanes));
}
__device__ __forceinline__ float2 range_ends(float2 m) { return m; }

// The ranges of eight rows, r[k] this lane's share of row k: lane c8 of the
// row's kLanes gets row c8 % 8's. Lanes swap halves of the rows, then quarters,
// then single rows: 8 shuffles instead of 32.
template <int kLanes, typename R>
__device__ __forceinline__ float2 scatter_ranges(R* r, int c8) {
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) {
    const bool up = (c8 & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const R keep = up ? r[i + o] : r[i], give = up ? r[i] : r[i + o];
      r[i] = range_join(keep, range_from(give, o));
    }
  }
  if (kLanes == 16) r[0] = range_join(r[0], range_from(r[0], 8));
  return range_ends(r[0]);
}

template <typename T> __device__ __forceinline__ void store8(T* p, const float* x);
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                            pack_bf16x2(x[6], x[7]));
}
template <> __device__ __forceinline__ void store8<float>(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The numbers of 8 values from float64 quotients (rare: kept out of line, its
// divisions would crowd the instruction cache).
template <typename T, int BITS>
__device__ __noinline__ uint2 quantise8_exact(const Raw8<T> x, float z, float s) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = x.pair(i).x;
    v[2 * i + 1] = x.pair(i).y;
  }
  uint32_t c[2] = {0u, 0u};
#pragma unroll 1
  for (int i = 0; i < 8; ++i) c[i >> 2] |= kvq_number_exact<BITS>(v[i], z, s) << (8 * (i & 3));
  return make_uint2(c[0], c[1]);
}

// The numbers of this lane's 8 channels, byte i of code = channel i; at 4 bits
// also as 4 bytes of two. They are those of the exact quotient, ties to even:
// - bf16: exact ties are common (8-bit values and steps). x - z is exact in
//   float32 unless the two are more than 2^16 apart: (x - z) + z tells where x
//   is the small one (that sum is exact then), `wide` where z is (a row at a
//   time; it reaches the lanes as the sign of s). The quotient corrected by its remainder is the exact one
//   rounded: it equals a border m + 1/2 only if the quotient does. (Off a border, 2 (x - z) and s (2 m + 1)
//   differ by a whole number of the smaller of their lowest bits; the first has 24 bits, the second at most 8 +
//   BITS + 1, so they differ by more than 2^-24 of themselves, and float32 rounds by at most 2^-24.)
// - float32: t = (x - z) (1 / s) is within 3 u t (u = 2^-24, t at most 2^BITS)
//   of the exact quotient; nearer than 2^-17 (4 bits) or 2^-14 (8 bits), twice
//   that, to a border, float64 decides.
// Differences that overflow fail both tests. s is at most 2^-8 of itself below
// (max - z) / (2^BITS - 1): n may reach 256 at 8 bits (held to 255), 15 at 4.
// inv = 0 (equal values, or a row with NaN or infinity) gives zeros.
template <typename T, int BITS>
__device__ __forceinline__ void quantise8(const Raw8<T>& x, float z, float s, float inv, uint32_t* code, uint32_t* packed) {
  constexpr float kMagic = 12582912.f;                   // 1.5 * 2^23: rounds to the nearest whole, ties to even
  constexpr bool kBf16 = sizeof(T) == 2;
  uint32_t b[8], off = __float_as_uint(s) >> 31;         // (a wide row)
  s = fabsf(s);
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = x.pair(i);
    const float2 d = fma_pair(both(-z), both(1.f), v);
    float2 t = fma_pair(d, both(inv), both(0.f));
    if (kBf16) {
      t = fma_pair(fma_pair(t, both(-s), d), both(inv), t);
      const float2 e = fma_pair(fma_pair(d, both(1.f), both(z)), both(-1.f), v);          // x - (d + z)
      off |= __float_as_uint(e.x) | __float_as_uint(e.y);
    }
    float2 f = fma_pair(t, both(1.f), both(kMagic));
    if (!kBf16) {
      const float2 r = fma_pair(fma_pair(f, both(1.f), both(-kMagic)), both(-1.f), t);
      far = fmaxf(far, fmaxf(fabsf(r.x), fabsf(r.y)));
      if (!(fabsf(t.x) + fabsf(t.y) < 4096.f)) far = 1.f;
    }
    if (BITS == 8) f = make_float2(fminf(f.x, kMagic + 255.f), fminf(f.y, kMagic + 255.f));
    b[2 * i] = __float_as_uint(f.x);
    b[2 * i + 1] = __float_as_uint(f.y);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
    code[q] = __byte_perm(__byte_perm(b[4 * q], b[4 * q + 1], 0x0040), __byte_perm(b[4 * q + 2], b[4 * q + 3], 0x0040), 0x5410);
  if (kBf16 ? off != 0u : far > 0.5f - (BITS == 4 ? 0x1p-17f : 0x1p-14f)) {
    // (a row with NaN or infinity comes here too, and holds zeros)
    const uint2 c = inv == 0.f ? make_uint2(0u, 0u) : quantise8_exact<T, BITS>(x, z, s);
    code[0] = c.x;
    code[1] = c.y;
  }
  if (BITS == 4) {
    const uint32_t lo = code[0] | (code[0] >> 4), hi = code[1] | (code[1] >> 4);   // two half-bytes a byte, at bytes 0 and 2
    *packed = __byte_perm(lo, hi, 0x6420);
  }
}

// Shared V numbers of a tile, a byte each: [T][D], rows padded so that the
// four token groups of a warp fall on different banks.
template <int D>
constexpr int kVStride = D + 4;

// V pieces of a tile: [T / ut][D] slots of 16 bytes, slot d at d ^ (d / 8 % 8)
// of its group of eight.
__device__ __forceinline__ int v_slot(int d) { return (d & ~7) | ((d ^ (d >> 3)) & 7); }

// 4x4 byte transpose: byte c of in[r] -> byte r of out[c].
__device__ __forceinline__ void transpose4(const uint32_t* in, uint32_t* out) {
  const uint32_t a = __byte_perm(in[0], in[1], 0x5140), b = __byte_perm(in[0], in[1], 0x7362);
  const uint32_t c = __byte_perm(in[2], in[3], 0x5140), d = __byte_perm(in[2], in[3], 0x7362);
  out[0] = __byte_perm(a, c, 0x5410);
  out[1] = __byte_perm(a, c, 0x7632);
  out[2] = __byte_perm(b, d, 0x5410);
  out[3] = __byte_perm(b, d, 0x7632);
}

// Bits of word w of a V piece (of `ut` tokens) whose tokens lie in [t0, t1).
template <int BITS>
__device__ __forceinline__ uint32_t token_mask(int w, int t0, int t1) {
  constexpr int kPer = 32 / BITS;
  const int a = max(0, min(kPer, t0 - w * kPer)) * BITS, b = max(0, min(kPer, t1 - w * kPer)) * BITS;
  const uint32_t below_b = b >= 32 ? ~0u : (1u << b) - 1u, below_a = a >= 32 ? ~0u : (1u << a) - 1u;
  return below_b & ~below_a;
}

// How a CTA is cut: tiles of TT tokens, kT threads each, four rows a lane.
template <int D, int P, int BITS>
struct Cut {
  static constexpr KvqLayout Y = kvq_layout(D, P, BITS);
  static constexpr int TT = P == 64 ? 32 : 16;           // tokens per tile
  static constexpr int kLanes = D / 8;                   // lanes per row
  static constexpr int NR = 4;                           // rows per lane
  static constexpr int kT = TT * kLanes / NR;            // threads per tile: 32, 64 or 128
  static constexpr int kTiles = kKvqThreads / kT;        // tiles per CTA
  static constexpr int kRowsPass = kT / kLanes;          // rows per pass of a tile's threads
  static constexpr int kPieces = TT / Y.ut;              // V pieces per channel in a tile
  static constexpr int kTg = TT / 8;                     // groups of eight tokens
  static constexpr int kVWords = TT * kVStride<D> / 4;
};

template <typename T, int D, int P, int BITS, bool PACK>
__global__ void __launch_bounds__(kKvqThreads, sizeof(T) == 2 ? 8 : 4) kvq_store_kernel(const KvqParams p) {
  using G = Cut<D, P, BITS>;
  constexpr KvqLayout Y = G::Y;
  constexpr int TT = G::TT, kLanes = G::kLanes, NR = G::NR, kT = G::kT, kRowsPass = G::kRowsPass, kPieces = G::kPieces;
  constexpr int kWords = Y.unit / 4;                     // words per V piece
  static_assert(2 * NR == 8 && (kLanes == 8 || kLanes == 16), "a lane for each row's parameters");
  __shared__ __align__(16) uint32_t s_va[G::kTiles * G::kVWords];
  __shared__ __align__(16) uint4 s_pa[G::kTiles * kPieces * D];
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int L = __ldcg(p.lens + b);
  int first, end;                                        // positions written
  bool bad;
  if (PACK) {
    end = L;
    first = p.n > 0 ? max(0, L - p.n) : 0;
    bad = L < 1 || L > p.max_pages * P || L > p.src_max_pages * P;
  } else {
    first = L - p.overwrite;
    end = first + p.n;
    bad = L < 0 || first < 0 || end < 1 || end > p.max_pages * P;
  }
  if (bad && tid == 0 && h == 0 && blockIdx.x == 0) flag_status(p.status, S3R_DEV_BAD_CONTEXT_LEN);
  // this thread's tile; a tile without work still takes part in the barriers
  const int sub = tid / kT, tt = tid % kT;
  uint32_t* const s_v = s_va + sub * G::kVWords;
  uint4* const s_piece = s_pa + sub * (kPieces * D);
  const int base = (first / TT + (int)blockIdx.x * G::kTiles + sub) * TT;   // first position of the tile
  bool work = !bad && base < end && first < end;
  const int page = base / P, in_page = base - page * P;
  int phys = -1, src = 0;
  if (work) {
    phys = p.block_table[(size_t)b * p.max_pages + page];
    bool ok = phys >= 0 && phys < p.num_pages_total;
    if (PACK) {
      src = p.src_table[(size_t)b * p.src_max_pages + page];
      ok = ok && src >= 0 && src < p.src_pages_total;
    }
    if (!ok) {
      if (tt == 0) flag_status(p.status, S3R_DEV_BAD_PAGE_ID);
      work = false;
    }
  }
  if (G::kTiles == 1 ? work : __syncthreads_or(work)) {
    uint8_t* const pg = p.pages + ((size_t)max(phys, 0) * p.Hkv + h) * Y.page_bytes;
    const int row0 = tt / kLanes, c8 = tt % kLanes;
    const int t0 = work ? max(first - base, 0) : 0, t1 = work ? min(end - base, TT) : 0;   // tokens of the tile written
    Raw8<T> xk[NR], xv[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int t = row0 + k * kRowsPass;
      xk[k].zero();
      xv[k].zero();
      if (t >= t0 && t < t1) {
        const size_t at = PACK ? (((size_t)src * p.Hkv + h) * P + in_page + t) * D + c8 * 8
                               : (((size_t)b * p.n + (base + t - first)) * p.Hkv + h) * D + c8 * 8;
        xk[k].load(static_cast<const T*>(p.k_src) + at);
        xv[k].load(static_cast<const T*>(p.v_src) + at);
      }
    }
    // lane i of each row group works out the parameters of its i-th row, so
    // that they cost one row's instructions
    decltype(range_of(xk[0])) part[2 * NR];
#pragma unroll
    for (int k = 0; k < 2 * NR; ++k) part[k] = range_of(k < NR ? xk[k] : xv[k - NR]);
    const float2 ends = scatter_ranges<kLanes>(part, c8);
    const KvqRow row = kvq_row<BITS>(ends.x, ends.y);
    if (c8 < 2 * NR) {
      const int t = row0 + (c8 % NR) * kRowsPass;
      if (t >= t0 && t < t1)
        *reinterpret_cast<uint32_t*>(pg + (c8 < NR ? Y.off_kp : Y.off_vp) + (in_page + t) * 4) = pack_bf16x2(row.s, row.z);
    }
    const int group = (tid & 31) & ~(kLanes - 1);
#pragma unroll
    for (int k = 0; k < 2 * NR; ++k) {
      const int t = row0 + (k % NR) * kRowsPass;
      const bool live = t >= t0 && t < t1;
      const float z = __shfl_sync(0xffffffffu, row.z, group + k), s = __shfl_sync(0xffffffffu, row.wide ? -row.s : row.s, group + k);
      const float inv = __shfl_sync(0xffffffffu, row.inv, group + k);
      uint32_t code[2], packed = 0u;
      quantise8<T, BITS>(k < NR ? xk[k] : xv[k - NR], z, s, inv, code, &packed);
      if (k >= NR) {
        s_v[(t * kVStride<D>) / 4 + c8 * 2] = code[0];
        s_v[(t * kVStride<D>) / 4 + c8 * 2 + 1] = code[1];
      } else if (live) {
        if (BITS == 4)
          *reinterpret_cast<uint32_t*>(pg + ((c8 >> 2) * P + in_page + t) * 16 + (c8 & 3) * 4) = packed;
        else
          *reinterpret_cast<uint2*>(pg + ((c8 >> 1) * P + in_page + t) * 16 + (c8 & 1) * 8) = make_uint2(code[0], code[1]);
      }
    }
    __syncthreads();
    // four channels x eight tokens per step: lanes take 8 channel groups x 4 token groups
    constexpr int kTg = G::kTg;
    for (int s = tt; s < (D / 4) * kTg; s += kT) {
      const int in = s % (8 * kTg), cg = (s / (8 * kTg)) * 8 + (in & 7), tg = in >> 3;
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = s_v[((tg * 8 + k) * kVStride<D>) / 4 + cg];
      uint32_t a[4], o[4];
      if (BITS == 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = w[2 * k] | (w[2 * k + 1] << 4);
        transpose4(a, o);
        const int piece = tg * 8 / Y.ut, word = (tg * 8 % Y.ut) / 8;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          reinterpret_cast<uint32_t*>(&s_piece[piece * D + v_slot(cg * 4 + c)])[word] = o[c];
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          transpose4(w + 4 * q, o);
          const int t = tg * 8 + 4 * q;
          const int piece = t / Y.ut, word = (t % Y.ut) / 4;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            reinterpret_cast<uint32_t*>(&s_piece[piece * D + v_slot(cg * 4 + c)])[word] = o[c];
        }
      }
    }
    __syncthreads();
    for (int s = tt; s < kPieces * D; s += kT) {
      const int piece = s / D, d = s - (s / D) * D;
      const int u0 = piece * Y.ut;                   // first token of the piece, within the tile
      const int a = t0 - u0, e = t1 - u0;
      if (e <= 0 || a >= Y.ut) continue;
      uint4 v = s_piece[piece * D + v_slot(d)];
      uint8_t* dst = pg + Y.off_v + ((in_page / Y.ut + piece) * D + d) * Y.unit;
      if (a > 0 || e < Y.ut) {                       // keep the other tokens' bits
        uint32_t* nv = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const uint32_t m = token_mask<BITS>(w, a, e);
          nv[w] = (nv[w] & m) | (reinterpret_cast<const uint32_t*>(dst)[w] & ~m);
        }
      }
      if (Y.unit == 16) *reinterpret_cast<uint4*>(dst) = v;
      else *reinterpret_cast<uint2*>(dst) = make_uint2(v.x, v.y);
    }
  }
  if (!PACK && p.lens_out) {
    // the last CTA of the sequence stores its new length
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      if (atomicAdd(p.tickets + b, 1u) == gridDim.x * gridDim.y - 1u) {
        if (!bad) p.lens_out[b] = end;
        p.tickets[b] = 0u;
      }
    }
  }
}

template <typename T, int D, int P, int BITS>
__global__ void __launch_bounds__(kKvqThreads) kvq_read_kernel(const KvqParams p) {
  using G = Cut<D, P, BITS>;
  constexpr KvqLayout Y = G::Y;
  constexpr int TT = G::TT, kLanes = G::kLanes, NR = G::NR, kT = G::kT, kRowsPass = G::kRowsPass, kPieces = G::kPieces;
  __shared__ __align__(16) uint32_t s_va[G::kTiles * G::kVWords];
  __shared__ __align__(16) uint4 s_pa[G::kTiles * kPieces * D];
  pdl_wait();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int L = __ldcg(p.lens + b);
  const int first = p.start ? __ldcg(p.start + b) : 0;
  if (L < 1 || L > p.max_pages * P || first < 0) {
    if (tid == 0 && h == 0 && blockIdx.x == 0) flag_status(p.status, S3R_DEV_BAD_CONTEXT_LEN);
    return;
  }
  const int end = p.n < L - first ? first + p.n : L;     // rows of positions >= L are left as they are
  const int sub = tid / kT, tt = tid % kT;               // this thread's tile; one without work still takes part in the barriers
  uint32_t* const s_v = s_va + sub * G::kVWords;
  uint4* const s_piece = s_pa + sub * (kPieces * D);
  if (first >= end) return;
  const int base = (first / TT + (int)blockIdx.x * G::kTiles + sub) * TT;
  bool work = base < end;
  const int page = base / P, in_page = base - page * P;
  int phys = -1;
  if (work) {
    phys = p.block_table[(size_t)b * p.max_pages + page];
    if (phys < 0 || phys >= p.num_pages_total) {
      if (tt == 0) flag_status(p.status, S3R_DEV_BAD_PAGE_ID);
      work = false;
    }
  }
  if (G::kTiles == 1 ? !work : !__syncthreads_or(work)) return;
  const uint8_t* pg = p.pages + ((size_t)max(phys, 0) * p.Hkv + h) * Y.page_bytes;
  const int row0 = tt / kLanes, c8 = tt % kLanes;
  const int t0 = work ? max(first - base, 0) : 0, t1 = work ? min(end - base, TT) : 0;
  // every load of the tile first
  if (work) for (int s = tt; s < kPieces * D; s += kT) {
    const int piece = s / D, d = s - (s / D) * D;
    const uint8_t* src = pg + Y.off_v + ((in_page / Y.ut + piece) * D + d) * Y.unit;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (Y.unit == 16) v = __ldcg(reinterpret_cast<const uint4*>(src));
    else {
      const uint2 a = __ldcg(reinterpret_cast<const uint2*>(src));
      v.x = a.x;
      v.y = a.y;
    }
    s_piece[piece * D + v_slot(d)] = v;
  }
  uint2 kc[NR];
  uint32_t kp[NR], vp[NR];
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const int t = in_page + row0 + k * kRowsPass;
    kc[k] = make_uint2(0u, 0u);
    kp[k] = vp[k] = 0u;
    if (G::kTiles > 1 && !work) continue;
    if (BITS == 4) kc[k].x = __ldcg(reinterpret_cast<const uint32_t*>(pg + ((c8 >> 2) * P + t) * 16 + (c8 & 3) * 4));
    else kc[k] = __ldcg(reinterpret_cast<const uint2*>(pg + ((c8 >> 1) * P + t) * 16 + (c8 & 1) * 8));
    kp[k] = __ldcg(reinterpret_cast<const uint32_t*>(pg + Y.off_kp + t * 4));
    vp[k] = __ldcg(reinterpret_cast<const uint32_t*>(pg + Y.off_vp + t * 4));
  }
  auto put = [&](void* out, int t, uint32_t lo, uint32_t hi, uint32_t par) {
    // bytes of lo, hi: the 8 channels' numbers
    const float s = __uint_as_float(par << 16), z = __uint_as_float(par & 0xffff0000u);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t n = ((i < 4 ? lo : hi) >> (8 * (i & 3))) & 0xffu;
      x[i] = fmaf(s, __uint_as_float(0x4b000000u | n) - 8388608.f, z);
    }
    store8<T>(static_cast<T*>(out) + (((size_t)b * p.n + (base + t - first)) * p.Hkv + h) * D + c8 * 8, x);
  };
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const int t = row0 + k * kRowsPass;
    if (t < t0 || t >= t1) continue;
    if (BITS == 4) {
      const uint32_t e = kc[k].x & 0x0f0f0f0fu, o = (kc[k].x >> 4) & 0x0f0f0f0fu;   // even, odd channels
      put(p.k_out, t, __byte_perm(e, o, 0x5140), __byte_perm(e, o, 0x7362), kp[k]);
    } else {
      put(p.k_out, t, kc[k].x, kc[k].y, kp[k]);
    }
  }
  __syncthreads();
  constexpr int kTg = G::kTg;
  for (int s = tt; s < (D / 4) * kTg; s += kT) {
    const int in = s % (8 * kTg), cg = (s / (8 * kTg)) * 8 + (in & 7), tg = in >> 3;
    uint32_t a[4], o[4];
    if (BITS == 4) {
      const int piece = tg * 8 / Y.ut, word = (tg * 8 % Y.ut) / 8;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        a[c] = reinterpret_cast<const uint32_t*>(&s_piece[piece * D + v_slot(cg * 4 + c)])[word];
      transpose4(a, o);                                  // o[k]: tokens 2k, 2k+1 of four channels
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s_v[((tg * 8 + 2 * k) * kVStride<D>) / 4 + cg] = o[k] & 0x0f0f0f0fu;
        s_v[((tg * 8 + 2 * k + 1) * kVStride<D>) / 4 + cg] = (o[k] >> 4) & 0x0f0f0f0fu;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int t = tg * 8 + 4 * q;
        const int piece = t / Y.ut, word = (t % Y.ut) / 4;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          a[c] = reinterpret_cast<const uint32_t*>(&s_piece[piece * D + v_slot(cg * 4 + c)])[word];
        transpose4(a, o);
#pragma unroll
        for (int k = 0; k < 4; ++k) s_v[((t + k) * kVStride<D>) / 4 + cg] = o[k];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NR; ++k) {
    const int t = row0 + k * kRowsPass;
    if (t < t0 || t >= t1) continue;
    put(p.v_out, t, s_v[(t * kVStride<D>) / 4 + c8 * 2], s_v[(t * kVStride<D>) / 4 + c8 * 2 + 1], vp[k]);
  }
}

__global__ void __launch_bounds__(kKvqThreads) kvq_rollback_kernel(const KvqParams p) {
  pdl_wait();
  const int b = blockIdx.x * kKvqThreads + threadIdx.x;
  if (b >= p.S) return;
  const int L = p.lens_out[b], nacc = p.num_accepted[b];
  const int new_len = L - p.rows + nacc + 1;
  if (nacc < 0 || nacc >= p.rows || L < 1 || new_len < 1 || L > p.max_pages * p.P) {
    flag_status(p.status, S3R_DEV_BAD_CONTEXT_LEN);
    return;
  }
  p.lens_out[b] = new_len;
}

KvqParams base_params(const s3r_paged_kvq& c, void* ws) {
  KvqParams p{};
  p.pages = static_cast<uint8_t*>(c.pages);
  p.block_table = c.block_table;
  p.lens = c.context_lens;
  p.S = c.num_seqs;
  p.Hkv = c.num_kv_heads;
  p.P = c.page_size;
  p.max_pages = c.max_pages_per_seq;
  p.num_pages_total = c.num_pages_total;
  p.status = static_cast<uint32_t*>(ws);
  p.tickets = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kWsHeader);
  return p;
}

// CTAs for the tiles that n consecutive positions may touch.
unsigned tile_ctas(int n, int D, int P) {
  const int tt = P == 64 ? 32 : 16, per = kKvqThreads / (tt * (D / 8) / 4);
  const int tiles = n <= 0 ? 1 : (n + tt - 2) / tt + 1;
  return (unsigned)((tiles + per - 1) / per);
}

enum KvqOp { kStoreRows, kStorePages, kRead };

template <typename T, int D, int P, int BITS>
cudaError_t launch_one(KvqOp op, const KvqParams& p, dim3 grid, cudaStream_t st) {
  const dim3 block(kKvqThreads);
  switch (op) {
    case kStoreRows: return launch_kernel(kvq_store_kernel<T, D, P, BITS, false>, grid, block, 0, st, 1, p);
    case kStorePages: return launch_kernel(kvq_store_kernel<T, D, P, BITS, true>, grid, block, 0, st, 1, p);
    default: return launch_kernel(kvq_read_kernel<T, D, P, BITS>, grid, block, 0, st, 1, p);
  }
}
template <typename T, int D, int P>
cudaError_t launch_bits(KvqOp op, int bits, const KvqParams& p, dim3 grid, cudaStream_t st) {
  return bits == 4 ? launch_one<T, D, P, 4>(op, p, grid, st) : launch_one<T, D, P, 8>(op, p, grid, st);
}
template <typename T>
cudaError_t launch_shape(KvqOp op, const s3r_paged_kvq& c, const KvqParams& p, dim3 grid, cudaStream_t st) {
  if (c.head_dim == 64)
    return c.page_size == 16 ? launch_bits<T, 64, 16>(op, c.bits, p, grid, st) : launch_bits<T, 64, 64>(op, c.bits, p, grid, st);
  return c.page_size == 16 ? launch_bits<T, 128, 16>(op, c.bits, p, grid, st) : launch_bits<T, 128, 64>(op, c.bits, p, grid, st);
}
cudaError_t launch_typed(KvqOp op, s3r_dtype dt, const s3r_paged_kvq& c, const KvqParams& p, dim3 grid, cudaStream_t st) {
  return dt == S3R_BF16 ? launch_shape<__nv_bfloat16>(op, c, p, grid, st) : launch_shape<float>(op, c, p, grid, st);
}

}  // namespace

cudaError_t launch_kvq_append(const s3r_paged_kvq& c, int32_t* lens, const void* k_new, const void* v_new, s3r_dtype dt,
                              int32_t n, int32_t overwrite, void* ws, cudaStream_t st) {
  KvqParams p = base_params(c, ws);
  p.lens_out = lens;
  p.k_src = k_new;
  p.v_src = v_new;
  p.n = n;
  p.overwrite = overwrite;
  return launch_typed(kStoreRows, dt, c, p, dim3(tile_ctas(n, c.head_dim, c.page_size), c.num_kv_heads, c.num_seqs), st);
}

cudaError_t launch_kvq_pack(const s3r_paged_kv& kv, const s3r_paged_kvq& c, int32_t last_n, void* ws, cudaStream_t st) {
  KvqParams p = base_params(c, ws);
  p.lens = kv.context_lens;
  p.k_src = kv.k_cache;
  p.v_src = kv.v_cache;
  p.src_table = kv.block_table;
  p.src_max_pages = kv.max_pages_per_seq;
  p.src_pages_total = kv.num_pages_total;
  p.n = last_n;
  const int cap = (c.max_pages_per_seq < kv.max_pages_per_seq ? c.max_pages_per_seq : kv.max_pages_per_seq) * c.page_size;
  const int n = last_n > 0 && last_n < cap ? last_n : cap;
  return launch_typed(kStorePages, kv.dtype, c, p, dim3(tile_ctas(n, c.head_dim, c.page_size), c.num_kv_heads, c.num_seqs), st);
}

cudaError_t launch_kvq_read(const s3r_paged_kvq& c, const int32_t* start, int32_t n, s3r_dtype dt, void* k_out, void* v_out,
                            void* ws, cudaStream_t st) {
  KvqParams p = base_params(c, ws);
  p.start = start;
  p.n = n;
  p.k_out = k_out;
  p.v_out = v_out;
  const int cap = c.max_pages_per_seq * c.page_size;
  return launch_typed(kRead, dt, c, p, dim3(tile_ctas(n < cap ? n : cap, c.head_dim, c.page_size), c.num_kv_heads, c.num_seqs), st);
}

cudaError_t launch_kvq_rollback(const s3r_paged_kvq& c, int32_t* lens, const int32_t* num_accepted, int32_t rows, void* ws,
                                cudaStream_t st) {
  KvqParams p = base_params(c, ws);
  p.lens_out = lens;
  p.num_accepted = num_accepted;
  p.rows = rows;
  return launch_kernel(kvq_rollback_kernel, dim3((c.num_seqs + kKvqThreads - 1) / kKvqThreads), dim3(kKvqThreads), 0, st, 1, p);
}

}  // namespace s3r
