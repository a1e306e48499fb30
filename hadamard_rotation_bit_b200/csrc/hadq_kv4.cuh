// A paged cache of int4 keys and values: appending rows to it, and attention
// of a sequence's newest tokens over it.
//
// Cache (one layer): pages of page_size positions, for K and for V
//   codes  [num_pages][kv_heads][page_size][D / 2]      two's-complement nibbles, element 2i low
//   scales [num_pages][kv_heads][page_size][D / GROUP]  fp16
// so 16 consecutive positions of one head are one contiguous run of codes and
// one of scales (page_size is a multiple of 16): the tile of both kernels.
#pragma once

#include <climits>

#include "hadq_device.cuh"

namespace hadq {
namespace kv4 {

// Fault bits (hadq_device_faults), beside those of the tensor-core kernels.
constexpr unsigned kFaultPage = 16u, kFaultLength = 32u, kFaultSlot = 64u;

static __device__ unsigned int hadq_kv4_fault;

// ------------------------------------------------------------------- append
//
// Rows are (token, head) pairs of D values.  K: z = x H_D, index bits in
// ascending order (the sum's order is part of the definition: equal inputs
// give equal codes), y = z / sqrt(D); V: y = x.  Per group of GROUP values
// with absmax m: s = fp16(min(m / 7, 65504)), q = clamp(rne(z f), -7, 7) with
// f = fp32(norm / s); s == 0 gives codes 0.
//
// A lane holds 32 consecutive values, D / 32 neighbouring lanes a row: five
// butterfly stages in registers, log2(D / 32) by shuffles.  Bound by memory.

// Eight codes of v * f, clamped to +-7: each exact product rounded once onto
// the integer grid.  For scales that were rounded far (subnormal or saturated);
// the others cannot reach 7.5 and take pack_int4x8.
__device__ __forceinline__ uint32_t int4_codes8(const float* v, float f) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = fminf(fmaxf(v[i] * f, -8.f), 8.f);      // only to bound the magnitude
    const float q = fabsf(p) < 8.f ? fmaf(v[i], f, kRoundMagic) : p + kRoundMagic;
    const int b = static_cast<int>(__float_as_uint(q) - kRoundMagicBits);
    w |= (static_cast<uint32_t>(min(max(b, -7), 7)) & 15u) << (4 * i);
  }
  return w;
}

// n / d for n < 2^31 by one product: m = floor(2^(31 + s) / d) + 1, s =
// ceil(log2 d) (Granlund and Montgomery, "Division by invariant integers using
// multiplication").
struct Divider {
  uint32_t m, s, d;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> (s - 1); }
};

struct AppendArgs {
  const void* x[2];          // K, V: row (t, h) at x + t * stride + h * D
  int64_t stride[2];         // elements between tokens
  uint8_t* codes[2];
  __half* scales[2];
  const int64_t* slots;      // position in the cache per token: page * page_size + offset; negative: no row
  int64_t num_slots;         // num_pages * page_size
  uint32_t rows;             // tokens * kv_heads, fewer than 2^31
  Divider kv_heads, page_size;
  int group;
  int rotate_k;              // 1: K rotated per head
  float norm;                // fp32(1 / sqrt(D))
};

// 32 consecutive values: 256-bit loads where they are 32-byte aligned (whole
// sectors), else 128-bit ones.
template <bool BF16>
__device__ __forceinline__ void load32(const void* x, int64_t e, float (&v)[32]) {
  constexpr int N = BF16 ? 4 : 8;
  const uint8_t* p = static_cast<const uint8_t*>(x) + e * (BF16 ? 2 : 4);
  uint4 w[N];
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) ld_stream32(p + 16 * i, w[i], w[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = ld_stream(reinterpret_cast<const uint4*>(p) + i);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (BF16) {
      unpack_bf16x2(w[i].x, v[8 * i + 0], v[8 * i + 1]);
      unpack_bf16x2(w[i].y, v[8 * i + 2], v[8 * i + 3]);
      unpack_bf16x2(w[i].z, v[8 * i + 4], v[8 * i + 5]);
      unpack_bf16x2(w[i].w, v[8 * i + 6], v[8 * i + 7]);
    } else {
      v[4 * i] = __uint_as_float(w[i].x), v[4 * i + 1] = __uint_as_float(w[i].y);
      v[4 * i + 2] = __uint_as_float(w[i].z), v[4 * i + 3] = __uint_as_float(w[i].w);
    }
  }
}

// Even CTAs store K, odd ones V, side by side: one computes, the other copies.
// Five CTAs an SM hide the loads (32768 tokens x 8 heads x 128: 38.0 us, 4.4
// TB/s; 41 with four, 43.3 with resident CTAs that load ahead into registers).
template <bool BF16, int D>
__global__ void __launch_bounds__(256, 5) kv4_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 32;                               // lanes per row
  static_assert(LPR == 2 || LPR == 4, "head sizes 64 and 128");
  grid_dependency_sync();
  const int which = blockIdx.x & 1;                         // 0: K, 1: V
  const uint32_t row = (blockIdx.x >> 1) * (256 / LPR) + threadIdx.x / LPR;
  const int part = threadIdx.x % LPR;
  const bool live = row < a.rows;
  const uint32_t token = live ? a.kv_heads(row) : 0;
  const int head = live ? static_cast<int>(row - token * a.kv_heads.d) : 0;
  const int64_t slot = live ? a.slots[token] : -1;
  float v[32];
  if (live) {
    load32<BF16>(a.x[which], static_cast<int64_t>(token) * a.stride[which] + static_cast<int64_t>(head) * D + part * 32, v);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
  }
  if (slot >= a.num_slots && part == 0) atomicOr(&hadq_kv4_fault, kFaultSlot);
  float norm = 1.f;
  if (which == 0 && a.rotate_k) {
    norm = a.norm;
    fwht_bits<32, 0, 5>(v);
#pragma unroll
    for (int b = 1; b < LPR; b <<= 1) {
      const float sgn = (part & b) ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {         // v + o or o - v: one rounding either way
        const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v[i], b), __shfl_xor_sync(0xffffffffu, v[i + 1], b));
        const float2 y = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(sgn, sgn), o);
        v[i] = y.x;
        v[i + 1] = y.y;
      }
    }
  }
  float m = absmax_regs(v, 0, 32);
  if (a.group >= 64) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (a.group >= 128) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (slot < 0 || slot >= a.num_slots) return;
  const float s32 = __fdiv_rn(__fmul_rn(m, norm), 7.0f);
  const __half s16 = __float2half_rn(s32 > 65504.f ? 65504.f : s32);      // a NaN stays one
  const float s = __half2float(s16);
  const float f = s > 0.f ? __fdiv_rn(norm, s) : 0.f;
  const uint32_t page = a.page_size(static_cast<uint32_t>(slot));
  const uint32_t off = static_cast<uint32_t>(slot) - page * a.page_size.d;
  const int64_t cell = static_cast<int64_t>(page * static_cast<uint64_t>(a.kv_heads.d) + head) * a.page_size.d + off;
  uint4 w;
  if (m * f < 7.25f)
    w = make_uint4(pack_int4x8<false>(v, 0, f), pack_int4x8<false>(v, 8, f), pack_int4x8<false>(v, 16, f), pack_int4x8<false>(v, 24, f));
  else
    w = make_uint4(int4_codes8(v, f), int4_codes8(v + 8, f), int4_codes8(v + 16, f), int4_codes8(v + 24, f));
  *reinterpret_cast<uint4*>(a.codes[which] + cell * (D / 2) + part * 16) = w;
  const int lanes = a.group / 32;                           // lanes per group
  if (part % lanes == 0) a.scales[which][cell * (D / a.group) + part / lanes] = s16;
}

// ---------------------------------------------------------------- attention
//
//   s_j = scale (q H) . k_j,  p_j = exp(s_j - max),  out = sum p_j v_j / sum p_j
//
// over the positions j that a query sees; K is cached rotated, and since
// H / sqrt(D) is orthonormal the query is rotated the same way here, once per
// CTA, instead of unrotating K.
//
// The cache is read once: one byte per K, V pair of codes, against 4 products
// per query row.  Reading it is the floor; what this kernel spends its time on
// is the unpacking of nibbles (half the integer pipe) and the latency of a
// warp's chain of products, maximum, exponentials and products.
//
// A warp takes steps of two tiles of 16 positions and computes S^T = K q^T and
// O^T = V^T P^T with 16 x 8 matrix instructions, positions and head elements on
// the side of 16, query rows on the side of 8, so that the 1 .. 8 rows of a
// group of heads fill the product.  The order of a contraction is free, so every
// thread reads whole words of codes from shared memory and uses the nibbles
// where they lie:
//   K, one scale per row: a nibble in the upper half of a byte is the signed
//     byte 16 code, two operations for eight of them; q goes in as two digits of
//     8 bits, and the sums are exact integers (m16n8k32).
//   K with more scales, V: nibbles in the low bits of 16-bit halves are fp16
//     subnormals, (code + 8) 2^-24, taken as they are (m16n8k16).  The 8 comes off
//     K's sums as a constant of the query row; off V's sums every fourth step
//     (one more product gives the sum of P), or code by code with more scales.
// P^T comes out of S^T by a transposition of 8 x 8 blocks (movmatrix).  Tiles
// reach shared memory by 16-byte asynchronous copies, two steps ahead of use,
// each warp in a ring of its own: the loop has no block-wide barrier.
//
// Measured (device time): 16 sequences x 32 heads x 3584 .. 4096 positions, 128
// wide, one scale per row: 56 us, 4.65 TB/s of codes and scales.  When it took
// 53.6 (a tile of rows had one unit, sequences no order), the fp16 form of K's
// products took 60.5 us, one tile a step 73, V's 8 taken off by products of its
// own 65, 24 warps instead of 16 (fewer registers) 64.  With its copies taken out
// the loop still takes 49: it is bound by issue, not by memory.
//
// Rounding: q to 2^-15 of its row's largest value (digits) or to fp16, P to
// fp16 (2^-11 relative; the running maximum bounds it by 2^8).  Codes are exact,
// scales multiply in fp32, and sums, maxima and the output accumulate in fp32.
//
// V's scales multiply P.  To keep P within fp16 whatever they are, the
// running maximum is taken over s_j + log2(scale of v_j) (in the base-2
// domain), not over s_j.

struct AttnArgs {
  const uint16_t* q;         // row (b, i, head) at q + (b * q_len + i) * q_stride + head * D
  int64_t q_stride;
  const uint8_t* k_codes;
  const __half* k_scales;
  const uint8_t* v_codes;
  const __half* v_scales;
  const int32_t* table;      // [batch][max_pages]
  const int32_t* lengths;    // [batch]
  uint16_t* out;             // [batch][q_len][heads][D]
  float* part_o;             // [split][unit][rows of a tile][D] (splits > 1)
  float2* part_ml;           // [split][unit][rows of a tile]: maximum, sum
  int64_t num_pages;
  int max_pages, page_size;
  int q_len;
  Divider kv_heads, ratio;   // heads = kv_heads * ratio
  Divider row_tiles;
  Divider blocks;            // page_size / 16
  int units, splits;
  int sorted;                // sequences, to be taken longest first; 0: as they come
  int rotate;
  float norm;                // fp32(1 / sqrt(D))
  float scale_log2;          // scale * log2(e)
};

constexpr int kWarps = 4;
constexpr float kLowest = -3.0e38f;           // no maximum yet: finite, so that its differences are numbers

// A step is two tiles: 32 positions whose products, maximum and exponentials
// interleave.
template <int D, int GROUP, int NT, int STAGES>
struct Cfg {
  static constexpr int G = D / GROUP;
  static constexpr int CODE_BYTES = 16 * D / 2;             // one tile's codes of K or V
  static constexpr int SCALE_BYTES = 16 * G * 2;
  static constexpr int STAGE_BYTES = 4 * (CODE_BYTES + SCALE_BYTES);   // K0 K1 V0 V1, then their scales
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;   // per warp
  static constexpr int ROWS = 8 * NT;
  static constexpr int JOIN_STRIDE = D + 4;                 // floats per row of a warp's partial output
  static constexpr int JOIN_BYTES = kWarps * ROWS * (JOIN_STRIDE + 2) * 4;
  static constexpr int MAIN_BYTES = kWarps * RING_BYTES;
  static constexpr int BUF_BYTES = MAIN_BYTES > JOIN_BYTES ? MAIN_BYTES : JOIN_BYTES;
  static constexpr int Q_AT = BUF_BYTES;                    // query rows as operands, and their units
  static constexpr int Q_BYTES = ROWS * D * 2;
  static constexpr int VALID_AT = Q_AT + Q_BYTES + ROWS * 4;   // valid positions of the tiles in flight
  static constexpr int SMEM_BYTES = VALID_AT + kWarps * STAGES * 8;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same of bytes, 32 deep: signed K times signed or unsigned digits of q.
template <bool SIGNED>
__device__ __forceinline__ void mma16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (SIGNED)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with sums that start at 0.
template <bool SIGNED>
__device__ __forceinline__ void mma16832_from0(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  if constexpr (SIGNED)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float log2_fast(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return h2_bits(__floats2half2_rn(lo, hi)); }

// Nibbles 0, 1, 2, 3 of both halves of w as fp16 pairs, without arithmetic: the
// low bits of an fp16 number with a zero exponent are a subnormal, which the
// products take exactly.  x[0], x[2]: (code + 8) 2^-24; x[1], x[3]: 16 times
// that.
__device__ __forceinline__ uint32_t mask_flip(uint32_t w, uint32_t mask, uint32_t flip) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(mask), "r"(flip));   // (w & mask) ^ flip
  return r;
}
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t (&x)[4]) {
  const uint32_t u = w >> 8;
  x[0] = mask_flip(w, 0x000F000Fu, 0x00080008u);
  x[1] = mask_flip(w, 0x00F000F0u, 0x00800080u);
  x[2] = mask_flip(u, 0x000F000Fu, 0x00080008u);
  x[3] = mask_flip(u, 0x00F000F0u, 0x00800080u);
}

// Byte offset of 16-byte chunk `ch` of position t in a tile's codes.  The XOR
// spreads the chunks that one load instruction reads over the banks: K with
// one scale a row is read 16 (or 8) bytes a lane and needs none; with more
// scales chunk by chunk for positions 0..7 at once, V for four at once.
template <int D, int G>
__device__ __forceinline__ int k_chunk(int t, int ch) {
  if constexpr (G == 1) return t * (D / 2) + (ch << 4);
  else if constexpr (D == 128) return t * 64 + ((ch ^ ((t >> 1) & 3)) << 4);
  else return t * 32 + ((ch ^ ((t >> 2) & 1)) << 4);
}
template <int D>
__device__ __forceinline__ int v_chunk(int t, int ch) {
  if constexpr (D == 128) return t * 64 + ((ch ^ (t & 2)) << 4);
  else return t * 32 + (ch << 4);
}

constexpr uint32_t kNoTile = 0xFFFFFFFFu;     // a page outside the cache

// A step's copies where a sequence ends or a page lies outside the cache: zeros
// in place of what must not be read (the positions are masked).  Out of line:
// the loop's code stays short.
template <int D, int G>
__device__ __noinline__ void copy_partial(uint32_t dst, const uint8_t* k_lane, const uint8_t* v_lane, const uint8_t* s_lane,
                                          uint32_t e0, uint32_t e1, int n0, int n1) {
  constexpr int NG = D / 32, CODE_BYTES = 8 * D, SCALE_BYTES = 32 * G;
  const int lane = threadIdx.x & 31;
  const uint64_t f0 = e0 == kNoTile ? 0 : e0, f1 = e1 == kNoTile ? 0 : e1;
  for (int u = 0; u < D / 64; ++u) {
    const int j = lane + 32 * u, t = j / NG, b0 = t < n0 ? 16 : 0, b1 = t < n1 ? 16 : 0;
    const uint32_t k = dst + k_chunk<D, G>(t, j % NG), v = dst + 2 * CODE_BYTES + v_chunk<D>(t, j % NG);
    cp_async16(k, k_lane + f0 * CODE_BYTES + 512 * u, b0);
    cp_async16(k + CODE_BYTES, k_lane + f1 * CODE_BYTES + 512 * u, b1);
    cp_async16(v, v_lane + f0 * CODE_BYTES + 512 * u, b0);
    cp_async16(v + CODE_BYTES, v_lane + f1 * CODE_BYTES + 512 * u, b1);
  }
  const int bytes = min(max((lane < 16 ? n0 : n1) * 2 * G - 16 * (lane & 7), 0), 16);
  if ((lane & 7) < 2 * G)
    cp_async16(dst + 4 * CODE_BYTES + ((lane >> 4) + ((lane & 8) ? 2 : 0)) * SCALE_BYTES + 16 * (lane & 7),
               s_lane + (lane < 16 ? f0 : f1) * SCALE_BYTES, bytes);
}

__device__ __forceinline__ int length_of(const AttnArgs& a, int b) {
  const int n = a.lengths[b], most = a.max_pages * a.page_size;
  return n < 0 ? 0 : n > most ? most : n;
}

// The sequence whose turn is `turn` when runs of 64 sequences go in order of
// their lengths, the longest first: more CTAs than the GPU holds then end with
// short ones.  Two threads to a sequence count those before it; runs of 256,
// eight times the counting, cost what they gained (300 sequences of about 750:
// 109 us, in no order 77).
__device__ __forceinline__ int by_length(const AttnArgs& a, int turn, int* lens) {
  constexpr int kRun = 16 * kWarps;
  __shared__ int chosen;
  const int first = turn & ~(kRun - 1), n = min(kRun, a.sorted - first);
  if (threadIdx.x < kRun) lens[threadIdx.x] = threadIdx.x < n ? a.lengths[first + threadIdx.x] : INT_MIN;
  __syncthreads();
  const int s = threadIdx.x >> 1, half = threadIdx.x & 1, mine = lens[s];
  int before = 0;
#pragma unroll
  for (int j = 0; j < kRun / 2; j += 4) {       // (length, place) is an order of all of them
    const int i = half * (kRun / 2) + j;
    const int4 x = *reinterpret_cast<const int4*>(lens + i);
    before += (x.x > mine || (x.x == mine && i < s)) + (x.y > mine || (x.y == mine && i + 1 < s)) +
              (x.z > mine || (x.z == mine && i + 2 < s)) + (x.w > mine || (x.w == mine && i + 3 < s));
  }
  before += __shfl_xor_sync(0xffffffffu, before, 1);
  if (before == turn - first && s < n) chosen = first + s;
  __syncthreads();                              // and `lens` is free again
  return chosen;
}

// Division of the work.  A unit is a (sequence, K/V head, tile of query rows);
// CTA (unit, split) takes the split's equal part of the sequence's steps, the
// longest sequences first where that shortens the grid's end (longest_first).  With
// more than one split the parts' sums go to the workspace, and kv4_join_kernel
// adds them in order.
template <int D, int GROUP, int NT, int STAGES>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 4 : 2) kv4_attention_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, GROUP, NT, STAGES>;
  constexpr int G = C::G;
  constexpr int NG = D / 32;                  // words of a row that one lane reads of K
  constexpr int MT = D / 16;                  // 16-element tiles of the output
  constexpr int TPG = GROUP / 16;             // of them in a scale group
  constexpr int TILE_SCALES = 32 * G;         // bytes of a tile's scales
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * C::RING_BYTES;
  int2* nvalid = reinterpret_cast<int2*>(smem + C::VALID_AT) + warp * STAGES;

  grid_dependency_sync();
  const int ratio = a.ratio.d, rows = a.q_len * ratio;
  const int split = blockIdx.y;
  const int turn = static_cast<int>(a.row_tiles(blockIdx.x)), rt = blockIdx.x - turn * a.row_tiles.d;
  int b = static_cast<int>(a.kv_heads(turn));
  const int h = turn - b * a.kv_heads.d;
  if (a.sorted > 0) b = by_length(a, b, reinterpret_cast<int*>(smem));
  const int unit = (b * a.kv_heads.d + h) * a.row_tiles.d + rt;
  // the query's values, on their way while the length and the page table are read
  constexpr int LPR = D / 8, PASS = kWarps * 32 / LPR;        // lanes per row, rows of a pass of all warps
  constexpr int PASSES = (C::ROWS + PASS - 1) / PASS;
  uint4 qraw[PASSES];
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    const int row = ps * PASS + threadIdx.x / LPR, rho = rt * C::ROWS + row;
    qraw[ps] = make_uint4(0u, 0u, 0u, 0u);
    if (row < C::ROWS && rho < rows) {
      const int i = static_cast<int>(a.ratio(rho)), head = h * ratio + rho - i * ratio;
      qraw[ps] = ld_stream(reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(b) * a.q_len + i) * a.q_stride +
                                                           static_cast<int64_t>(head) * D + 8 * (threadIdx.x % LPR)));
    }
  }
  const int len = length_of(a, b);
  if (threadIdx.x == 0 && len != a.lengths[b]) atomicOr(&hadq_kv4_fault, kFaultLength);
  const int64_t part = (static_cast<int64_t>(split) * a.units + unit) * C::ROWS;   // first row in the workspace
  const int steps = (len + 31) >> 5, per = (steps + a.splits - 1) / a.splits;
  const int t0 = min(split * per, steps), count = min(per, steps - t0);
  if (a.splits > 1 && count == 0) {             // nothing here: no part (the join skips sums of 0)
    if (threadIdx.x < C::ROWS) a.part_ml[part + threadIdx.x] = make_float2(kLowest, 0.f);
    return;
  }
  const int mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;   // steps, interleaved over the warps

  // ---- copies.  Lane l holds the entry of tile l & 1 of the warp's step
  // i0 + l / 2: the number of the 16-position run in the cache (fewer than
  // 2^32: a run takes 512 bytes or more), or kNoTile for a page outside it.
  uint32_t entry = kNoTile;
  auto load_entries = [&](int i0) {
    const int tile = (t0 + warp + (i0 + (lane >> 1)) * kWarps) * 2 + (lane & 1);
    entry = kNoTile;
    if (tile * 16 < len) {
      const int p = static_cast<int>(a.blocks(tile));
      const int page = a.table[static_cast<int64_t>(b) * a.max_pages + p];
      if (page < 0 || page >= a.num_pages) atomicOr(&hadq_kv4_fault, kFaultPage);
      else entry = (static_cast<uint32_t>(page) * a.kv_heads.d + h) * a.blocks.d + (tile - p * a.blocks.d);
    }
  };
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  // this lane's 16-byte chunks: of codes, `lane` and (D = 128) lane + 32 of a
  // tile; of scales, chunk lane & 7 of K (lane bit 3: V) of tile lane / 16
  const uint8_t* k_lane = a.k_codes + 16 * lane;
  const uint8_t* v_lane = a.v_codes + 16 * lane;
  const uint8_t* s_lane = reinterpret_cast<const uint8_t*>((lane & 8) ? a.v_scales : a.k_scales) + 16 * (lane & 7);
  const bool s_live = (lane & 7) < 2 * G;
  const uint32_t s_dst = ring_u + 4 * C::CODE_BYTES + ((lane >> 4) + ((lane & 8) ? 2 : 0)) * C::SCALE_BYTES + 16 * (lane & 7);
  uint32_t k_dst[D / 64], v_dst[D / 64];
#pragma unroll
  for (int u = 0; u < D / 64; ++u) {
    const int j = lane + 32 * u;
    k_dst[u] = ring_u + k_chunk<D, G>(j / NG, j % NG);
    v_dst[u] = ring_u + 2 * C::CODE_BYTES + v_chunk<D>(j / NG, j % NG);
  }
  auto issue = [&](int i, int stage) {
    if (i < mine) {
      if ((i & 15) == 0) load_entries(i);
      const uint32_t e0 = __shfl_sync(0xffffffffu, entry, (i & 15) * 2), e1 = __shfl_sync(0xffffffffu, entry, (i & 15) * 2 + 1);
      const uint32_t st = stage * C::STAGE_BYTES;
      const int left = len - (t0 + warp + i * kWarps) * 32;
      const uint32_t es = lane < 16 ? e0 : e1;
      if (left >= 32 && e0 != kNoTile && e1 != kNoTile) {
        if (lane == 0) nvalid[stage] = make_int2(16, 16);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
          cp_async16(st + k_dst[u], k_lane + static_cast<uint64_t>(e0) * C::CODE_BYTES + 512 * u);
          cp_async16(st + k_dst[u] + C::CODE_BYTES, k_lane + static_cast<uint64_t>(e1) * C::CODE_BYTES + 512 * u);
          cp_async16(st + v_dst[u], v_lane + static_cast<uint64_t>(e0) * C::CODE_BYTES + 512 * u);
          cp_async16(st + v_dst[u] + C::CODE_BYTES, v_lane + static_cast<uint64_t>(e1) * C::CODE_BYTES + 512 * u);
        }
        if (s_live) cp_async16(st + s_dst, s_lane + static_cast<uint64_t>(es) * TILE_SCALES);
      } else {
        const int n0 = e0 == kNoTile ? 0 : min(16, left), n1 = e1 == kNoTile ? 0 : min(16, max(left - 16, 0));
        if (lane == 0) nvalid[stage] = make_int2(n0, n1);
        copy_partial<D, G>(ring_u + st, k_lane, v_lane, s_lane, e0, e1, n0, n1);
      }
    }
    cp_async_commit();
  };
#pragma unroll 1                              // the code is fetched once
  for (int i = 0; i < STAGES - 1; ++i) issue(i, i);

  // ---- query rows.  A lane's words of a K row, w = 0 .. NG - 1: with one scale
  // per row elements c D / 4 + 8 w .. (consecutive: one load), else 32 w + 8 c ..
  // (every word in a group of its own).  D / 8 lanes rotate a row, 8 elements
  // each, and leave it in the order in which lane (r, c) takes row r.
  uint4* qs = reinterpret_cast<uint4*>(smem + C::Q_AT);       // [row / 8][word][lane]
  float* row_unit = reinterpret_cast<float*>(smem + C::Q_AT + C::Q_BYTES);
  float v[PASSES][8], f = a.scale_log2;
  if (a.rotate) f *= a.norm;
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    const int part8 = threadIdx.x % LPR;
    const uint4 w = qraw[ps];
    unpack_bf16x2(w.x, v[ps][0], v[ps][1]);
    unpack_bf16x2(w.y, v[ps][2], v[ps][3]);
    unpack_bf16x2(w.z, v[ps][4], v[ps][5]);
    unpack_bf16x2(w.w, v[ps][6], v[ps][7]);
    if (a.rotate) {
      fwht_bits<8, 0, 3>(v[ps]);
#pragma unroll
      for (int s = 1; s < LPR; s <<= 1) {
        const float sgn = (part8 & s) ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[ps][i] = fmaf(v[ps][i], sgn, __shfl_xor_sync(0xffffffffu, v[ps][i], s));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[ps][i] *= f;
  }
#pragma unroll
  for (int ps = 0; ps < PASSES; ++ps) {
    const int row = ps * PASS + threadIdx.x / LPR, part8 = threadIdx.x % LPR;
    const int w = G == 1 ? part8 % NG : part8 / 4, qc = G == 1 ? part8 / NG : part8 % 4;
    // a row of its own size: 2^e <= its largest value < 2^(e + 1).  Magnitudes
    // compare as integers, and so do infinities and NaNs, which max would drop.
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(v[ps][i]) & 0x7fffffffu);
#pragma unroll
    for (int s = 1; s < LPR; s <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const int eb = min(max(static_cast<int>(mx >> 23), 16), 220);
    const float up = __uint_as_float(static_cast<uint32_t>(eb) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(254 - eb) << 23);
    uint4 x;
    if constexpr (G == 1) {
      // digits of round(q 2^14 / 2^e) = 256 high + low: even elements' high
      // ones, odd ones', then the low ones
      uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = min(max(__float2int_rn(v[ps][i] * down * 16384.f), -32768), 32767);
        hi[i & 1] |= (static_cast<uint32_t>(q >> 8) & 255u) << (8 * (i >> 1));
        lo[i & 1] |= (static_cast<uint32_t>(q) & 255u) << (8 * (i >> 1));
      }
      x = make_uint4(hi[0], hi[1], lo[0], lo[1]);
    } else {
      // fp16 pairs, in the units of K's nibbles
      x.x = pack_half2(v[ps][0] * down, v[ps][4] * down);
      x.y = pack_half2(v[ps][1] * (down * 0.0625f), v[ps][5] * (down * 0.0625f));
      x.z = pack_half2(v[ps][2] * down, v[ps][6] * down);
      x.w = pack_half2(v[ps][3] * (down * 0.0625f), v[ps][7] * (down * 0.0625f));
    }
    if (row < C::ROWS) {
      qs[((row >> 3) * NG + w) * 32 + (row & 7) * 4 + qc] = x;
      // of its products' sums; no number for a row that is none, or beyond 2^94
      if (part8 == 0) row_unit[row] = (mx >> 23) > 220u ? __uint_as_float(0x7fc00000u) : up * (G == 1 ? 1.f / 262144.f : 16777216.f);
    }
  }
  __syncthreads();
  uint4 qb[NT == 1 ? NG : 1];                 // one tile of rows: in registers; two: read at each use
  auto query = [&](int nt, int w) { return NT == 1 ? qb[w] : qs[(nt * NG + w) * 32 + lane]; };
  float bias[NT][G][2];                       // G > 1: what the 8 in (code + 8) adds to a row's sums, negative
  float qf[NT][2];                            // units of the sums of rows 2c, 2c + 1
  int limit[NT][2];                           // first position that they do not see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float eight[4] = {0.f, 0.f, 0.f, 0.f};  // equal for every row of the product
#pragma unroll
      for (int w = g * (GROUP / 32); w < (g + 1) * (GROUP / 32); ++w) {
        const uint4 x = qs[(nt * NG + w) * 32 + lane];
        if constexpr (NT == 1) qb[w] = x;
        if constexpr (G > 1) {
          mma16816(eight, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, x.x, x.y);
          mma16816(eight, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, x.z, x.w);
        }
      }
      bias[nt][g][0] = eight[0];
      bias[nt][g][1] = eight[1];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = rt * C::ROWS + nt * 8 + 2 * c + e;
      limit[nt][e] = len - a.q_len + 1 + static_cast<int>(a.ratio(col));
      qf[nt][e] = row_unit[nt * 8 + 2 * c + e];
    }
  }

  float o[MT][NT][4];
  float m[NT][2], l[NT][2];
  float ones[NT][4];                          // G == 1: 8 times P's sums, in the units of even and odd nibbles
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) m[nt][e] = kLowest, l[nt][e] = 0.f, ones[nt][e] = ones[nt][2 + e] = 0.f;

  // positions below this are seen by every row of the tile
  const int seen_by_all = len - a.q_len + 1 + static_cast<int>(a.ratio(rt * C::ROWS));

  // Row i of a tile's products is position pi(i): pi(2c) = c, pi(2c + 1) = 4 +
  // (c ^ 1), pi(i + 8) = pi(i) + 8.  The four lanes c then read four
  // neighbouring positions of V at a time, and lanes r, r + 1 positions of K
  // that differ in their lowest bit (different banks).
  const int pr = (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1;   // pi(r)
  int k_at[G == 1 ? 1 : NG], v_at[G][2];      // this lane's words in a tile
  if constexpr (G == 1) {
    k_at[0] = pr * (D / 2) + c * (D / 8);
  } else {
#pragma unroll
    for (int w = 0; w < NG; ++w) k_at[w] = k_chunk<D, G>(pr, w) + 4 * c;
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = e ? 4 + (c ^ 1) : c;
      if constexpr (GROUP == 128) v_at[g][e] = v_chunk<D>(t, r >> 1) + (r & 1) * 8;
      else if constexpr (GROUP == 64) v_at[g][e] = v_chunk<D>(t, 2 * g + (r >> 2)) + (r & 3) * 4;
      else v_at[g][e] = v_chunk<D>(t, g) + r * 2;
    }

  int stage = 0;
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    issue(i + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);   // the stage consumed in the last round
    const uint8_t* kt = ring + stage * C::STAGE_BYTES;
    const uint8_t* vt = kt + 2 * C::CODE_BYTES;
    const __half* kst = reinterpret_cast<const __half*>(kt + 4 * C::CODE_BYTES) + pr * G;
    const __half* vst = kst + 32 * G;
    const int2 nv = nvalid[stage];
    stage = stage == STAGES - 1 ? 0 : stage + 1;
    const int pos = (t0 + warp + i * kWarps) * 32;

    // ---- S^T = K q^T: s times kk are the base-2 scores
    float s[2][NT][4], kk[2][2];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float acc[2][NT][4];
      uint32_t kw[2][2][GROUP / 32];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* at = kt + tt * C::CODE_BYTES + e * (C::CODE_BYTES / 2);
          if constexpr (G == 1 && D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(at + k_at[0]);
            kw[tt][e][0] = x.x, kw[tt][e][1] = x.y, kw[tt][e][2] = x.z, kw[tt][e][3] = x.w;
          } else if constexpr (G == 1) {
            const uint2 x = *reinterpret_cast<const uint2*>(at + k_at[0]);
            kw[tt][e][0] = x.x, kw[tt][e][1] = x.y;
          } else {
#pragma unroll
            for (int w = 0; w < GROUP / 32; ++w) kw[tt][e][w] = *reinterpret_cast<const uint32_t*>(at + k_at[g * (GROUP / 32) + w]);
          }
        }
      if constexpr (G == 1) {
        int high[2][NT][4], low[2][NT][4];
#pragma unroll
        for (int w = 0; w < NG; ++w)
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) {
            // a nibble in the upper half of a byte is the signed byte 16 code
            const uint32_t a0 = (kw[tt][0][w] << 4) & 0xF0F0F0F0u, a2 = kw[tt][0][w] & 0xF0F0F0F0u;
            const uint32_t a1 = (kw[tt][1][w] << 4) & 0xF0F0F0F0u, a3 = kw[tt][1][w] & 0xF0F0F0F0u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 q = query(nt, w);
              if (w == 0) {
                mma16832_from0<true>(high[tt][nt], a0, a1, a2, a3, q.x, q.y);
                mma16832_from0<false>(low[tt][nt], a0, a1, a2, a3, q.z, q.w);
              } else {
                mma16832<true>(high[tt][nt], a0, a1, a2, a3, q.x, q.y);
                mma16832<false>(low[tt][nt], a0, a1, a2, a3, q.z, q.w);
              }
            }
          }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[tt][nt][k] = __int2float_rn(high[tt][nt][k] * 256 + low[tt][nt][k]);
      } else {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[tt][nt][k] = bias[nt][g][k & 1];
#pragma unroll
        for (int w = 0; w < GROUP / 32; ++w)
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) {
            uint32_t xa[4], xb[4];
            unpack4(kw[tt][0][w], xa);
            unpack4(kw[tt][1][w], xb);
            const int gw = g * (GROUP / 32) + w;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 q = query(nt, gw);
              mma16816(acc[tt][nt], xa[0], xb[0], xa[1], xb[1], q.x, q.y);
              mma16816(acc[tt][nt], xa[2], xb[2], xa[3], xb[3], q.z, q.w);
            }
          }
      }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        float k2[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          k2[e] = __half2float(kst[tt * 16 * G + 8 * e * G + g]);
          kk[tt][e] = G == 1 ? k2[e] : 1.f;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            s[tt][nt][k] = G == 1 ? acc[tt][nt][k] * qf[nt][k & 1]
                           : g == 0 ? acc[tt][nt][k] * k2[k >> 1]
                                    : fmaf(acc[tt][nt][k], k2[k >> 1], s[tt][nt][k]);
      }
    }
    if constexpr (G > 1) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[tt][nt][k] *= qf[nt][k & 1];
    }
    // V's scales of this lane's four positions, and log2 of the largest of each
    float sv[2][2][G], lv[2][2];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int g = 0; g < G; ++g) sv[tt][e][g] = __half2float(vst[tt * 16 * G + 8 * e * G + g]);
    const bool masked = nv.x + nv.y < 32 || pos + 32 > seen_by_all;
    float none[2][2] = {};
    if (masked) {
      // finite scales, so that a position that a row does not see adds 0 whatever
      // lies there; the score of a row that does see it takes the NaN
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 0; g < G; ++g) none[tt][e] = fmaf(sv[tt][e][g], 0.f, none[tt][e]);
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 0; g < G; ++g) sv[tt][e][g] = fminf(fmaxf(sv[tt][e][g], -65504.f), 65504.f);
    }
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fabsf(sv[tt][e][0]);
#pragma unroll
        for (int g = 1; g < G; ++g) top = fmaxf(top, fabsf(sv[tt][e][g]));
        lv[tt][e] = fminf(fmaxf(log2_fast(top), -24.f), 16.f);   // fp16 above zero: 2^-24 to 2^16
      }
    if (masked) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = pr + 8 * (k >> 1);
          const bool there = at < (tt ? nv.y : nv.x);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            s[tt][nt][k] = there && pos + 16 * tt + at < limit[nt][k & 1] ? fmaf(s[tt][nt][k], kk[tt][k >> 1], none[tt][k >> 1])
                                                                                : -INFINITY;
        }
        kk[tt][0] = kk[tt][1] = 1.f;
      }
    }
    // The running maximum moves only when a value passes it by 2^8: P stays
    // below 2^8, and most steps need one vote instead of the exchange.
    float up[NT][2];
    bool rise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        up[nt][e] = fmaxf(fmaxf(fmaf(s[0][nt][e], kk[0][0], lv[0][0]), fmaf(s[0][nt][2 + e], kk[0][1], lv[0][1])),
                          fmaxf(fmaf(s[1][nt][e], kk[1][0], lv[1][0]), fmaf(s[1][nt][2 + e], kk[1][1], lv[1][1])));
        rise |= up[nt][e] > m[nt][e] + 8.f;
      }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = up[nt][e];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          t = t > m[nt][e] + 8.f ? t : m[nt][e];     // no row depends on its neighbours' sizes
          const float f = exp2_fast(m[nt][e] - t);
          m[nt][e] = t;
          l[nt][e] *= f;
          ones[nt][e] *= f;
          ones[nt][2 + e] *= f;
#pragma unroll
          for (int k = 0; k < MT; ++k) {
            o[k][nt][e] *= f;
            o[k][nt][2 + e] *= f;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          s[tt][nt][e] = exp2_fast(fmaf(s[tt][nt][e], kk[tt][0], -m[nt][e]));
          s[tt][nt][2 + e] = exp2_fast(fmaf(s[tt][nt][2 + e], kk[tt][1], -m[nt][e]));
        }
        l[nt][e] += (s[0][nt][e] + s[0][nt][2 + e]) + (s[1][nt][e] + s[1][nt][2 + e]);
      }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[nt][0] = transpose8x8(pack_half2(s[tt][nt][0] * sv[tt][0][g], s[tt][nt][1] * sv[tt][0][g]));
          pb[nt][1] = transpose8x8(pack_half2(s[tt][nt][2] * sv[tt][1][g], s[tt][nt][3] * sv[tt][1][g]));
        }
        if constexpr (G == 1) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(ones[nt], 0x00080008u, 0x00800080u, 0x00080008u, 0x00800080u, pb[nt][0], pb[nt][1]);
        }
        // lane (r, c): elements g GROUP + r GROUP / 8 + 0..GROUP / 8 - 1 of positions pi(2c), pi(2c + 1), + 8
        uint32_t w[4][2];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint8_t* at = vt + tt * C::CODE_BYTES + (t >> 1) * (C::CODE_BYTES / 2) + v_at[g][t & 1];
          if constexpr (GROUP == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            w[t][0] = x.x;
            w[t][1] = x.y;
          } else if constexpr (GROUP == 64) {
            w[t][0] = *reinterpret_cast<const uint32_t*>(at);
          } else {
            w[t][0] = *reinterpret_cast<const uint16_t*>(at);
          }
        }
#pragma unroll
        for (int q4 = 0; q4 < TPG / 2; ++q4) {    // four nibbles, two tiles of the output at a time
          const uint32_t sel = (q4 & 1) ? 0x7632u : 0x5410u;
          uint32_t xa[4], xb[4];
          unpack4(__byte_perm(w[0][q4 >> 1], w[1][q4 >> 1], sel), xa);
          unpack4(__byte_perm(w[2][q4 >> 1], w[3][q4 >> 1], sel), xb);
          if constexpr (G > 1) {
            // the 8 leaves each code here (below, it would take sums for every scale)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2 e8 = bits_h2((j & 1) ? 0x00800080u : 0x00080008u);
              xa[j] = h2_bits(__hsub2(bits_h2(xa[j]), e8));
              xb[j] = h2_bits(__hsub2(bits_h2(xb[j]), e8));
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float(&o0)[4] = o[g * TPG + 2 * q4][nt], (&o1)[4] = o[g * TPG + 2 * q4 + 1][nt];
            mma16816(o0, xa[0], xa[1], xb[0], xb[1], pb[nt][0], pb[nt][1]);
            mma16816(o1, xa[2], xa[3], xb[2], xb[3], pb[nt][0], pb[nt][1]);
          }
        }
      }
    // The 8 in (code + 8) leaves the sums every fourth step: before it outgrows them.
    if (G == 1 && ((i & 3) == 3 || i == mine - 1)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int t = 0; t < MT; ++t) o[t][nt][k] -= ones[nt][k];
          ones[nt][k] = 0.f;
        }
    }
  }
  cp_async_wait<0>();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);

  // ---- join the warps: partial outputs through shared memory, warps in order
  __syncthreads();                            // every ring is drained
  float* jo = reinterpret_cast<float*>(smem);                       // [warp][row][JOIN_STRIDE]
  float2* jml = reinterpret_cast<float2*>(jo + kWarps * C::ROWS * C::JOIN_STRIDE);   // [warp][row]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = nt * 8 + 2 * c + e;
      float* dst = jo + (warp * C::ROWS + row) * C::JOIN_STRIDE + r * (GROUP / 8);
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int t = 0; t < TPG; t += 2) {      // even nibbles in units of 2^-24, odd ones 2^-20
          const float(&x)[4] = o[g * TPG + t][nt], (&y)[4] = o[g * TPG + t + 1][nt];
          *reinterpret_cast<float4*>(dst + g * GROUP + 2 * t) =
              make_float4(x[e] * 16777216.f, x[2 + e] * 1048576.f, y[e] * 16777216.f, y[2 + e] * 1048576.f);
        }
      if (r == 0) jml[warp * C::ROWS + row] = make_float2(m[nt][e], l[nt][e]);
    }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < C::ROWS * (D / 4); i += 32 * kWarps) {
    const int row = i / (D / 4), d = (i % (D / 4)) * 4;
    const int rho = rt * C::ROWS + row;
    if (rho >= rows) continue;
    float2 ml[kWarps];
    float top = kLowest, sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ml[w] = jml[w * C::ROWS + row];
      top = fmaxf(top, ml[w].x);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2_fast(ml[w].x - top);
      const float4 x = *reinterpret_cast<const float4*>(jo + (w * C::ROWS + row) * C::JOIN_STRIDE + d);
      sum = fmaf(ml[w].y, f, sum);
      y = make_float4(fmaf(x.x, f, y.x), fmaf(x.y, f, y.y), fmaf(x.z, f, y.z), fmaf(x.w, f, y.w));
    }
    if (a.splits == 1) {
      const int qi = static_cast<int>(a.ratio(rho));
      const int64_t orow = (static_cast<int64_t>(b) * a.q_len + qi) * (a.kv_heads.d * ratio) + h * ratio + rho - qi * ratio;
      const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);     // a row that sees nothing: zeros
      *reinterpret_cast<uint2*>(a.out + orow * D + d) = make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
    } else {
      *reinterpret_cast<float4*>(a.part_o + (part + row) * D + d) = y;
      if (d == 0) a.part_ml[part + row] = make_float2(top, sum);
    }
  }
}

// Adds the splits' parts, one CTA per unit: one to kPieces warps a row
// (blockDim.x), each its share of the splits in order, then the shares in order.
template <int ROWS>
constexpr int kPieces = ROWS == 8 ? 4 : 2;

template <int D, int ROWS>
__global__ void __launch_bounds__(32 * ROWS * kPieces<ROWS>, 1) kv4_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float part[kPieces<ROWS>][ROWS][D];
  __shared__ float2 part_ml[kPieces<ROWS>][ROWS];
  grid_dependency_sync();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = warp % ROWS, piece = warp / ROWS, pieces = blockDim.x / (32 * ROWS);
  const int unit = blockIdx.x;
  const int bh = static_cast<int>(a.row_tiles(unit)), rt = unit - bh * a.row_tiles.d;
  const int b = static_cast<int>(a.kv_heads(bh)), h = bh - b * a.kv_heads.d;
  const int ratio = a.ratio.d, rho = rt * ROWS + row, qi = static_cast<int>(a.ratio(rho));
  const bool live = rho < a.q_len * ratio;
  const int s0 = a.splits * piece / pieces, s1 = live ? a.splits * (piece + 1) / pieces : s0;
  auto part_row = [&](int s) { return (static_cast<int64_t>(s) * a.units + unit) * ROWS + row; };
  float top = kLowest;
  for (int s = s0 + lane; s < s1; s += 32) top = fmaxf(top, a.part_ml[part_row(s)].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float sum = 0.f, v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = 0.f;
#pragma unroll 8
  for (int s = s0; s < s1; ++s) {
    const int64_t r = part_row(s);
    const float2 ml = a.part_ml[r];
    const float f = exp2_fast(ml.x - top);
    const float* p = a.part_o + r * D + lane * E;
    float y[E];
    if constexpr (E == 4) {
      const float4 x = *reinterpret_cast<const float4*>(p);
      y[0] = x.x, y[1] = x.y, y[2] = x.z, y[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(p);
      y[0] = x.x, y[1] = x.y;
    }
    sum = fmaf(ml.y, f, sum);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = ml.y == 0.f ? v[i] : fmaf(y[i], f, v[i]);   // an empty part was not written
  }
#pragma unroll
  for (int i = 0; i < E; ++i) part[piece][row][lane * E + i] = v[i];
  if (lane == 0) part_ml[piece][row] = make_float2(top, sum);
  __syncthreads();
  if (piece != 0 || !live) return;
  float all = kLowest;
  for (int i = 0; i < pieces; ++i) all = fmaxf(all, part_ml[i][row].x);
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = 0.f;
  for (int q = 0; q < pieces; ++q) {
    const float2 ml = part_ml[q][row];
    const float f = exp2_fast(ml.x - all);
    sum = fmaf(ml.y, f, sum);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = fmaf(part[q][row][lane * E + i], f, v[i]);
  }
  const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.f, sum);
  const int64_t orow = (static_cast<int64_t>(b) * a.q_len + qi) * (a.kv_heads.d * ratio) + h * ratio + rho - qi * ratio;
#pragma unroll
  for (int i = 0; i < E; i += 2)
    *reinterpret_cast<uint32_t*>(a.out + orow * D + lane * E + i) = pack_bf16x2(v[i] * inv, v[i + 1] * inv);
}

}  // namespace kv4
}  // namespace hadq
