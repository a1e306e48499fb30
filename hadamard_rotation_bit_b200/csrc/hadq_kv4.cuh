// A paged cache of int4 keys and values: appending rows to it, and attention
// of a sequence's newest tokens over it.
//
// Cache (one layer): pages of page_size positions, for K and for V
//   codes  [num_pages][kv_heads][page_size][D / 2]      two's-complement nibbles, element 2i low
//   scales [num_pages][kv_heads][page_size][D / GROUP]  fp16
// so 16 consecutive positions of one head are one contiguous run of codes and
// one of scales (page_size is a multiple of 16): the tile of both kernels.
#pragma once

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

struct AppendArgs {
  const void* x[2];          // K, V: row (t, h) at x + t * stride + h * D
  int64_t stride[2];         // elements between tokens
  uint8_t* codes[2];
  __half* scales[2];
  const int64_t* slots;      // position in the cache per token: page * page_size + offset; negative: no row
  int64_t tokens;
  int64_t num_slots;         // num_pages * page_size
  int kv_heads, page_size, group;
  int rotate_k;              // 1: K rotated per head
  float norm;                // fp32(1 / sqrt(D))
};

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

template <bool BF16, int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 32;                               // lanes per row
  static_assert(LPR == 2 || LPR == 4, "head sizes 64 and 128");
  grid_dependency_sync();
  const int which = blockIdx.y;                             // 0: K, 1: V
  const int64_t rows = a.tokens * a.kv_heads;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / LPR;
  const int part = threadIdx.x % LPR;
  const bool live = row < rows;
  const int64_t token = live ? row / a.kv_heads : 0;
  const int head = live ? static_cast<int>(row - token * a.kv_heads) : 0;
  const int64_t slot = live ? a.slots[token] : -1;
  if (live && slot >= a.num_slots && part == 0) atomicOr(&hadq_kv4_fault, kFaultSlot);
  const bool ok = slot >= 0 && slot < a.num_slots;

  float v[32];
  if (ok) {
    load_elems<BF16, 32>(a.x[which], token * a.stride[which] + static_cast<int64_t>(head) * D + part * 32, v);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
  }
  float norm = 1.f;
  if (which == 0 && a.rotate_k) {
    norm = a.norm;
    fwht_bits<32, 0, 5>(v);
#pragma unroll
    for (int b = 1; b < LPR; b <<= 1) {
      const float sgn = (part & b) ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, v[i], b);
        v[i] = fmaf(v[i], sgn, o);              // v + o or o - v: one rounding either way
      }
    }
  }
  float m = absmax_regs(v, 0, 32);
  if (a.group >= 64) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (a.group >= 128) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (!ok) return;
  const __half s16 = __float2half_rn(fminf(__fdiv_rn(__fmul_rn(m, norm), 7.0f), 65504.f));
  const float s = __half2float(s16);
  const float f = s > 0.f ? __fdiv_rn(norm, s) : 0.f;
  const uint32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page_size);
  const uint32_t off = static_cast<uint32_t>(slot) - page * a.page_size;
  const int64_t cell = (static_cast<int64_t>(page) * a.kv_heads + head) * a.page_size + off;
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
// warp, instead of unrotating K.
//
// The cache is read once: 1 byte per K, V element pair, against 4 D products
// per row and position, so with few rows the kernel is bound by memory and
// above that by the unpacking of nibbles.  Layout of the work: a warp takes
// tiles of 16 positions and computes S^T = K q^T and O^T = V^T P^T with
// m16n8k16 products, positions (and head elements) on the side of 16, query
// rows on the side of 8, so that the 1 .. 8 rows of a group of heads fill the
// product.  The nibbles become fp16 operands in registers: a masked pair of
// nibbles under the exponent of 1024 is the fp16 number 1024 + (code + 8), and
// one subtraction leaves the code, exactly.  The order of the contraction is
// free, so every thread reads whole words from shared memory; P^T comes out
// of S^T by a transposition of 8 x 8 blocks (movmatrix).  Tiles reach shared
// memory by 16-byte asynchronous copies, STAGES - 1 tiles ahead of use, each
// warp in a ring of its own: the loop has no block-wide barrier.
//
// Rounding: q to fp16 (scaled by a power of 2 so that the row's largest value
// is in [1, 2): 2^-12 relative), P to fp16 (2^-11 relative; the running
// maximum below bounds it by 2^8).  Codes are exact, scales multiply in fp32,
// and sums, maxima and the output accumulate in fp32.
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
  float* part_o;             // [splits][batch * q_len * heads][D] (splits > 1)
  float2* part_ml;           // [splits][batch * q_len * heads]
  int64_t num_pages;
  int64_t out_rows;          // batch * q_len * heads
  int max_pages, page_size;
  int q_len, kv_heads, ratio;   // heads = kv_heads * ratio
  int row_tiles, splits;
  int rotate;
  float norm;                // fp32(1 / sqrt(D))
  float scale_log2;          // scale * log2(e)
};

constexpr int kWarps = 4;

template <int D, int GROUP, int NT, int STAGES>
struct Cfg {
  static constexpr int G = D / GROUP;
  static constexpr int CODE_BYTES = 16 * D / 2;             // one tile's codes of K or V
  static constexpr int SCALE_BYTES = 16 * G * 2;
  static constexpr int STAGE_BYTES = 2 * CODE_BYTES + 2 * SCALE_BYTES;
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES;   // per warp
  static constexpr int ROWS = 8 * NT;
  static constexpr int JOIN_STRIDE = D + 4;                 // floats per row of a warp's partial output
  static constexpr int JOIN_BYTES = kWarps * ROWS * (JOIN_STRIDE + 2) * 4;
  static constexpr int MAIN_BYTES = kWarps * RING_BYTES;
  static constexpr int BUF_BYTES = MAIN_BYTES > JOIN_BYTES ? MAIN_BYTES : JOIN_BYTES;
  static constexpr int SMEM_BYTES = BUF_BYTES + kWarps * STAGES * 4;   // + valid positions per tile in flight
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
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

// The codes of nibbles 0, 1, 2, 3 of both halves of w as fp16 pairs.  Under
// 0x6400 (1024, unit steps) nibble n reads 1024 + (n ^ 8) = 1032 + code; one
// nibble further up the steps are 16: 1024 + 16 (code + 8) = 1152 + 16 code.
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t (&x)[4]) {
  const __half2 k1032 = bits_h2(0x64086408u), k16th = bits_h2(0x2C002C00u), km72 = bits_h2(0xD480D480u);
  const uint32_t u = w >> 8;
  x[0] = h2_bits(__hsub2(bits_h2((w & 0x000F000Fu) ^ 0x64086408u), k1032));
  x[1] = h2_bits(__hfma2(bits_h2((w & 0x00F000F0u) ^ 0x64806480u), k16th, km72));
  x[2] = h2_bits(__hsub2(bits_h2((u & 0x000F000Fu) ^ 0x64086408u), k1032));
  x[3] = h2_bits(__hfma2(bits_h2((u & 0x00F000F0u) ^ 0x64806480u), k16th, km72));
}

// Byte offset of 16-byte chunk `ch` of position t in a tile's codes.  The XOR
// spreads the chunks that one load instruction reads over the banks: K is read
// chunk by chunk for positions 0..7 at once, V for four positions at once.
template <int D>
__device__ __forceinline__ int k_chunk(int t, int ch) {
  if constexpr (D == 128) return t * 64 + ((ch ^ ((t >> 1) & 3)) << 4);
  else return t * 32 + ((ch ^ ((t >> 2) & 1)) << 4);
}
template <int D>
__device__ __forceinline__ int v_chunk(int t, int ch) {
  if constexpr (D == 128) return t * 64 + ((ch ^ (t & 2)) << 4);
  else return t * 32 + (ch << 4);
}

template <int D, int GROUP, int NT, int STAGES>
__global__ void __launch_bounds__(32 * kWarps) kv4_attention_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<D, GROUP, NT, STAGES>;
  constexpr int G = C::G;
  constexpr int NG = D / 32;                  // words of a row that one lane reads of K
  constexpr int MT = D / 16;                  // 16-element tiles of the output
  constexpr int TPG = GROUP / 16;             // of them in a scale group
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * C::RING_BYTES;
  int* nvalid = reinterpret_cast<int*>(smem + C::BUF_BYTES) + warp * STAGES;

  grid_dependency_sync();
  const int unit = blockIdx.x, split = blockIdx.y;
  const int rt = unit % a.row_tiles;
  const int bh = unit / a.row_tiles;
  const int h = bh % a.kv_heads, b = bh / a.kv_heads;
  const int rows = a.q_len * a.ratio;
  const int capacity = a.max_pages * a.page_size;
  int len = a.lengths[b];
  if (len < 0 || len > capacity) {
    if (threadIdx.x == 0) atomicOr(&hadq_kv4_fault, kFaultLength);
    len = len < 0 ? 0 : capacity;
  }

  // tiles of this split, interleaved over the warps
  const int tiles = (len + 15) >> 4;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int t0 = min(split * per, tiles), t1 = min(t0 + per, tiles);
  const int mine = t1 - t0 > warp ? (t1 - t0 - warp + kWarps - 1) / kWarps : 0;

  // ---- page entries of the warp's next 32 tiles, one per lane
  int ent_page = -1, ent_off = 0;
  const int blocks = a.page_size >> 4;
  auto load_entries = [&](int i0) {
    const int i = i0 + lane;
    ent_page = -1;
    if (i < mine) {
      const int tile = t0 + warp + i * kWarps;
      const int p = tile / blocks;
      ent_off = (tile - p * blocks) << 4;
      ent_page = a.table[static_cast<int64_t>(b) * a.max_pages + p];
      if (ent_page < 0 || ent_page >= a.num_pages) {
        atomicOr(&hadq_kv4_fault, kFaultPage);
        ent_page = -1;
      }
    }
  };
  const uint32_t ring_u = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  auto issue = [&](int i) {
    if (i < mine) {
      if ((i & 31) == 0) load_entries(i);
      const int page = __shfl_sync(0xffffffffu, ent_page, i & 31);
      const int off = __shfl_sync(0xffffffffu, ent_off, i & 31);
      const int st = i % STAGES;
      const int tile = t0 + warp + i * kWarps;
      // a page outside the cache: nothing is read, its positions are masked
      const int nv = page < 0 ? 0 : min(16, len - tile * 16);
      if (lane == 0) nvalid[st] = nv;
      const int64_t cell = (static_cast<int64_t>(page < 0 ? 0 : page) * a.kv_heads + h) * a.page_size + (page < 0 ? 0 : off);
      const uint8_t* kc = a.k_codes + cell * (D / 2);
      const uint8_t* vc = a.v_codes + cell * (D / 2);
      const uint32_t dst = ring_u + st * C::STAGE_BYTES;
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        const int j = lane + 32 * u, t = j / NG, ch = j % NG;
        const int bytes = t < nv ? 16 : 0;
        cp_async16(dst + k_chunk<D>(t, ch), kc + 16 * j, bytes);
        cp_async16(dst + C::CODE_BYTES + v_chunk<D>(t, ch), vc + 16 * j, bytes);
      }
      const int j = lane & 15;
      if (j < 2 * G) {                        // scales: lanes 0.. of K, 16.. of V
        const int bytes = min(max(nv * 2 * G - 16 * j, 0), 16);
        const uint8_t* src = reinterpret_cast<const uint8_t*>((lane < 16 ? a.k_scales : a.v_scales) + cell * G) + 16 * j;
        cp_async16(dst + 2 * C::CODE_BYTES + (lane < 16 ? 0 : C::SCALE_BYTES) + 16 * j, src, bytes);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue(i);

  // ---- query rows: lane (r, c) holds elements 32 g + 8 c + 0..7 of row r
  uint32_t qb[NT][NG][4];
  float qf[NT][2];                            // factor of rows 2c, 2c + 1 to base-2 scores
  int limit[NT][2];                           // first position that the row does not see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rho = rt * C::ROWS + nt * 8 + r;
    float v[D / 4];
    if (rho < rows) {
      const int i = rho / a.ratio;
      const int head = h * a.ratio + rho - i * a.ratio;
      const uint16_t* p = a.q + (static_cast<int64_t>(b) * a.q_len + i) * a.q_stride + static_cast<int64_t>(head) * D + 8 * c;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint4 w = *reinterpret_cast<const uint4*>(p + 32 * g);
        unpack_bf16x2(w.x, v[8 * g + 0], v[8 * g + 1]);
        unpack_bf16x2(w.y, v[8 * g + 2], v[8 * g + 3]);
        unpack_bf16x2(w.z, v[8 * g + 4], v[8 * g + 5]);
        unpack_bf16x2(w.w, v[8 * g + 6], v[8 * g + 7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 4; ++i) v[i] = 0.f;
    }
    if (a.rotate) {
      fwht_bits<D / 4, 0, (D == 128 ? 5 : 4)>(v);
#pragma unroll
      for (int s = 1; s < 4; s <<= 1) {
        const float sgn = (c & s) ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) v[i] = fmaf(v[i], sgn, __shfl_xor_sync(0xffffffffu, v[i], s));
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) v[i] *= a.norm;
    }
    float mx = absmax_regs(v, 0, D / 4);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int eb = min(max(static_cast<int>(__float_as_uint(mx) >> 23), 1), 253);
    const float down = __uint_as_float(static_cast<uint32_t>(254 - eb) << 23);   // 2^-e: the largest in [1, 2)
    const float up = __uint_as_float(static_cast<uint32_t>(eb) << 23) * a.scale_log2;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) qb[nt][g][j] = pack_half2(v[8 * g + j] * down, v[8 * g + j + 4] * down);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qf[nt][e] = __shfl_sync(0xffffffffu, up, (2 * c + e) * 4);
      const int col = rt * C::ROWS + nt * 8 + 2 * c + e;
      limit[nt][e] = len - a.q_len + 1 + (col < rows ? col / a.ratio : 0);
    }
  }

  float o[MT][NT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][nt][k] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) m[nt][e] = -1.0e30f, l[nt][e] = 0.f;

  // Row i of a tile's products is position pi(i): pi(2c) = c, pi(2c + 1) = 4 + c,
  // pi(2c + 8) = 8 + c, pi(2c + 9) = 12 + c, so the four lanes c read four
  // neighbouring positions of V.
  const int pr = (r & 1) * 4 + (r >> 1);      // pi(r); pi(r + 8) = pr + 8

  for (int i = 0; i < mine; ++i) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    issue(i + STAGES - 1);                    // into the stage consumed in the last round
    const int st = i % STAGES;
    const uint8_t* kt = ring + st * C::STAGE_BYTES;
    const uint8_t* vt = kt + C::CODE_BYTES;
    const __half* kst = reinterpret_cast<const __half*>(kt + 2 * C::CODE_BYTES);
    const __half* vst = kst + 16 * G;
    const int nv = nvalid[st];
    const int pos = (t0 + warp + i * kWarps) * 16 + pr;

    // ---- S^T = K q^T, K's scales applied to the sums of each group
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[nt][k] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[nt][k] = 0.f;
#pragma unroll
      for (int w = g * (GROUP / 32); w < (g + 1) * (GROUP / 32); ++w) {
        uint32_t xa[4], xb[4];
        unpack4(*reinterpret_cast<const uint32_t*>(kt + k_chunk<D>(pr, w) + 4 * c), xa);
        unpack4(*reinterpret_cast<const uint32_t*>(kt + k_chunk<D>(pr + 8, w) + 4 * c), xb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(acc[nt], xa[0], xb[0], xa[1], xb[1], qb[nt][w][0], qb[nt][w][1]);
          mma16816(acc[nt], xa[2], xb[2], xa[3], xb[3], qb[nt][w][2], qb[nt][w][3]);
        }
      }
      const float k0 = __half2float(kst[pr * G + g]), k1 = __half2float(kst[(pr + 8) * G + g]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        s[nt][0] = fmaf(acc[nt][0], k0, s[nt][0]);
        s[nt][1] = fmaf(acc[nt][1], k0, s[nt][1]);
        s[nt][2] = fmaf(acc[nt][2], k1, s[nt][2]);
        s[nt][3] = fmaf(acc[nt][3], k1, s[nt][3]);
      }
    }
    // V's scales of positions pr, pr + 8, and log2 of the largest of a position
    float sv[2][G], lv[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // finite, so that a position that a row does not see adds 0 whatever its scale
        sv[e][g] = fminf(fmaxf(__half2float(vst[(pr + 8 * e) * G + g]), -65504.f), 65504.f);
        top = fmaxf(top, fabsf(sv[e][g]));
      }
      lv[e] = log2_fast(fmaxf(top, 5.9604645e-8f));     // at least the least fp16 above zero
    }
    const bool seen0 = pr < nv, seen1 = pr + 8 < nv;
    bool rise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[nt][e] = seen0 && pos < limit[nt][e] ? s[nt][e] * qf[nt][e] : -INFINITY;
        s[nt][2 + e] = seen1 && pos + 8 < limit[nt][e] ? s[nt][2 + e] * qf[nt][e] : -INFINITY;
        rise |= s[nt][e] + lv[0] > m[nt][e] + 8.f || s[nt][2 + e] + lv[1] > m[nt][e] + 8.f;
      }
    }
    // The running maximum moves only when a value passes it by 2^8: P stays
    // below 2^8, and most tiles need one vote instead of the exchange.
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[nt][e] + lv[0], s[nt][2 + e] + lv[1]);
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          t = fmaxf(t, m[nt][e]);
          const float f = exp2_fast(m[nt][e] - t);
          m[nt][e] = t;
          l[nt][e] *= f;
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
        s[nt][e] = exp2_fast(s[nt][e] - m[nt][e]);
        s[nt][2 + e] = exp2_fast(s[nt][2 + e] - m[nt][e]);
        l[nt][e] += s[nt][e] + s[nt][2 + e];
      }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int g = 0; g < G; ++g) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pb[nt][0] = transpose8x8(pack_half2(s[nt][0] * sv[0][g], s[nt][1] * sv[0][g]));
        pb[nt][1] = transpose8x8(pack_half2(s[nt][2] * sv[1][g], s[nt][3] * sv[1][g]));
      }
      // lane (r, c): elements g GROUP + r GROUP / 8 + 0..GROUP / 8 - 1 of positions c, 4 + c, 8 + c, 12 + c
      uint32_t w[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int p = 4 * t + c;
        if constexpr (GROUP == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(vt + v_chunk<D>(p, r >> 1) + (r & 1) * 8);
          w[t][0] = x.x;
          w[t][1] = x.y;
        } else if constexpr (GROUP == 64) {
          w[t][0] = *reinterpret_cast<const uint32_t*>(vt + v_chunk<D>(p, 2 * g + (r >> 2)) + (r & 3) * 4);
        } else {
          w[t][0] = *reinterpret_cast<const uint16_t*>(vt + v_chunk<D>(p, g) + r * 2);
        }
      }
#pragma unroll
      for (int q4 = 0; q4 < TPG / 2; ++q4) {      // four nibbles, two tiles at a time
        const uint32_t sel = (q4 & 1) ? 0x7632u : 0x5410u;
        uint32_t xa[4], xb[4];
        unpack4(__byte_perm(w[0][q4 >> 1], w[1][q4 >> 1], sel), xa);
        unpack4(__byte_perm(w[2][q4 >> 1], w[3][q4 >> 1], sel), xb);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(o[g * TPG + 2 * q4][nt], xa[0], xa[1], xb[0], xb[1], pb[nt][0], pb[nt][1]);
          mma16816(o[g * TPG + 2 * q4 + 1][nt], xa[2], xa[3], xb[2], xb[3], pb[nt][0], pb[nt][1]);
        }
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
        for (int t = 0; t < TPG; ++t) {
          dst[g * GROUP + 2 * t] = o[g * TPG + t][nt][e];
          dst[g * GROUP + 2 * t + 1] = o[g * TPG + t][nt][2 + e];
        }
      if (r == 0) jml[warp * C::ROWS + row] = make_float2(m[nt][e], l[nt][e]);
    }
  __syncthreads();
  for (int x = threadIdx.x; x < C::ROWS * (D / 2); x += 32 * kWarps) {
    const int row = x / (D / 2), d = (x % (D / 2)) * 2;
    const int rho = rt * C::ROWS + row;
    if (rho >= rows) continue;
    float top = -1.0e30f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, jml[w * C::ROWS + row].x);
    float sum = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = jml[w * C::ROWS + row];
      const float f = exp2_fast(ml.x - top);
      const float2 y = *reinterpret_cast<const float2*>(jo + (w * C::ROWS + row) * C::JOIN_STRIDE + d);
      sum = fmaf(ml.y, f, sum);
      v0 = fmaf(y.x, f, v0);
      v1 = fmaf(y.y, f, v1);
    }
    const int qi = rho / a.ratio;
    const int64_t orow = (static_cast<int64_t>(b) * a.q_len + qi) * (a.kv_heads * a.ratio) + h * a.ratio + rho - qi * a.ratio;
    if (a.splits == 1) {
      const float inv = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;      // a row that sees nothing: zeros
      *reinterpret_cast<uint32_t*>(a.out + orow * D + d) = pack_bf16x2(v0 * inv, v1 * inv);
    } else {
      const int64_t prow = split * a.out_rows + orow;
      *reinterpret_cast<float2*>(a.part_o + prow * D + d) = make_float2(v0, v1);
      if (d == 0) a.part_ml[prow] = make_float2(top, sum);
    }
  }
}

// Joins the splits of a row, in order: one warp per row, D / 32 values per lane.
template <int D>
__global__ void __launch_bounds__(128) kv4_join_kernel(const float* __restrict__ part_o,
                                                       const float2* __restrict__ part_ml, int64_t out_rows,
                                                       int splits, uint16_t* __restrict__ out) {
  constexpr int E = D / 32;
  grid_dependency_sync();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= out_rows) return;
  float top = -1.0e30f;
  for (int s = lane; s < splits; s += 32) top = fmaxf(top, part_ml[s * out_rows + row].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float sum = 0.f, v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float2 ml = part_ml[s * out_rows + row];
    const float f = exp2_fast(ml.x - top);
    const float* p = part_o + (s * out_rows + row) * D + lane * E;
    sum = fmaf(ml.y, f, sum);
    if constexpr (E == 4) {
      const float4 y = *reinterpret_cast<const float4*>(p);
      v[0] = fmaf(y.x, f, v[0]), v[1] = fmaf(y.y, f, v[1]), v[2] = fmaf(y.z, f, v[2]), v[3] = fmaf(y.w, f, v[3]);
    } else {
      const float2 y = *reinterpret_cast<const float2*>(p);
      v[0] = fmaf(y.x, f, v[0]), v[1] = fmaf(y.y, f, v[1]);
    }
  }
  const float inv = sum > 0.f ? __fdiv_rn(1.f, sum) : 0.f;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(out + row * D + lane * 4) =
        make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(out + row * D + lane * 2) = pack_bf16x2(v[0] * inv, v[1] * inv);
}

}  // namespace kv4
}  // namespace hadq
