// Matrix product of int8 codes with a scale per token and per output channel:
//
//   y[i][j] = (sum_k a[i][k] w[j][k]) * sa[i] * sw[j] + bias[j],
//
// on the tensor cores (tcgen05.mma kind::i8, 32-bit integer sums in tensor
// memory).  The sums are exact for k < 131072, so their order is free: a split
// of k adds up to the same bits, and every kernel here gives the same result.
//
// Four kernels.
//
//   imm_row_kernel    a handful of tokens: bound by reading w, and by what it
//       takes to begin.  Warps read rows of w straight from global memory and
//       form four-way byte products; nothing is set up first.  4096 x 14336: 9.5
//       us with 1 token (6.2 TB/s), 10.4 with 4, against 13.6 and 13.8 of the
//       split kernel; with 8 tokens 17.3 against 13.8, the byte products'
//       operands no longer fit beside the loads.
//   imm_warp_kernel   up to 16 tokens: the same, with the warps' matrix
//       instructions.  8 and 16 tokens, 4096 x 4096: 4.7 and 4.9 us against 6.5
//       and 6.5 of the split kernel; 4096 x 14336: 13.0 and 13.1 against 13.4
//       and 13.4.  From 32 tokens on the token loads of every warp cost more
//       (8.4 against 7.4).
//   imm_split_kernel  up to a few hundred tokens: bound by reading w.  Output
//       channels are the MMA's 128 rows and TN tokens its columns, so one token
//       costs no more traffic than it has, and the CTAs of a cluster share the k
//       of a tile, adding their sums through distributed shared memory.  48 x
//       14336 x 4096: 13.6 us, of which the loads alone take 9 and launch, start
//       and epilogue the rest; tiles of 96 to 120 channels, so that every SM has
//       one, take as long (13.5): memory is what all of them wait for.
//   imm_pair_kernel   many tokens: bound by the tensor cores.  CTA pairs
//       compute 256 x 256 tiles (cta_group::2), which halves the shared-memory
//       and L2 reads per product of a single CTA's tile; persistent, two
//       accumulators, so that the epilogue of a tile runs under the products
//       of the next: eight warps, since with four it outlasted the products of
//       k = 1024 (4096 x 4096: 24.7 us, with four 31.3).  8192 x 4096 x 14336: 305 us.
//
// The last two stage 128-byte slices of k by TMA (128-byte swizzle; the tail of
// k and rows beyond a matrix are filled with zeros) into a ring that one thread
// feeds and one thread consumes.
#pragma once

#include "hadq_tc.cuh"

namespace hadq {
namespace imm {

using tc::mbar_arrive_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;
using tc::smem_desc;
using tc::smem_u32;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_wait_ld;

struct Args {
  const int8_t* a;
  const int8_t* w;
  const float* sa;
  const float* sw;
  const float* bias;   // nullptr: none
  void* out;
  int m, n, k;         // tokens, channels
  int tokens;          // of a CTA of the split kernel
};

constexpr int kSlice = 128;   // bytes of k per stage

// Instruction descriptor of kind::i8: signed A and B, 32-bit integer D, both
// operands K-major.
__host__ __device__ constexpr uint32_t idesc_i8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc),
        "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc),
        "r"(accumulate));
}

// 32 consecutive columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32i(uint32_t taddr, int (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld16i(uint32_t taddr, int* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(c0), "r"(c1) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Address in the cluster's shared memory of `addr` (this CTA's) in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// (sum * sa) * sw + bias, rounded step by step, so that every kernel's result
// is the same.
__device__ __forceinline__ float scaled(int acc, float sa) { return __fmul_rn(__int2float_rn(acc), sa); }
__device__ __forceinline__ float finish(float t, float sw, bool biased, float bias) {
  const float y = __fmul_rn(t, sw);
  return biased ? __fadd_rn(y, bias) : y;
}

template <bool OUT_BF16>
__device__ __forceinline__ void store_one(void* out, int64_t e, float y) {
  if constexpr (OUT_BF16) static_cast<__nv_bfloat16*>(out)[e] = __float2bfloat16_rn(y);
  else static_cast<float*>(out)[e] = y;
}

// ---------------------------------------------------- a handful of tokens

constexpr int kRowWarps = 8;

// A warp takes four channels and one of `parts` runs of k (16-byte chunks, lane
// by lane); the CTA's warps are 8 / parts such quads of channels.  M: tokens,
// rounded up to 1, 2 or 4 (those beyond p.m repeat the last one, unwritten).
template <int M, bool OUT_BF16>
__global__ void __launch_bounds__(32 * kRowWarps) imm_row_kernel(const __grid_constant__ Args p, int parts) {
  __shared__ int sums[kRowWarps][4 * M];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = kRowWarps / parts, quad = warp / parts, part = warp - quad * parts;
  const int ch0 = (blockIdx.x * quads + quad) * 4;
  const int chunks = p.k >> 4;
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * part / parts);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / parts);
  const int8_t* w[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) w[r] = p.w + static_cast<int64_t>(min(ch0 + r, p.n - 1)) * p.k;
  if (lane < 4 && c1 > c0)                     // a hint: it may precede the wait for the previous kernel
    prefetch_l2(w[lane] + 16 * c0, static_cast<uint32_t>(min((c1 - c0) * 16, 2048)));
  grid_dependency_sync();
  constexpr int kAhead = M == 1 ? 4 : M == 2 ? 2 : 1;   // rounds in flight, as the registers allow
  int acc[4][M];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < M; ++t) acc[r][t] = 0;
#pragma unroll kAhead
  for (int c = c0 + lane; c < c1; c += 32) {
    uint4 x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = ld_stream(reinterpret_cast<const uint4*>(w[r]) + c);
#pragma unroll
    for (int t = 0; t < M; ++t) {
      const int4 a = reinterpret_cast<const int4*>(p.a + static_cast<int64_t>(min(t, p.m - 1)) * p.k)[c];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[r][t] = __dp4a(static_cast<int>(x[r].x), a.x, acc[r][t]);
        acc[r][t] = __dp4a(static_cast<int>(x[r].y), a.y, acc[r][t]);
        acc[r][t] = __dp4a(static_cast<int>(x[r].z), a.z, acc[r][t]);
        acc[r][t] = __dp4a(static_cast<int>(x[r].w), a.w, acc[r][t]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < M; ++t) {
      const int s = __reduce_add_sync(0xffffffffu, acc[r][t]);
      if (lane == 0) sums[warp][r * M + t] = s;
    }
  __syncthreads();
  if (threadIdx.x < quads * 4 * M) {
    const int q = threadIdx.x / (4 * M), i = threadIdx.x - q * 4 * M, t = i % M;
    const int ch = (blockIdx.x * quads + q) * 4 + i / M;
    int sum = 0;
    for (int s = 0; s < parts; ++s) sum += sums[q * parts + s][i];
    if (ch < p.n && t < p.m)
      store_one<OUT_BF16>(p.out, static_cast<int64_t>(t) * p.n + ch,
                          finish(scaled(sum, p.sa[t]), p.sw[ch], p.bias != nullptr, p.bias != nullptr ? p.bias[ch] : 0.f));
  }
}

// ------------------------------------------------------------ up to 16 tokens

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp takes 16 MT channels (the rows of its products), all 8 NT tokens (their
// columns) and one of `parts` runs of k, 64 bytes at a time: lane (r, c) holds
// bytes 16 c .. of channel rows r, r + 8 and of token r, which are the operands of
// two products as they lie (the order of a contraction is free).  Weights come
// straight from global memory, two rounds ahead; tokens, read by every warp,
// through L1.  The warps' sums meet in shared memory, by integer atomics (exact
// in any order).
template <int MT, int NT, bool OUT_BF16>
__global__ void __launch_bounds__(32 * kRowWarps, 2) imm_warp_kernel(const __grid_constant__ Args p, int parts) {
  constexpr int CH = 16 * MT, TOK = 8 * NT;
  extern __shared__ int sums[];                // [group of channels][token][CH]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int groups = kRowWarps / parts, group = warp / parts, part = warp - group * parts;
  const int ch0 = (blockIdx.x * groups + group) * CH;
  const int rounds = (p.k + 63) >> 6;
  const int i0 = static_cast<int>(static_cast<int64_t>(rounds) * part / parts);
  const int i1 = static_cast<int>(static_cast<int64_t>(rounds) * (part + 1) / parts);
  if (lane < CH && i1 > i0 && ch0 + lane < p.n)  // a hint: it may precede the wait for the previous kernel
    prefetch_l2(p.w + static_cast<int64_t>(ch0 + lane) * p.k + 64 * i0, static_cast<uint32_t>(min(min((i1 - i0) * 64, p.k - 64 * i0), 512)));
  for (int i = threadIdx.x; i < groups * TOK * CH; i += 32 * kRowWarps) sums[i] = 0;
  const int8_t* w[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) w[t][e] = p.w + static_cast<int64_t>(min(ch0 + 16 * t + 8 * e + r, p.n - 1)) * p.k + 16 * c;
  const int8_t* a[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) a[t] = p.a + static_cast<int64_t>(min(8 * t + r, p.m - 1)) * p.k + 16 * c;
  __syncthreads();
  grid_dependency_sync();

  int acc[MT][NT][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[t][u][k] = 0;
  uint4 x[2][MT][2];
  auto load = [&](int i, uint4 (&y)[MT][2]) {  // zeros past the end of k
    const bool in = i < i1 && 64 * i + 16 * c < p.k;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        y[t][e] = in ? ld_stream(reinterpret_cast<const uint4*>(w[t][e] + 64 * i)) : make_uint4(0u, 0u, 0u, 0u);
  };
  auto step = [&](int i, uint4 (&y)[MT][2]) {
    const int at = 64 * i + 16 * c < p.k ? 64 * i : -16 * c;   // any bytes of the row will do against zeros
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const uint4 b = *reinterpret_cast<const uint4*>(a[u] + at);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        mma_s8(acc[t][u], y[t][0].x, y[t][1].x, y[t][0].y, y[t][1].y, b.x, b.y);
        mma_s8(acc[t][u], y[t][0].z, y[t][1].z, y[t][0].w, y[t][1].w, b.z, b.w);
      }
    }
  };
  load(i0, x[0]);
  load(i0 + 1, x[1]);
#pragma unroll 1
  for (int i = i0; i < i1; i += 2) {
    step(i, x[0]);
    load(i + 2, x[0]);
    if (i + 1 < i1) step(i + 1, x[1]);
    load(i + 3, x[1]);
  }
  int* mine = sums + group * TOK * CH;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        int* at = mine + (8 * u + 2 * c + (k & 1)) * CH + 16 * t + 8 * (k >> 1) + r;
        if (parts > 1) atomicAdd(at, acc[t][u][k]);
        else *at = acc[t][u][k];
      }
  __syncthreads();
  // channels along the lanes
  for (int i = threadIdx.x; i < groups * CH * p.m; i += 32 * kRowWarps) {
    const int col = i % (groups * CH), tok = i / (groups * CH), g = col / CH;
    const int ch = blockIdx.x * groups * CH + col;
    if (ch < p.n)
      store_one<OUT_BF16>(p.out, static_cast<int64_t>(tok) * p.n + ch,
                          finish(scaled(sums[(g * TOK + tok) * CH + col - g * CH], p.sa[tok]), p.sw[ch], p.bias != nullptr,
                                 p.bias != nullptr ? p.bias[ch] : 0.f));
  }
}

// ------------------------------------------------------------- few tokens

template <int TN_, int STAGES_>
struct SplitCfg {
  static constexpr int TN = TN_, STAGES = STAGES_;
  static constexpr int W_BYTES = 128 * kSlice, A_BYTES = TN * kSlice;
  static constexpr int STAGE_BYTES = W_BYTES + A_BYTES;
  static_assert(TN % 32 == 0, "a rank of up to 8 takes four columns or more");
  static constexpr int TMEM_COLS = TN;
  static constexpr int THREADS = 128;
  static constexpr int SM_RING = 0;
  static constexpr int SM_JOIN = STAGES * STAGE_BYTES;                // [source rank][quad of columns][channel][4]
  static constexpr int SM_SA = SM_JOIN + TN * 128 * 4;                // the tokens' scales
  static constexpr int SM_BARS = SM_SA + TN * 4;
  static constexpr int SM_SLOT = SM_BARS + 8 * (2 * STAGES + 1);
  static constexpr int SMEM_BYTES = SM_SLOT + 16 + 1024;
  static constexpr int CTAS = 228 * 1024 / (SMEM_BYTES + 1024);       // on an SM
};

// CTA (tile, rank): channels ch0 .. ch0 + 127, tokens t0 .. t0 + TN - 1, the
// rank's share of k.  Every rank then finishes TN / splits of the tokens.
template <class C, bool OUT_BF16>
__global__ void __launch_bounds__(C::THREADS)
imm_split_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ Args p, int splits, int token_tiles) {
  constexpr int TN = C::TN, STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::smem_align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::SM_BARS);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::SM_SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int rank = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / splits;
  const int ch0 = (tile / token_tiles) * 128, t0 = (tile % token_tiles) * p.tokens;
  const int slices = (p.k + kSlice - 1) / kSlice;
  const int s0 = static_cast<int>(static_cast<int64_t>(slices) * rank / splits);
  const int iters = static_cast<int>(static_cast<int64_t>(slices) * (rank + 1) / splits) - s0;   // >= 1

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(C::TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
  }
  if (splits > 1) cluster_arrive();           // waited for before the first access to another CTA's memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  // While the previous kernel drains, ask L2 for the first weights (a hint: it
  // reads nothing, so it may precede the wait).
  if (threadIdx.x == 0)
    for (int i = 0; i < min(iters, 3); ++i) prefetch_tile(&map_w, (s0 + i) * kSlice, ch0);
  grid_dependency_sync();
  // What the epilogue reads, while the products run: a channel's scale and bias
  // in its thread, the tokens' scales in shared memory.
  float* sa = reinterpret_cast<float*>(smem + C::SM_SA);
  const int ch = ch0 + threadIdx.x;           // TMEM lane = thread
  const bool live = ch < p.n, biased = p.bias != nullptr;
  float sw = 0.f, bias = 0.f;
  if (warp >= 2 || lane != 0) {
    if (warp >= 2)
      for (int t = threadIdx.x - 64; t < TN; t += 64) sa[t] = t0 + t < p.m ? p.sa[t0 + t] : 0.f;
    if (live) sw = p.sw[ch];
    if (live && biased) bias = p.bias[ch];
  }

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------- producer
    for (int i = 0; i < iters; ++i) {
      const int s = i % STAGES;
      if (i >= STAGES && !mbar_wait(&empty[s], ((i / STAGES) & 1) ^ 1)) {
        atomicOr(&tc::hadq_tc_fault, tc::kFaultProducer);
        tc::drain_loads(full, STAGES, i);
        break;
      }
      mbar_arrive_expect_tx(&full[s], C::W_BYTES + p.tokens * kSlice);   // whole boxes
      uint8_t* dst = smem + C::SM_RING + s * C::STAGE_BYTES;
      tc::tma_load_2d(dst, &map_w, (s0 + i) * kSlice, ch0, &full[s]);
      tc::tma_load_2d(dst + C::W_BYTES, &map_a, (s0 + i) * kSlice, t0, &full[s]);
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------------ MMA
    int i = 0;
    for (; i < iters; ++i) {
      const int s = i % STAGES;
      if (!mbar_wait(&full[s], (i / STAGES) & 1)) {
        atomicOr(&tc::hadq_tc_fault, tc::kFaultMma);
        tc::drain_mmas(empty, STAGES, i);
        break;
      }
      tc_fence_after();
      const uint32_t wb = smem_u32(smem + C::SM_RING + s * C::STAGE_BYTES), ab = wb + C::W_BYTES;
#pragma unroll
      for (int kk = 0; kk < kSlice / 32; ++kk)
        mma_i8<1>(tmem, smem_desc(wb + 32 * kk, 16, 1024, tc::kSwizzle128), smem_desc(ab + 32 * kk, 16, 1024, tc::kSwizzle128),
                  idesc_i8(128, TN), (i | kk) != 0 ? 1u : 0u);
      tc::mma_commit(&empty[s]);
    }
    if (i == iters) tc::mma_commit(done);
  }
  __syncwarp();

  // --------------------------------------------------------------- epilogue
  if (warp < 2 && lane == 0) {                // the threads that fed the loop
    if (live) sw = p.sw[ch];
    if (live && biased) bias = p.bias[ch];
  }
  bool ok = mbar_wait(done, 0);
  if (!ok && lane == 0) atomicOr(&tc::hadq_tc_fault, tc::kFaultEpilogue);
  ok = __all_sync(0xffffffffu, ok);
  __syncthreads();                            // sa
  tc_fence_after();
  const int cols = min(p.tokens, p.m - t0);   // of this tile
  // N columns of the tile from their sums: all of them computed before the first
  // is stored, so that their latencies overlap (one after the other, each behind
  // its own condition, they took 105 clocks a column).
  auto put = [&](int col, const auto& acc) {
    constexpr int N = sizeof(acc) / sizeof(int);
    float y[N];
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 s = *reinterpret_cast<const float4*>(sa + col + j);
      y[j] = finish(scaled(acc[j], s.x), sw, biased, bias);
      y[j + 1] = finish(scaled(acc[j + 1], s.y), sw, biased, bias);
      y[j + 2] = finish(scaled(acc[j + 2], s.z), sw, biased, bias);
      y[j + 3] = finish(scaled(acc[j + 3], s.w), sw, biased, bias);
    }
    int64_t e = static_cast<int64_t>(t0 + col) * p.n + ch;
#pragma unroll
    for (int j = 0; j < N; ++j, e += p.n)
      if (live && col + j < cols) store_one<OUT_BF16>(p.out, e, y[j]);
  };
  const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  if (splits == 1) {
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < cols; c += 16) {
        int v[16];
        tmem_ld16i(taddr + c, v);
        tmem_wait_ld();
        put(c, v);
      }
    }
  } else {
    // Token column c goes to rank c / mine; there, the sources' sums are added
    // (integers: in any order the same).  Four columns of a channel travel
    // together.
    const int mine = TN / splits, lg = __ffs(mine) - 1;   // 4 or more, a power of 2
    cluster_wait();
    const uint32_t join = smem_u32(smem + C::SM_JOIN);
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
      int v[16];
      tmem_ld16i(taddr + c, v);
      tmem_wait_ld();
      if (!ok) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0;
      }
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const uint32_t at = join + (((rank << lg) + ((c + j) & (mine - 1))) * 128 + threadIdx.x * 4) * 4;
        asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(map_rank(at, (c + j) >> lg)), "r"(v[j]),
                     "r"(v[j + 1]), "r"(v[j + 2]), "r"(v[j + 3])
                     : "memory");
      }
    }
    cluster_arrive();
    cluster_wait();
    const int* got = reinterpret_cast<const int*>(smem + C::SM_JOIN);
#pragma unroll 2
    for (int col = 0; col < min(mine, cols - rank * mine); col += 4) {
      int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < splits) {
          const int4 x = *reinterpret_cast<const int4*>(got + ((r << lg) + col) * 128 + threadIdx.x * 4);
          sum = make_int4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
        }
      const int v[4] = {sum.x, sum.y, sum.z, sum.w};
      put(rank * mine + col, v);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
  }
}

// ------------------------------------------------------------ many tokens

struct PairCfg {
  static constexpr int STAGES = 6;
  static constexpr int TILE = 256;                                    // tokens and channels of a pair's tile
  static constexpr int OP_BYTES = 128 * kSlice;                       // one CTA's half of an operand
  static constexpr int STAGE_BYTES = 2 * OP_BYTES;
  static constexpr int EPI_WARPS = 8;                                 // two for each quarter of the rows
  static constexpr int THREADS = 32 * (2 + EPI_WARPS);                // producer, MMA, epilogue
  static constexpr int SM_RING = 0;
  static constexpr int SM_BARS = STAGES * STAGE_BYTES;
  static constexpr int SM_SLOT = SM_BARS + 8 * (2 * STAGES + 4);
  static constexpr int SM_TURN = SM_SLOT + 16;                        // per epilogue warp: 32 rows x 33 words
  static constexpr int SMEM_BYTES = SM_TURN + EPI_WARPS * 32 * 33 * 4 + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// Arrive on the barrier at this offset in both CTAs of the pair once the
// MMAs issued so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Tile t of the grid: bands of 8 token tiles, channels outer, so that the
// tiles in flight share their operands in L2.
__device__ __forceinline__ void tile_at(int t, int mt, int nt, int* im, int* in) {
  const int band = 8 * nt, b = t / band, rest = t - b * band;
  const int h = min(8, mt - 8 * b);
  *in = rest / h;
  *im = 8 * b + rest - *in * h;
}

template <bool OUT_BF16>
__global__ void __launch_bounds__(PairCfg::THREADS, 1)
imm_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ Args p) {
  using C = PairCfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::smem_align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::SM_BARS);    // used in the first CTA of the pair
  uint64_t* empty = full + STAGES;                                    // in both
  uint64_t* acc_full = empty + STAGES;                                // in both
  uint64_t* acc_empty = acc_full + 2;                                 // in the first
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::SM_SLOT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::EPI_WARPS);                     // the epilogue warps of each CTA
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::);
  }
  tc_fence_before();
  cluster_arrive();                                                   // barriers and tensor memory of both are ready
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *slot;
  grid_dependency_sync();

  const int mt = (p.m + C::TILE - 1) / C::TILE, nt = (p.n + C::TILE - 1) / C::TILE;
  const int tiles = mt * nt, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int slices = (p.k + kSlice - 1) / kSlice;

  if (warp == 0) {
    if (lane == 0) {
      // ----------------------------------------------- producer, both CTAs
      uint32_t it = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs) {
        int im, in;
        tile_at(t, mt, nt, &im, &in);
        const int row_a = im * C::TILE + rank * 128, row_w = in * C::TILE + rank * 128;
        for (int i = 0; i < slices; ++i, ++it) {
          const int s = it % STAGES;
          if (it >= STAGES && !mbar_wait(&empty[s], ((it / STAGES) & 1) ^ 1)) {
            atomicOr(&tc::hadq_tc_fault, tc::kFaultProducer);
            if (rank == 0) tc::drain_loads(full, STAGES, it);
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);   // the loads of both CTAs
          const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
          uint8_t* dst = smem + C::SM_RING + s * C::STAGE_BYTES;
          tma_load_pair(dst, &map_a, i * kSlice, row_a, bar);
          tma_load_pair(dst + C::OP_BYTES, &map_w, i * kSlice, row_w, bar);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // --------------------------------------------------- MMA, first CTA
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs, ++n) {
        const uint32_t b = n & 1;
        if (n >= 2 && !mbar_wait(&acc_empty[b], ((n >> 1) & 1) ^ 1)) ok = false;
        tc_fence_after();
        for (int i = 0; ok && i < slices; ++i, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&full[s], (it / STAGES) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ab = smem_u32(smem + C::SM_RING + s * C::STAGE_BYTES), wb = ab + C::OP_BYTES;
#pragma unroll
          for (int kk = 0; kk < kSlice / 32; ++kk)
            mma_i8<2>(tmem + b * 256, smem_desc(ab + 32 * kk, 16, 1024, tc::kSwizzle128),
                      smem_desc(wb + 32 * kk, 16, 1024, tc::kSwizzle128), idesc_i8(256, 256), (i | kk) != 0 ? 1u : 0u);
          commit_pair(&empty[s]);
        }
        if (ok) {
          commit_pair(&acc_full[b]);
        } else {
          atomicOr(&tc::hadq_tc_fault, tc::kFaultMma);
          tc::drain_mmas(empty, STAGES, it);
        }
      }
    }
  } else {
    // ---------------------------------------------------- epilogue, both CTAs
    const int quarter = warp & 3, c0 = (warp - 2) / 4 * 128;          // rows, first column of the warp
    const bool biased = p.bias != nullptr;
    uint32_t n = 0;
    float* turn = reinterpret_cast<float*>(smem + C::SM_TURN) + (warp - 2) * 32 * 33;
    const uint32_t release = map_rank(smem_u32(acc_empty), 0);
    for (int t = pair; t < tiles; t += pairs, ++n) {
      int im, in;
      tile_at(t, mt, nt, &im, &in);
      const uint32_t b = n & 1;
      const int row0 = im * C::TILE + rank * 128 + quarter * 32, col0 = in * C::TILE;
      const int row = row0 + lane, rows = min(32, p.m - row0);
      // scales and biases, while the products run
      const float sa = row < p.m ? p.sa[row] : 0.f;
      float sw[4], bias[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = col0 + c0 + 32 * i + lane;
        sw[i] = at < p.n ? p.sw[at] : 0.f;
        bias[i] = biased && at < p.n ? p.bias[at] : 0.f;
      }
      const bool ok = mbar_wait(&acc_full[b], (n >> 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) atomicOr(&tc::hadq_tc_fault, tc::kFaultEpilogue);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + b * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 32 * i;
        int v[32];
        tmem_ld32i(taddr + c, v);
        tmem_wait_ld();
        if (i == 3) {                                                 // the last read: the MMAs may overwrite
          tc_fence_before();
          __syncwarp();
          if (lane == 0)
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(release + 8 * b) : "memory");
        }
        const int col = col0 + c;
        if (col >= p.n) continue;
        // Rows are turned through shared memory, so that a warp stores runs of
        // columns (any n, any alignment); eight are read before the first is stored.
#pragma unroll
        for (int j = 0; j < 32; ++j) turn[lane * 33 + j] = scaled(v[j], sa);
        __syncwarp();
        int64_t e = static_cast<int64_t>(row0) * p.n + col + lane;
        const bool in_n = col + lane < p.n;
#pragma unroll 1
        for (int r = 0; r < rows; r += 8) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = finish(turn[(r + j) * 33 + lane], sw[i], biased, bias[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j, e += p.n)
            if (in_n && r + j < rows) store_one<OUT_BF16>(p.out, e, y[j]);
        }
        __syncwarp();
      }
    }
  }
  // Neither CTA leaves while the other may reach its barriers or operands.
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

}  // namespace imm
}  // namespace hadq
