// Root-mean-square norm with the residual's addition and int8 codes per token.
//
//   h = x + r (rounded to the stored type), t = h w,
//   q = rne(127 t / max|t|),  s = max|t| / (127 sqrt(mean(h^2) + eps)).
//
// The norm's factor is common to a row, so it cancels in the codes: they
// depend on t alone, whose only rounding is the fp32 product (none for bf16),
// and the sum of squares enters only the scale.  Both reductions therefore
// run in one pass over the row, which stays in registers: x and r are read
// once and the codes, the scale and the stream written once.
//
// Bound by memory.  A row takes T threads with NV chunks of 8 elements each;
// one barrier joins the warps' (sum, max) pairs.  Two kernels:
//   rmsnorm_quant_kernel  a row per CTA (or per warp), straight from global
//       memory: the shortest way through for few rows, and for short ones.
//   rmsnorm_ring_kernel   many rows: CTAs stay and take rows in turn, which bulk
//       copies bring into a ring in shared memory, so that the loads of the next
//       rows are in flight while a row is reduced, coded and stored.  bf16 rows
//       with a residual, 16384 of n: 8192 154.7 us (6.07 TB/s) against 194.3
//       with the other kernel, 14336 272 against 511, 4096 78.3 against 85.2,
//       2048 42 against 43 (there the other one is kept).
#pragma once

#include "hadq_tc.cuh"   // mbarriers with bounded waits

namespace hadq {
namespace norm {

// 8 consecutive elements (x may be the buffer that the kernel also writes).
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t e, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = ld_stream(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
    unpack_bf16x2(w.x, v[0], v[1]);
    unpack_bf16x2(w.y, v[2], v[3]);
    unpack_bf16x2(w.z, v[4], v[5]);
    unpack_bf16x2(w.w, v[6], v[7]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 w = ld_stream(reinterpret_cast<const uint4*>(static_cast<const float*>(p) + e + 4 * h));
      v[4 * h] = __uint_as_float(w.x), v[4 * h + 1] = __uint_as_float(w.y);
      v[4 * h + 2] = __uint_as_float(w.z), v[4 * h + 3] = __uint_as_float(w.w);
    }
  }
}

// Weights: read by every row, so kept in L1.
template <bool BF16>
__device__ __forceinline__ void load8_weight(const void* p, int e, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e);
    unpack_bf16x2(w.x, v[0], v[1]);
    unpack_bf16x2(w.y, v[2], v[3]);
    unpack_bf16x2(w.z, v[4], v[5]);
    unpack_bf16x2(w.w, v[6], v[7]);
  } else {
    const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e)[0];
    const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// Two values to bf16, in one conversion.
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rounds v to the stored type, in place, and stores it.
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t e, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = make_uint4(pair_bf16(v[0], v[1]), pair_bf16(v[2], v[3]), pair_bf16(v[4], v[5]), pair_bf16(v[6], v[7]));
    unpack_bf16x2(w.x, v[0], v[1]);
    unpack_bf16x2(w.y, v[2], v[3]);
    unpack_bf16x2(w.z, v[4], v[5]);
    unpack_bf16x2(w.w, v[6], v[7]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) = w;
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The nearest whole number to 127 t / m, ties to even, for |t| <= m: out of
// line, since almost no element needs it.  `q` (not negative) is the nearest
// or next nearest below 127 |t| / m; 254 |t| against (2 q + 1) m decides, both
// exact in 64 bits (32 bits of significand at most).
static __device__ __noinline__ int exact_code(float t, float m, float q) {
  const double d = 254.0 * fabsf(t) - (2.0 * q + 1.0) * m;
  const int k = static_cast<int>(q) + (d > 0.0 || (d == 0.0 && (static_cast<int>(q) & 1)) ? 1 : 0);
  return t < 0.f ? -k : k;
}

// The same where m is too small for a quotient in fp32.  With 24-bit t and m, a
// quotient of at least a quarter that is not exactly k + 1/2 is at least 2^-35
// from it, and the 53-bit rounding (2^-47 below 128) cannot reach or cross it.
static __device__ __noinline__ int tiny_code(float t, float m) {
  return m > 0.f ? __double2int_rn(127.0 * static_cast<double>(t) / static_cast<double>(m)) : 0;
}

// Eight codes of t against the row's m, f = 127 / m.  t f + 1.5 2^23 leaves
// the whole number nearest to t f; f is off by 2^-24 (relative), so t f by less
// than 1e-5 code units, which decides unless it is within 4e-5 of a half.
__device__ __forceinline__ uint2 codes8(const float (&t)[8], float m, float f) {
  const float2 f2 = make_float2(f, f), magic = make_float2(kRoundMagic, kRoundMagic), minus = make_float2(-1.f, -1.f);
  float far = 0.f;
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = make_float2(t[i], t[i + 1]);
    const float2 r = __ffma2_rn(v, f2, magic);
    const float2 d = __ffma2_rn(v, f2, __ffma2_rn(r, minus, magic));   // t f minus its whole number
    b[i] = __float_as_uint(r.x);
    b[i + 1] = __float_as_uint(r.y);
    far = max3abs(far, d.x, d.y);
  }
  if (!(far < 0.49996f) || !(m > 1.0e-30f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = fabsf(t[i]) * f, q = floorf(p);
      if (!(m > 1.0e-30f)) b[i] = static_cast<uint32_t>(tiny_code(t[i], m));   // f may be infinite
      else if (fabsf(p - q - 0.5f) < 1.0e-4f) b[i] = static_cast<uint32_t>(exact_code(t[i], m, q));
    }
  }
  const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return make_uint2(lo, hi);
}

// Adds eight values h to the sum of squares, and turns them into t = h w and
// their largest.
__device__ __forceinline__ void absorb8(float (&t)[8], const float (&w)[8], float2& ss, float& m) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 h = make_float2(t[i], t[i + 1]);
    ss = __ffma2_rn(h, h, ss);
    const float2 y = __fmul2_rn(h, make_float2(w[i], w[i + 1]));
    t[i] = y.x;
    t[i + 1] = y.y;
    m = max3abs(m, y.x, y.y);
  }
}

__device__ __forceinline__ void add8(float (&t)[8], const float (&r)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 y = __fadd2_rn(make_float2(t[i], t[i + 1]), make_float2(r[i], r[i + 1]));
    t[i] = y.x;
    t[i + 1] = y.y;
  }
}

// CTAs of T threads times RPC rows; T = 32 takes a warp per row (no barrier).
template <bool BF16, bool RES, int T, int RPC, int NV>
__global__ void __launch_bounds__(T * RPC)
rmsnorm_quant_kernel(const void* x, const void* res, const void* weight, int64_t rows, int n, float eps,
                     void* stream_out, int8_t* __restrict__ codes, float* __restrict__ scales) {
  static_assert(T == 32 || RPC == 1, "rows of several warps have a CTA of their own");
  grid_dependency_sync();
  const int tid = threadIdx.x % T;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPC + threadIdx.x / T;
  if (row >= rows) return;                      // whole warps (T = 32) or never (RPC = 1)
  const int64_t e0 = row * n;
  const int chunks = n >> 3;

  float t[NV][8];
  float2 ss2 = make_float2(0.f, 0.f);
  float m = 0.f;
  {
    float r[RES ? NV : 1][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {            // every load first
      const int c = tid + j * T;
      if (c < chunks) {
        load8<BF16>(x, e0 + 8 * c, t[j]);
        if constexpr (RES) load8<BF16>(res, e0 + 8 * c, r[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * T;
      if (c < chunks) {
        if constexpr (RES) {
          add8(t[j], r[j]);
          store8<BF16>(stream_out, e0 + 8 * c, t[j]);
        }
        float w[8];
        load8_weight<BF16>(weight, 8 * c, w);
        absorb8(t[j], w, ss2, m);
      }
    }
  }
  float ss = ss2.x + ss2.y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, off);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  }
  if constexpr (T > 32) {
    __shared__ float2 part[T / 32];
    if ((tid & 31) == 0) part[tid >> 5] = make_float2(ss, m);
    __syncthreads();
    // every warp adds the partial sums in the same order
    const float2 p = (tid & 31) < T / 32 ? part[tid & 31] : make_float2(0.f, 0.f);
    ss = p.x;
    m = p.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, off);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
  }
  const float f = __fdiv_rn(127.0f, m);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = tid + j * T;
    if (c < chunks) *reinterpret_cast<uint2*>(codes + e0 + 8 * c) = codes8(t[j], m, f);
  }
  if (tid == 0) {
    const float rms = __fsqrt_rn(__fdiv_rn(ss, static_cast<float>(n)) + eps);
    scales[row] = m == 0.f && ss == 0.f ? 0.f : __fdiv_rn(__fdiv_rn(m, rms), 127.0f);   // eps may be 0
  }
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

template <bool BF16>
__device__ __forceinline__ void read8(const uint8_t* row, int c, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + 16 * c);
    unpack_bf16x2(w.x, v[0], v[1]);
    unpack_bf16x2(w.y, v[2], v[3]);
    unpack_bf16x2(w.z, v[4], v[5]);
    unpack_bf16x2(w.w, v[6], v[7]);
  } else {
    const float4 a = reinterpret_cast<const float4*>(row + 32 * c)[0], b = reinterpret_cast<const float4*>(row + 32 * c)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

constexpr int kMaxStages = 8;

// `stages` rows of x (and of the residual) in flight per CTA.
template <bool BF16, bool RES, int T, int NV>
__global__ void __launch_bounds__(T)
rmsnorm_ring_kernel(const void* x, const void* res, const void* weight, int64_t rows, int n, float eps,
                    void* stream_out, int8_t* __restrict__ codes, float* __restrict__ scales, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float2 part[2][T / 32];
  const int tid = threadIdx.x, chunks = n >> 3;
  const uint32_t row_bytes = static_cast<uint32_t>(n) * (BF16 ? 2 : 4);
  const uint32_t stage_bytes = row_bytes * (RES ? 2 : 1);
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) tc::mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  grid_dependency_sync();
  auto issue = [&](int64_t row, int s) {        // thread 0
    if (row >= rows) return;
    tc::mbar_arrive_expect_tx(&full[s], stage_bytes);
    bulk_load(ring + s * stage_bytes, static_cast<const uint8_t*>(x) + row * row_bytes, row_bytes, &full[s]);
    if constexpr (RES)
      bulk_load(ring + s * stage_bytes + row_bytes, static_cast<const uint8_t*>(res) + row * row_bytes, row_bytes, &full[s]);
  };
  if (tid == 0)
    for (int s = 0; s < stages; ++s) issue(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);

  int s = 0, phase = 0, turn = 0;
#pragma unroll 1
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const bool ok = tc::mbar_wait(&full[s], phase);
    if (!ok) atomicOr(&tc::hadq_tc_fault, tc::kFaultProducer);
    const uint8_t* xs = ring + s * stage_bytes;
    const int64_t e0 = row * n;
    float t[NV][8], m = 0.f;
    float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * T;
      if (c < chunks) {
        read8<BF16>(xs, c, t[j]);
        if constexpr (RES) {
          float r[8];
          read8<BF16>(xs + row_bytes, c, r);
          add8(t[j], r);
          store8<BF16>(stream_out, e0 + 8 * c, t[j]);
        }
        float w[8];
        load8_weight<BF16>(weight, 8 * c, w);
        absorb8(t[j], w, ss2, m);
      }
    }
    float ss = ss2.x + ss2.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, off);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
    if ((tid & 31) == 0) part[turn][tid >> 5] = make_float2(ss, m);
    // A wait that ran out ends the CTA (the row is not written): the vote is
    // the barrier that frees the stage and joins the sums.
    if (__syncthreads_or(!ok)) {
      if (tid == 0)                             // copies still in flight, waited for with a limit
        for (int i = 0; i < stages; ++i)
          if (row + static_cast<int64_t>(i) * gridDim.x < rows) {
            const int q = (s + i) % stages;
            if (!tc::mbar_wait(&full[q], q < s ? phase ^ 1 : phase)) break;
          }
      return;
    }
    if (tid == 0) issue(row + static_cast<int64_t>(stages) * gridDim.x, s);
    ss = 0.f;
    m = 0.f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {          // in the same order everywhere
      const float2 p = part[turn][w];
      ss += p.x;
      m = fmaxf(m, p.y);
    }
    turn ^= 1;
    if (++s == stages) s = 0, phase ^= 1;
    const float f = __fdiv_rn(127.0f, m);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * T;
      if (c < chunks) *reinterpret_cast<uint2*>(codes + e0 + 8 * c) = codes8(t[j], m, f);
    }
    if (tid == 0) {
      const float rms = __fsqrt_rn(__fdiv_rn(ss, static_cast<float>(n)) + eps);
      scales[row] = m == 0.f && ss == 0.f ? 0.f : __fdiv_rn(__fdiv_rn(m, rms), 127.0f);   // eps may be 0
    }
  }
}

}  // namespace norm
}  // namespace hadq
