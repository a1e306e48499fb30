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
// one barrier joins the warps' (sum, max) pairs.
#pragma once

#include "hadq_device.cuh"

namespace hadq {
namespace norm {

// 8 consecutive elements; x may be the buffer that the kernel also writes, so
// no read-only-cache load.
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t e, float (&v)[8]) {
  if constexpr (BF16) {
    uint4 w;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(static_cast<const uint16_t*>(p) + e));
    unpack_bf16x2(w.x, v[0], v[1]);
    unpack_bf16x2(w.y, v[2], v[3]);
    unpack_bf16x2(w.z, v[4], v[5]);
    unpack_bf16x2(w.w, v[6], v[7]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                   : "l"(static_cast<const float*>(p) + e + 4 * h));
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

// Rounds v to the stored type, in place, and stores it.
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t e, float (&v)[8]) {
  if constexpr (BF16) {
    uint4 w;
    w.x = pack_bf16x2(v[0], v[1]);
    w.y = pack_bf16x2(v[2], v[3]);
    w.z = pack_bf16x2(v[4], v[5]);
    w.w = pack_bf16x2(v[6], v[7]);
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

// The nearest whole number to 127 t / m, ties to even, for |t| <= m.  A
// quotient in 64 bits decides: with 24-bit t and m, a quotient of at least a
// quarter that is not exactly k + 1/2 is at least 2^-35 from it, and the
// 53-bit rounding (2^-47 below 128) cannot reach or cross it.
__device__ __noinline__ int exact_code(float t, float m) {
  return m > 0.f ? __double2int_rn(127.0 * static_cast<double>(t) / static_cast<double>(m)) : 0;
}

// Eight codes of t against the row's m, f = 127 / m.  The fp32 product is off
// by at most 127 * 2^-23 < 1.6e-5 code units (two roundings), so it decides
// unless it is within 4e-5 of a half; then the quotient in 64 bits does.
__device__ __forceinline__ uint2 codes8(const float (&t)[8], float m, float f) {
  float far = 0.f;
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = t[i] * f;
    const float r = __fadd_rn(p, kRoundMagic);
    b[i] = __float_as_uint(r);
    far = fmaxf(far, fabsf(p - __fsub_rn(r, kRoundMagic)));
  }
  if (!(far < 0.49996f) || !(m > 1.0e-30f)) {   // tiny m: f may be infinite
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = static_cast<uint32_t>(exact_code(t[i], m));
  }
  const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return make_uint2(lo, hi);
}

// CTAs of T threads times RPC rows; T = 32 takes a warp per row (no barrier).
template <bool BF16, bool RES, int T, int RPC, int NV>
__global__ void __launch_bounds__(T * RPC)
rmsnorm_quant_kernel(const void* x, const void* res, const void* __restrict__ weight, int64_t rows, int n, float eps,
                     void* stream_out, int8_t* __restrict__ codes, float* __restrict__ scales) {
  static_assert(T == 32 || RPC == 1, "rows of several warps have a CTA of their own");
  grid_dependency_sync();
  const int tid = threadIdx.x % T;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPC + threadIdx.x / T;
  if (row >= rows) return;                      // whole warps (T = 32) or never (RPC = 1)
  const int64_t e0 = row * n;
  const int chunks = n >> 3;

  float t[NV][8];
  float ss = 0.f, m = 0.f;
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
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j][i] = __fadd_rn(t[j][i], r[j][i]);
          store8<BF16>(stream_out, e0 + 8 * c, t[j]);
        }
        float w[8];
        load8_weight<BF16>(weight, 8 * c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(t[j][i], t[j][i], ss);
          t[j][i] = __fmul_rn(t[j][i], w[i]);
          m = fmaxf(m, fabsf(t[j][i]));
        }
      }
    }
  }
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
    scales[row] = __fdiv_rn(__fdiv_rn(m, rms), 127.0f);
  }
}

}  // namespace norm
}  // namespace hadq
