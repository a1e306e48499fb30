// Matrix product of int8 codes with a scale per token and per output channel:
//   y[i][j] = (sum_k a[i][k] w[j][k]) * sa[i] * sw[j] + bias[j].
// The sum is exact in 32-bit integers (k < 131072), so its order is free.
#pragma once

#include "hadq_device.cuh"

namespace hadq {
namespace imm {

struct Args {
  const int8_t* a;
  const int8_t* w;
  const float* sa;
  const float* sw;
  const float* bias;   // nullptr: none
  void* out;
  int m, n, k;
};

// 64 x 64 outputs per CTA, four-way byte products.
template <bool OUT_BF16>
__global__ void __launch_bounds__(256) imm_plain_kernel(const __grid_constant__ Args p) {
  __shared__ int as[64][17], ws[64][17];
  grid_dependency_sync();
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += 64) {
    const int rr = threadIdx.x >> 2, cc = threadIdx.x & 3;
    int4 va = make_int4(0, 0, 0, 0), vw = va;
    if (k0 + cc * 16 < p.k) {
      if (i0 + rr < p.m) va = *reinterpret_cast<const int4*>(p.a + static_cast<int64_t>(i0 + rr) * p.k + k0 + cc * 16);
      if (j0 + rr < p.n) vw = *reinterpret_cast<const int4*>(p.w + static_cast<int64_t>(j0 + rr) * p.k + k0 + cc * 16);
    }
    as[rr][cc * 4] = va.x, as[rr][cc * 4 + 1] = va.y, as[rr][cc * 4 + 2] = va.z, as[rr][cc * 4 + 3] = va.w;
    ws[rr][cc * 4] = vw.x, ws[rr][cc * 4 + 1] = vw.y, ws[rr][cc * 4 + 2] = vw.z, ws[rr][cc * 4 + 3] = vw.w;
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = __dp4a(as[ty + 16 * u][kk], ws[tx + 16 * v][kk], acc[u][v]);
    __syncthreads();
  }
  for (int u = 0; u < 4; ++u)
    for (int v = 0; v < 4; ++v) {
      const int i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
      if (i >= p.m || j >= p.n) continue;
      float y = __int2float_rn(acc[u][v]) * p.sa[i] * p.sw[j];
      if (p.bias) y += p.bias[j];
      const int64_t e = static_cast<int64_t>(i) * p.n + j;
      if constexpr (OUT_BF16) static_cast<__nv_bfloat16*>(p.out)[e] = __float2bfloat16_rn(y);
      else static_cast<float*>(p.out)[e] = y;
    }
}

}  // namespace imm
}  // namespace hadq
