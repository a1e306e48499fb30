// Kernel entry points as the host launcher sees them.
//
// The kernels are instantiated in their own translation units
// (kernels_segment.cu, kernels_team.cu, kernels_tc.cu, kernels_tck.cu, ...), which nvcc compiles in
// parallel; each exports a lookup that returns the instantiation for a call's
// shape, output mode and sign variant.  SG selects the random Hadamard
// (signed) instantiation; the deterministic ones are compiled without any
// sign code.  A nullptr / fn == nullptr result means "no such instantiation".
#pragma once

#include <cuda.h>
#include <cstdint>

#include "hadq_device.cuh"

namespace hadq {
namespace launch {

using SegFn = void (*)(const void*, int64_t, int, float, int, void*, void*, Signs);
using SegRowFn = void (*)(const void*, int64_t, int64_t, int, float, int8_t*, float*, Signs);
using TeamFn = void (*)(const void*, int64_t, float, int, void*, void*, Signs);
using TeamRowFn = void (*)(const void*, int64_t, int64_t, float, int8_t*, float*, Signs);
using TcFn = void (*)(const CUtensorMap, const uint16_t*, int64_t, int, float, int, void*, void*, Signs);
using Tc128Fn = void (*)(const CUtensorMap, const CUtensorMap, const uint16_t*, int64_t, int, float, int, void*, void*,
                         Signs, int);
}  // namespace launch
namespace ksize {
struct StageArgs;
}
namespace kv4 {
struct AppendArgs;
struct AttnArgs;
}
namespace imm {
struct Args;
}
namespace launch {
using KsFn = void (*)(const ksize::StageArgs);

struct TcVariant {
  TcFn fn;
  int threads, smem, tile_n;
};

struct Tc128Variant {
  Tc128Fn fn;
  int threads, smem;
};

using TckFn = void (*)(const CUtensorMap, const CUtensorMap, const uint16_t*, int64_t, float, int, void*, void*, int);
using TcrFn = void (*)(const CUtensorMap, const uint16_t*, int64_t, int, float, int, void*, void*, const int32_t*,
                       const int8_t*, const double*);

struct TcrVariant {
  TcrFn fn;
  int threads, smem;
};

struct TckVariant {
  TckFn fn;
  int threads, smem, np;   // np: MMA N = chunks per block rounded up to 16
};

// Segment kernels (b <= 128): log2 of the per-thread segment `logs`, FULL when
// b equals the segment.  mode: OutMode.
SegFn segment_kernel_for(bool bf16, bool full, int logs, int mode, bool sg);
SegRowFn segment_row_kernel_for(bool bf16, bool full, int logs, bool sg);

// Team kernels (256 <= b <= 8192); one unit per input dtype
// (kernels_team.cu: fp32 and the dispatch, kernels_team_bf16.cu: bf16).
TeamFn team_kernel_for(bool bf16, int logb, int mode, bool sg);
TeamRowFn team_row_kernel_for(bool bf16, int logb, bool sg);
TeamFn team_kernel_bf16(int logb, int mode, bool sg);
TeamRowFn team_row_kernel_bf16(int logb, bool sg);

// Tensor-core kernels: full size 2^(7 + lo), lo = 5 or 6; block 128 (mode -1 =
// per-token int8).
TcVariant tc_kernel_for(int lo, int mode, int side);   // side: hadq::SignSide
// Block-128 kernel; e > 0: blocks of 2^e * 128 (1 <= e <= 4), the last e
// stages across neighbouring lanes, no signs and no per-token int8.
Tc128Variant tc128_kernel_for(int mode, int e);   // e = 0: signs of either side folded into B
TcrVariant tcr_kernel_for(int mode);       // RPBH at full size 4096 (permutation gathered in shared memory)

// Shared-memory staged kernels: blocks of K * 2^m elements (K a covered Paley
// order 12 .. 108, or 1 with the RPBH permutation or the codebook quantizer);
// shi = pieces of the 2^m factor mixed in the column stage; mode -1 =
// per-token int8; sgk: ksize::StageSigns.  One unit per input dtype
// (kernels_ksize.cu: fp32 and the dispatch, kernels_ksize_bf16.cu: bf16).
KsFn staged_kernel_for(int k, int shi, bool bf16, int mode, int sgk);
KsFn staged_kernel_f32(int k, int shi, int mode, int sgk);
KsFn staged_kernel_bf16(int k, int shi, int mode, int sgk);

// Tensor-core kernels for blocks of K * 128 * hi elements (K a Paley order,
// K * hi <= 128 chunks of 128); mode OUT_F32 / OUT_BF16, -1 = per-token int8
// (block = row), or OUT_INT4 / OUT_MXFP4 / OUT_NVFP4.
TckVariant tck_kernel_for(int k, int hi, int mode);

// Norm kernels: rows per CTA and threads of the variant for a row length, and
// the kernel for many rows (its ring in dynamic shared memory).
using NormFn = void (*)(const void*, const void*, const void*, int64_t, int, float, void*, int8_t*, float*);
struct NormVariant {
  NormFn fn;
  int threads, rows_per_cta;
};
NormVariant norm_kernel_for(bool bf16, bool residual, int64_t rows, int64_t n);
using NormRingFn = void (*)(const void*, const void*, const void*, int64_t, int, float, void*, int8_t*, float*, int);
struct NormRingVariant {
  NormRingFn fn;
  int threads;
};
NormRingVariant norm_ring_for(bool bf16, bool residual, int64_t n);
int norm_fault_bits(int clear);

// int8 matrix product: the kernels for up to 4 and 16 tokens (imm::kRowWarps
// warps), the one for few (up to `tokens` per CTA) and the one for many.
using ImmRowFn = void (*)(const imm::Args, int);
ImmRowFn imm_row_for(int64_t m, bool out_bf16);
struct ImmWarpVariant {
  ImmRowFn fn;
  int channels, tokens;   // of a warp
};
ImmWarpVariant imm_warp_for(int64_t m, bool two, bool out_bf16);   // m <= 16; two: 32 channels a warp
using ImmSplitFn = void (*)(const CUtensorMap, const CUtensorMap, const imm::Args, int, int);
using ImmPairFn = void (*)(const CUtensorMap, const CUtensorMap, const imm::Args);
struct ImmSplitVariant {
  ImmSplitFn fn;
  int threads, smem, tokens, ctas;           // ctas: on an SM
};
struct ImmPairVariant {
  ImmPairFn fn;
  int threads, smem;
};
ImmSplitVariant imm_split_for(int64_t m, bool half, bool out_bf16);
ImmPairVariant imm_pair_for(bool out_bf16);
int imm_fault_bits(int clear);

// int4 cache: append, and attention for `rows` query rows per K/V head: the
// kernel (variant.rows of them per CTA, variant.ctas CTAs at once on an SM) and
// the join of its splits (at most `pieces` warps a row).
using AppendFn = void (*)(const kv4::AppendArgs);
using AttnFn = void (*)(const kv4::AttnArgs);
struct AttnVariant {
  AttnFn fn, join;
  int threads, smem, rows, ctas, pieces;
};
AppendFn kv4_append_for(bool bf16, int d);
AttnVariant kv4_attention_for(int d, int group, int rows);
int kv4_fault_bits(int clear);

// The tensor-core kernels' sticky fault words (bounded waits that ran out),
// one per translation unit; cleared when `clear` is non-zero.  -1 on a CUDA
// error.
int tc_fault_bits(int clear);
int tck_fault_bits(int clear);

}  // namespace launch
}  // namespace hadq
