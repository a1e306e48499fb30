// Host side of the operators around the rotation: the int8 norm and matrix
// product, and the int4 cache.  As everywhere in the library every check runs
// before the first CUDA call, and nothing is allocated.
#include "hadq_host.h"
#include "hadq_imm.cuh"
#include "hadq_kv4.cuh"
#include "hadq_launch.h"
#include "hadq_norm.cuh"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

namespace {

using namespace hadq::host;
namespace hl = hadq::launch;

// No exception leaves a C entry point (host memory can run out in a message
// or a launch cache).
template <typename F>
hadq_status entry(F&& body) {
  try {
    clear_error();
    return body();
  } catch (...) {
    return HADQ_ERR_CUDA;
  }
}

hadq_status invalid(const char* msg) { return fail(HADQ_ERR_INVALID_ARG, msg); }
hadq_status unsupported(const char* msg) { return fail(HADQ_ERR_UNSUPPORTED, msg); }

bool dtype_ok(hadq_dtype d) { return d == HADQ_F32 || d == HADQ_BF16; }

// Outputs must not overlap an input or one another.
hadq_status disjoint(const Span* outs, int nouts, const Span* ins, int nins, const char* msg) {
  for (int i = 0; i < nouts; ++i) {
    for (int j = 0; j < nins; ++j)
      if (overlaps(outs[i], ins[j])) return invalid(msg);
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return invalid(msg);
  }
  return HADQ_OK;
}

constexpr int64_t kMaxNormN = 32768;
// Whether many rows of `stage` input bytes each go through the ring kernel, and
// how many a CTA holds: three or more, in as many CTAs (up to 4) as the shared
// memory allows.  Rows of up to 2048 are short enough without; up to 4096 it
// pays from thousands of rows (2000 rows: 12.9 us against 11.7), above from
// hundreds (2000 rows of 8192: 23.0 against 24.5).  The widest rows take 512
// threads, one CTA to an SM, which needs 32 KB rows to keep the memory busy
// (14336, no residual: bf16 109 us against 90, fp32 127 against 173).
bool norm_takes_ring(int64_t rows, int64_t n, int64_t stage, int* stages) {
  if (n <= 2048 || n > 16384 || rows < (n <= 4096 ? 4096 : 1000)) return false;
  if (n > 8192 && stage < 32 * 1024) return false;
  constexpr int64_t kRoom = 220 * 1024;
  const int64_t ctas = n > 8192 ? 1 : std::min<int64_t>(std::max<int64_t>(kRoom / (3 * stage), 1), 4);
  *stages = static_cast<int>(std::min<int64_t>(kRoom / ctas / stage, hadq::norm::kMaxStages));
  return *stages >= 2;
}

constexpr int64_t kMaxK = 131071;        // 128 * 128 * k < 2^31
constexpr int64_t kMaxDim = int64_t(1) << 30;

// A tensor map over a row-major int8 matrix: boxes of 128 bytes of k times
// `box_rows` rows, 128-byte swizzle, zeros outside.
hadq_status int8_map(const int8_t* p, int64_t rows, int64_t k, int box_rows, CUtensorMap* map) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
  if (encode == nullptr) return fail(HADQ_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(k)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(hadq::imm::kSlice), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? HADQ_OK : fail(HADQ_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

hadq_status launch_imm(hadq::imm::Args p, bool out_bf16, cudaStream_t stream) {
  if (p.m <= 4) {
    // k is divided among a CTA's warps until there are two CTAs to an SM, as
    // long as a warp has four rounds over it (1 x 4096 x 14336 undivided
    // took 14.5 us where divided it took 11.6).
    const int64_t rounds = ceil_div(p.k, 512);
    int parts = 1;
    while (parts < 8 && ceil_div(p.n, 32 / parts) < 148 * 2 && rounds >= 8 * parts) parts *= 2;
    return launch_result(launch_pdl(hl::imm_row_for(p.m, out_bf16), ceil_div(p.n, 32 / parts), 32 * hadq::imm::kRowWarps, 0,
                                    stream, p, parts),
                         "int8 matrix product launch");
  }
  int sms = 0, dev = 0, occ = 0;
  hadq_status st = device_sms(&sms, &dev);
  if (st != HADQ_OK) return st;
  if (p.m <= 16) {
    // 32 channels a warp where that still makes a CTA for every SM (14336 x 4096
    // with 8 tokens: 10.4 us against 14.9 with 16), k divided until there is one
    // and a warp has eight rounds over it.
    const bool two = p.n >= 8192;
    const hl::ImmWarpVariant v = hl::imm_warp_for(p.m, two, out_bf16);
    const int64_t rounds = ceil_div(p.k, 64);
    int parts = 1;
    while (parts < 8 && ceil_div(p.n, v.channels * (8 / parts)) < 148 && rounds >= 8 * parts) parts *= 2;
    const int smem = 8 / parts * v.channels * v.tokens * 4;
    return launch_result(launch_pdl(v.fn, ceil_div(p.n, v.channels * (8 / parts)), 32 * hadq::imm::kRowWarps, smem, stream, p, parts),
                         "int8 matrix product launch");
  }
  CUtensorMap map_a, map_w;
  const int64_t pair_tiles = ceil_div(p.m, 256) * ceil_div(p.n, 256);
  // Many tokens: from 40 tiles of 256 x 256 on, half of the GPU's 74 pairs.
  // 768 x 4096 x 4096 (48 tiles) takes 17.7 us in pairs and 30.8 split, 512 x
  // 4096 x 4096 (32 tiles) 16.7 and 16.3.  Up to 128 tokens half of a tile is
  // empty, and pairs pay once the split kernel's tiles no longer fit the SMs at
  // once: 96 x 28672 x 4096 (112 tiles) 30.9 and 34.1, 96 x 14336 x 4096 (56) 18.3
  // and 17.6.
  if (p.m > 128 ? pair_tiles >= 40 : p.m > 64 && pair_tiles > sms / 2) {
    const hl::ImmPairVariant v = hl::imm_pair_for(out_bf16);
    st = occupancy(reinterpret_cast<const void*>(v.fn), dev, v.threads, v.smem, &occ);
    if (st == HADQ_OK) st = int8_map(p.a, p.m, p.k, 128, &map_a);
    if (st == HADQ_OK) st = int8_map(p.w, p.n, p.k, 128, &map_w);
    if (st != HADQ_OK) return st;
    if (pair_tiles > INT32_MAX) return unsupported("too many output tiles");
    const int64_t grid = 2 * std::min<int64_t>(pair_tiles, sms / 2);
    return launch_result(launch_pdl3(v.fn, dim3(static_cast<unsigned>(grid)), 2, v.threads, v.smem, stream, map_a, map_w, p),
                         "int8 matrix product launch");
  }
  // Tiles that do not fit the SMs at once share them, two to an SM with half the
  // ring each, where the rings are small enough: 48 x 28672 x 4096 22.9 us, 28.2
  // with one; 48 x 14336 x 4096 fits, 13.7 with the whole ring and 15.7 with half.
  // Above 64 tokens such tiles of 64 tokens also beat those of 128, whose joins and
  // epilogues are longer, until reading the weights again outweighs it, at about 14
  // slices of a 128 x 128 tile an SM: 128 x 2048 x 4096 (512 slices) 7.5 and 8.5 us,
  // 96 x 6144 x 4096 (1536) 12.2 and 13.1, 256 x 4096 x 4096 (2048) 12.9 and 13.0,
  // 333 x 4096 x 4096 (half as much again) 16.0 and 15.3, 200 x 8192 x 8192 (8192) 27.9 and 25.7;
  // against the rule 333 x 1001 x 4112 (792) 10.1 and 9.6.
  const int64_t work = ceil_div(p.m, 128) * ceil_div(p.n, 128) * ceil_div(p.k, hadq::imm::kSlice);
  const bool half = p.m > 64 ? work < 14 * sms : ceil_div(p.n, 128) > sms;
  const hl::ImmSplitVariant v = hl::imm_split_for(p.m, half, out_bf16);
  st = occupancy(reinterpret_cast<const void*>(v.fn), dev, v.threads, v.smem, &occ);
  const int64_t token_tiles = ceil_div(p.m, v.tokens);
  p.tokens = static_cast<int>(ceil_div(ceil_div(p.m, token_tiles), 8) * 8);
  if (st == HADQ_OK) st = int8_map(p.a, p.m, p.k, p.tokens, &map_a);
  if (st == HADQ_OK) st = int8_map(p.w, p.n, p.k, 128, &map_w);
  if (st != HADQ_OK) return st;
  const int64_t tiles = ceil_div(p.n, 128) * token_tiles;
  const int64_t slices = ceil_div(p.k, hadq::imm::kSlice);
  // k is split as long as every CTA is resident at once (333 x 1001 x 4112: 13.5
  // us with 48 CTAs, 10.0 with 96, 17.0 with 192; 48 x 2048 x 4096: 6.5 with 64,
  // 10.3 with 128 in clusters of 8, of which 15 fit) and has four slices, or eight
  // where two CTAs share an SM (24 tokens, 4096 x 14336: 13.4 with 256 CTAs, 14.8
  // with 128; 4096 x 4096: 7.2 and 6.9).
  int splits = 1;
  for (; splits < 8; splits *= 2) {
    const int64_t ctas = tiles * splits * 2;
    // what fits at once (of 148 SMs): clusters of 4 and 8 leave some SMs of a GPC without a CTA
    const int lost = splits == 4 ? (v.ctas > 1 ? 16 : 28) : splits == 2 ? (v.ctas > 1 ? 6 : 16) : 0;
    if (ctas > int64_t(sms - lost) * v.ctas || slices < (ctas <= sms ? 4 : 8) * 2 * splits) break;
  }
  if (tiles * splits > INT32_MAX) return unsupported("too many output tiles");
  return launch_result(launch_pdl3(v.fn, dim3(static_cast<unsigned>(tiles * splits)), splits, v.threads, v.smem, stream, map_w,
                                   map_a, p, splits, static_cast<int>(token_tiles)),
                       "int8 matrix product launch");
}

// What the two cache entry points share.
struct Cache {
  int64_t kv_heads, head_dim, group, num_pages, page_size;
  const void *k_codes, *k_scales, *v_codes, *v_scales;
};

hadq_status check_cache_shape(const Cache& c) {
  if (c.kv_heads <= 0 || c.num_pages <= 0 || c.page_size <= 0) return invalid("kv_heads, num_pages and page_size must be > 0");
  if (c.group != 32 && c.group != 64 && c.group != 128) return invalid("int4 group must be 32, 64 or 128");
  if (c.head_dim != 64 && c.head_dim != 128) return unsupported("head_dim must be 64 or 128");
  if (c.head_dim % c.group != 0) return invalid("int4 group must divide head_dim");
  if (c.page_size % 16 != 0) return unsupported("page_size must be a multiple of 16");
  if (c.page_size > kMaxDim || c.num_pages > kMaxDim || c.num_pages * c.page_size > INT32_MAX)
    return unsupported("the cache must hold fewer than 2^31 positions");
  if (c.kv_heads > 65536) return unsupported("at most 65536 K/V heads");
  if (c.num_pages * c.page_size / 16 * c.kv_heads > UINT32_MAX - 1) return unsupported("the cache is larger than any device's memory");
  return HADQ_OK;
}

hadq_status check_cache_pointers(const Cache& c, Span (&spans)[4]) {
  if (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales) return invalid("null pointer");
  if (!aligned16(c.k_codes) || !aligned16(c.k_scales) || !aligned16(c.v_codes) || !aligned16(c.v_scales))
    return fail(HADQ_ERR_MISALIGNED, "the cache's pointers must be 16-byte aligned");
  const int64_t cells = c.num_pages * c.page_size * c.kv_heads;
  const int64_t cb = cells * (c.head_dim / 2), sb = cells * (c.head_dim / c.group) * 2;
  spans[0] = span(c.k_codes, cb);
  spans[1] = span(c.k_scales, sb);
  spans[2] = span(c.v_codes, cb);
  spans[3] = span(c.v_scales, sb);
  return disjoint(spans, 4, nullptr, 0, "the cache's four tensors must not overlap");
}

hadq::kv4::Divider divider(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return hadq::kv4::Divider{static_cast<uint32_t>((uint64_t(1) << (31 + s)) / d + 1), s, d};
}

// block: the whole head, or 1 (H_1: none).
hadq_status check_block(int64_t block, int64_t head_dim, int* rotate) {
  if (block == 0 || block == -1 || block == head_dim) *rotate = 1;
  else if (block == 1) *rotate = 0;
  else return unsupported("block must be 0 or head_dim (each head rotated in full) or 1 (no rotation)");
  return HADQ_OK;
}

hadq_status check_attention_shape(int64_t batch, int64_t q_len, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                  int64_t max_positions) {
  if (batch < 0) return invalid("batch must be >= 0");
  if (q_len < 1 || heads < 1 || kv_heads < 1) return invalid("q_len, heads and kv_heads must be > 0");
  if (heads % kv_heads != 0) return invalid("heads must be a multiple of kv_heads");
  if (head_dim != 64 && head_dim != 128) return unsupported("head_dim must be 64 or 128");
  if (q_len > 64) return unsupported("q_len above 64: this call is for the newest tokens of a sequence");
  if (heads > 65536 || batch > kMaxDim) return unsupported("batch or heads too large");
  if (max_positions < 1) return invalid("max_pages must be > 0");
  if (max_positions > kMaxDim) return unsupported("sequences of more than 2^30 positions");
  if (batch * q_len * heads > INT32_MAX) return unsupported("batch * q_len * heads too large");
  return HADQ_OK;
}

// Splits of a sequence over CTAs, from sizes alone, so that a captured call and
// its workspace hold for any lengths.  Few units: 256 CTAs, under two to an SM (a
// grid that just fills two leaves some SMs with three), as long as each of their
// warps has a step of 32 positions, but no more than 32 splits (the join then
// takes one round), or twice that where it leaves a warp more than 16 steps.
// (Device us, 8 units: 32768 positions 14.2 with 32 splits, 16.4 with 37, 17.3
// with 16; 8192 positions 8.2, 9.6, 8.4; 131072 positions 36.0 with 64, 43.5 with
// 37.  32 units of 8192: 13.8 with 8 splits, 16.2 with 9.)
// Many: about 1.75 for each CTA that fits the GPU at once, so that a second,
// shorter round evens out unequal lengths (512 units of 4096: 60.7 us with 2
// splits, 64.3 with 1, 64.4 with 3).
int attention_splits(const hl::AttnVariant& v, int64_t units, int64_t max_positions) {
  const int64_t slots = 148 * v.ctas, steps = ceil_div(max_positions, 32), some = std::max<int64_t>(units, 1);
  int64_t want = (7 * slots + 2 * some) / (4 * some);
  if (some <= 256) want = steps <= 64 * 32 ? std::min<int64_t>(256 / some, 32) : std::min<int64_t>(512 / some, 64);
  return static_cast<int>(std::max<int64_t>(1, std::min(want, steps / 4)));
}

// Sequences by length where the grid's end would otherwise wait for a long one:
// more CTAs than fit at once, but no more than three times as many, of 1024
// positions or more.  (Device us in this order and as they come: 64 sequences of
// 0 to 6000 positions, 512 CTAs of 296 places, 76.6 and 103; of 1792 to 3584, 73.4
// and 82.7; all of 3584, 97.5 and 97.3; 1024 CTAs of 592 places, 118 and 126, equal
// lengths 145 and 144.  What the counting costs shows with many or short CTAs: 3200
// of 296 places 103 and 99, 2048 of 592 with 256 positions 32.4 and 30.4.)
bool longest_first(const hl::AttnVariant& v, int64_t ctas, int64_t positions) {
  const int64_t slots = 148 * v.ctas;
  return ctas > slots && ctas <= 3 * slots && positions >= 1024;
}

int64_t attention_units(const hl::AttnVariant& v, int64_t batch, int64_t rows, int64_t kv_heads) {
  return batch * kv_heads * ceil_div(rows, v.rows);
}

int64_t attention_workspace(const hl::AttnVariant& v, int64_t units, int splits, int64_t head_dim) {
  return splits == 1 ? 0 : splits * units * v.rows * (head_dim + 2) * 4;
}

}  // namespace

extern "C" {

hadq_status hadq_rmsnorm_quant(const void* x, hadq_dtype x_dtype, int64_t rows, int64_t n, const void* residual,
                               const void* weight, float eps, void* residual_out, int8_t* codes, float* scales,
                               void* stream) {
  return entry([&]() -> hadq_status {
    if (!dtype_ok(x_dtype)) return invalid("x_dtype must be HADQ_F32 or HADQ_BF16");
    if (rows < 0) return invalid("rows must be >= 0");
    if (n <= 0) return invalid("n must be > 0");
    if (!(std::isfinite(eps) && eps >= 0.f)) return invalid("eps must be finite and >= 0");
    if (n % 8 != 0) return unsupported("n must be a multiple of 8");
    if (n > kMaxNormN) return unsupported("the norm supports n <= 32768");
    if (rows > INT64_MAX / 8 / n) return invalid("rows * n overflows");
    if ((residual == nullptr) != (residual_out == nullptr) && rows > 0)
      return invalid("residual and residual_out are given together or not at all");
    if (rows == 0) return HADQ_OK;
    if (!x || !weight || !codes || !scales) return invalid("null pointer");
    if (!aligned16(x) || !aligned16(weight) || !aligned16(codes) || !aligned16(scales) || !aligned16(residual) ||
        !aligned16(residual_out))
      return fail(HADQ_ERR_MISALIGNED, "every pointer must be 16-byte aligned");
    const int64_t bytes = rows * n * esize(x_dtype);
    const Span outs[3] = {span(codes, rows * n), span(scales, rows * 4), span(residual_out, residual ? bytes : 0)};
    const Span ins[3] = {span(x, bytes), span(weight, n * esize(x_dtype)), span(residual, residual ? bytes : 0)};
    hadq_status st = disjoint(outs, 2, ins, 3, "codes and scales must not overlap an input or each other");
    if (st != HADQ_OK) return st;
    if (residual) {
      for (int i = 0; i < 3; ++i)
        if (overlaps(outs[2], ins[i]) && !(i != 1 && outs[2].lo == ins[i].lo))
          return invalid("residual_out may be x or residual, and must not overlap an input otherwise");
      if (overlaps(outs[2], outs[0]) || overlaps(outs[2], outs[1])) return invalid("outputs must not overlap");
    }
    int stages = 0;
    const int64_t row_in = n * esize(x_dtype) * (residual ? 2 : 1);
    if (norm_takes_ring(rows, n, row_in, &stages)) {
      const hl::NormRingVariant v = hl::norm_ring_for(x_dtype == HADQ_BF16, residual != nullptr, n);
      int sms = 0, dev = 0, occ = 0;
      st = device_sms(&sms, &dev);
      if (st != HADQ_OK) return st;
      const int smem = static_cast<int>(stages * row_in);
      st = occupancy(reinterpret_cast<const void*>(v.fn), dev, v.threads, smem, &occ);
      if (st != HADQ_OK) return st;
      return launch_result(launch_pdl(v.fn, std::min<int64_t>(rows, int64_t(sms) * occ), v.threads, smem,
                                      static_cast<cudaStream_t>(stream), x, residual, weight, rows, static_cast<int>(n), eps,
                                      residual_out, codes, scales, stages),
                           "norm kernel launch");
    }
    const hl::NormVariant v = hl::norm_kernel_for(x_dtype == HADQ_BF16, residual != nullptr, rows, n);
    const int64_t grid = ceil_div(rows, v.rows_per_cta);
    if (grid > INT32_MAX) return unsupported("too many rows");
    return launch_result(launch_pdl(v.fn, grid, v.threads, 0, static_cast<cudaStream_t>(stream), x, residual, weight,
                                    rows, static_cast<int>(n), eps, residual_out, codes, scales),
                         "norm kernel launch");
  });
}

hadq_status hadq_matmul_int8(const int8_t* a, const float* a_scales, int64_t rows, const int8_t* w,
                             const float* w_scales, int64_t cols, int64_t k, const float* bias, void* out,
                             hadq_dtype out_dtype, void* stream) {
  return entry([&]() -> hadq_status {
    if (!dtype_ok(out_dtype)) return invalid("out_dtype must be HADQ_F32 or HADQ_BF16");
    if (rows < 0 || cols < 0) return invalid("rows and cols must be >= 0");
    if (k <= 0) return invalid("k must be > 0");
    if (k % 16 != 0) return unsupported("k must be a multiple of 16");
    if (k > kMaxK) return unsupported("k above 131071 could leave 32-bit sums");
    if (rows > kMaxDim || cols > kMaxDim) return unsupported("rows and cols must be at most 2^30");
    if (rows == 0 || cols == 0) return HADQ_OK;
    if (!a || !a_scales || !w || !w_scales || !out) return invalid("null pointer");
    if (!aligned16(a) || !aligned16(a_scales) || !aligned16(w) || !aligned16(w_scales) || !aligned16(bias) ||
        !aligned16(out))
      return fail(HADQ_ERR_MISALIGNED, "every pointer must be 16-byte aligned");
    const Span o = span(out, rows * cols * esize(out_dtype));
    const Span ins[5] = {span(a, rows * k), span(a_scales, rows * 4), span(w, cols * k), span(w_scales, cols * 4),
                         span(bias, bias ? cols * 4 : 0)};
    hadq_status st = disjoint(&o, 1, ins, 5, "out must not overlap an input");
    if (st != HADQ_OK) return st;
    const hadq::imm::Args p{a, w, a_scales, w_scales, bias, out, static_cast<int>(rows), static_cast<int>(cols),
                            static_cast<int>(k), 0};
    return launch_imm(p, out_dtype == HADQ_BF16, static_cast<cudaStream_t>(stream));
  });
}

hadq_status hadq_kv4_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, hadq_dtype dtype,
                            int64_t tokens, int64_t kv_heads, int64_t head_dim, int64_t block, int64_t group,
                            const int64_t* slots, int64_t num_pages, int64_t page_size, void* k_codes, void* k_scales,
                            void* v_codes, void* v_scales, void* stream) {
  return entry([&]() -> hadq_status {
    if (!dtype_ok(dtype)) return invalid("dtype must be HADQ_F32 or HADQ_BF16");
    if (tokens < 0) return invalid("tokens must be >= 0");
    const Cache c{kv_heads, head_dim, group, num_pages, page_size, k_codes, k_scales, v_codes, v_scales};
    hadq_status st = check_cache_shape(c);
    if (st != HADQ_OK) return st;
    int rotate = 0;
    st = check_block(block, head_dim, &rotate);
    if (st != HADQ_OK) return st;
    const int64_t width = kv_heads * head_dim, unit = 16 / esize(dtype);
    if (k_stride < width || v_stride < width) return invalid("k_stride and v_stride must be at least kv_heads * head_dim");
    if (k_stride % unit != 0 || v_stride % unit != 0) return fail(HADQ_ERR_MISALIGNED, "k_stride and v_stride must be multiples of 16 bytes");
    if (tokens > kMaxDim || k_stride > kMaxDim || v_stride > kMaxDim) return unsupported("tokens and strides must be at most 2^30");
    if (tokens * kv_heads > INT32_MAX) return unsupported("tokens * kv_heads must be below 2^31");
    if (tokens == 0) return HADQ_OK;
    if (!k || !v || !slots) return invalid("null pointer");
    if (!aligned16(k) || !aligned16(v) || !aligned16(slots)) return fail(HADQ_ERR_MISALIGNED, "k, v and slots must be 16-byte aligned");
    Span outs[4];
    st = check_cache_pointers(c, outs);
    if (st != HADQ_OK) return st;
    const int64_t es = esize(dtype);
    const Span ins[3] = {span(k, ((tokens - 1) * k_stride + width) * es), span(v, ((tokens - 1) * v_stride + width) * es),
                         span(slots, tokens * 8)};
    st = disjoint(outs, 4, ins, 3, "the cache must not overlap k, v or slots");
    if (st != HADQ_OK) return st;
    hadq::kv4::AppendArgs p;
    p.x[0] = k, p.x[1] = v;
    p.stride[0] = k_stride, p.stride[1] = v_stride;
    p.codes[0] = static_cast<uint8_t*>(k_codes), p.codes[1] = static_cast<uint8_t*>(v_codes);
    p.scales[0] = static_cast<__half*>(k_scales), p.scales[1] = static_cast<__half*>(v_scales);
    p.slots = slots;
    p.rows = static_cast<uint32_t>(tokens * kv_heads);
    p.num_slots = num_pages * page_size;
    p.kv_heads = divider(static_cast<uint32_t>(kv_heads));
    p.page_size = divider(static_cast<uint32_t>(page_size));
    p.group = static_cast<int>(group);
    p.rotate_k = rotate;
    p.norm = static_cast<float>(1.0 / std::sqrt(static_cast<double>(head_dim)));
    const hl::AppendFn fn = hl::kv4_append_for(dtype == HADQ_BF16, static_cast<int>(head_dim));
    const int64_t grid = 2 * ceil_div(tokens * kv_heads * (head_dim / 32), 256);
    return launch_result(launch_pdl(fn, grid, 256, 0, static_cast<cudaStream_t>(stream), p), "cache append launch");
  });
}

int64_t hadq_kv4_attention_workspace(int64_t batch, int64_t q_len, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                     int64_t max_positions) {
  int64_t bytes = -1;
  const hadq_status st = entry([&]() -> hadq_status {
    const hadq_status s = check_attention_shape(batch, q_len, heads, kv_heads, head_dim, max_positions);
    if (s != HADQ_OK) return s;
    const int64_t rows = q_len * (heads / kv_heads);
    // every group's variant has the same shape
    const hl::AttnVariant v = hl::kv4_attention_for(static_cast<int>(head_dim), 32, static_cast<int>(rows));
    const int64_t units = attention_units(v, batch, rows, kv_heads);
    bytes = batch == 0 ? 0 : attention_workspace(v, units, attention_splits(v, units, max_positions), head_dim);
    return HADQ_OK;
  });
  return st == HADQ_OK ? bytes : -1;
}

hadq_status hadq_kv4_attention(const void* q, int64_t q_stride, hadq_dtype dtype, int64_t batch, int64_t q_len,
                               int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t block, int64_t group,
                               const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                               int64_t num_pages, int64_t page_size, const int32_t* page_table, int64_t max_pages,
                               const int32_t* lengths, float scale, void* out, void* workspace, int64_t workspace_bytes,
                               void* stream) {
  return entry([&]() -> hadq_status {
    if (!dtype_ok(dtype)) return invalid("dtype must be HADQ_F32 or HADQ_BF16");
    if (dtype != HADQ_BF16) return unsupported("attention takes bf16 queries");
    const Cache c{kv_heads, head_dim, group, num_pages, page_size, k_codes, k_scales, v_codes, v_scales};
    hadq_status st = check_cache_shape(c);
    if (st != HADQ_OK) return st;
    if (max_pages < 1 || max_pages > kMaxDim) return invalid("max_pages must be > 0");
    st = check_attention_shape(batch, q_len, heads, kv_heads, head_dim, max_pages * page_size);
    if (st != HADQ_OK) return st;
    int rotate = 0;
    st = check_block(block, head_dim, &rotate);
    if (st != HADQ_OK) return st;
    if (!std::isfinite(scale)) return invalid("scale must be finite");
    if (q_stride < heads * head_dim) return invalid("q_stride must be at least heads * head_dim");
    if (q_stride % 8 != 0) return fail(HADQ_ERR_MISALIGNED, "q_stride must be a multiple of 16 bytes");
    if (q_stride > kMaxDim) return unsupported("q_stride must be at most 2^30");
    if (batch == 0) return HADQ_OK;
    if (!q || !page_table || !lengths || !out) return invalid("null pointer");
    if (!aligned16(q) || !aligned16(page_table) || !aligned16(lengths) || !aligned16(out) || !aligned16(workspace))
      return fail(HADQ_ERR_MISALIGNED, "every pointer must be 16-byte aligned");
    Span cache[4];
    st = check_cache_pointers(c, cache);
    if (st != HADQ_OK) return st;
    const int ratio = static_cast<int>(heads / kv_heads);
    const int64_t rows = q_len * ratio;
    const hl::AttnVariant v = hl::kv4_attention_for(static_cast<int>(head_dim), static_cast<int>(group), static_cast<int>(rows));
    if (v.fn == nullptr) return unsupported("no attention kernel for this head_dim and group");
    const int64_t units = attention_units(v, batch, rows, kv_heads);
    const int splits = attention_splits(v, units, max_pages * page_size);
    const int64_t need = attention_workspace(v, units, splits, head_dim);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
      return invalid("workspace is smaller than hadq_kv4_attention_workspace says");
    const int64_t out_rows = batch * q_len * heads;
    const Span outs[2] = {span(out, out_rows * head_dim * 2), span(workspace, need)};
    const Span ins[7] = {span(q, ((batch * q_len - 1) * q_stride + heads * head_dim) * 2), span(page_table, batch * max_pages * 4),
                         span(lengths, batch * 4), cache[0], cache[1], cache[2], cache[3]};
    st = disjoint(outs, need > 0 ? 2 : 1, ins, 7, "out and workspace must not overlap an input or each other");
    if (st != HADQ_OK) return st;
    hadq::kv4::AttnArgs p;
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride = q_stride;
    p.k_codes = static_cast<const uint8_t*>(k_codes);
    p.k_scales = static_cast<const __half*>(k_scales);
    p.v_codes = static_cast<const uint8_t*>(v_codes);
    p.v_scales = static_cast<const __half*>(v_scales);
    p.table = page_table;
    p.lengths = lengths;
    p.out = static_cast<uint16_t*>(out);
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + (need > 0 ? splits * units * v.rows * head_dim : 0));
    p.num_pages = num_pages;
    p.max_pages = static_cast<int>(max_pages);
    p.page_size = static_cast<int>(page_size);
    p.q_len = static_cast<int>(q_len);
    p.kv_heads = divider(static_cast<uint32_t>(kv_heads));
    p.ratio = divider(static_cast<uint32_t>(ratio));
    p.row_tiles = divider(static_cast<uint32_t>(ceil_div(rows, v.rows)));
    p.blocks = divider(static_cast<uint32_t>(page_size / 16));
    p.units = static_cast<int>(units);
    p.splits = splits;
    p.sorted = longest_first(v, units * splits, max_pages * page_size / splits) ? static_cast<int>(batch) : 0;
    p.rotate = rotate;
    p.norm = static_cast<float>(1.0 / std::sqrt(static_cast<double>(head_dim)));
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    int sms = 0, dev = 0, occ = 0;
    st = device_sms(&sms, &dev);
    if (st != HADQ_OK) return st;
    st = occupancy(reinterpret_cast<const void*>(v.fn), dev, v.threads, v.smem, &occ);
    if (st != HADQ_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = launch_result(launch_pdl3(v.fn, dim3(static_cast<unsigned>(units), static_cast<unsigned>(splits)), 1, v.threads, v.smem, s, p),
                       "cache attention launch");
    if (st != HADQ_OK || splits == 1) return st;
    const int pieces = static_cast<int>(std::min<int64_t>(v.pieces, ceil_div(splits, 8)));   // 8 parts in flight a warp
    return launch_result(launch_pdl(v.join, units, 32 * v.rows * pieces, 0, s, p), "cache attention join launch");
  });
}

}  // extern "C"
