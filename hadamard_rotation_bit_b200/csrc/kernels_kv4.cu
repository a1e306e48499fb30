// Instantiations of the int4 cache kernels and their lookup; this unit also
// owns their fault word (hadq_kv4_fault).
#include "hadq_launch.h"
#include "hadq_kv4.cuh"

namespace hadq {
namespace launch {
namespace {

template <int D, int GROUP, int NT>
AttnVariant attn() {
  using C = kv4::Cfg<D, GROUP, NT, 3>;
  return AttnVariant{&kv4::kv4_attention_kernel<D, GROUP, NT, 3>, &kv4::kv4_join_kernel<D, C::ROWS>, 32 * kv4::kWarps,
                     C::SMEM_BYTES, C::ROWS, NT == 1 ? 4 : 2, kv4::kPieces<C::ROWS>};
}

template <int D, int GROUP>
AttnVariant attn_rows(int rows) {
  return rows <= 8 ? attn<D, GROUP, 1>() : attn<D, GROUP, 2>();
}

}  // namespace

AttnVariant kv4_attention_for(int d, int group, int rows) {
  if (d == 128) {
    if (group == 128) return attn_rows<128, 128>(rows);
    if (group == 64) return attn_rows<128, 64>(rows);
    if (group == 32) return attn_rows<128, 32>(rows);
  } else if (d == 64) {
    if (group == 64) return attn_rows<64, 64>(rows);
    if (group == 32) return attn_rows<64, 32>(rows);
  }
  return AttnVariant{nullptr, nullptr, 0, 0, 0, 0, 0};
}

AppendFn kv4_append_for(bool bf16, int d) {
  if (d == 128) return bf16 ? &kv4::kv4_append_kernel<true, 128> : &kv4::kv4_append_kernel<false, 128>;
  return bf16 ? &kv4::kv4_append_kernel<true, 64> : &kv4::kv4_append_kernel<false, 64>;
}

int kv4_fault_bits(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, kv4::hadq_kv4_fault, sizeof(v)) != cudaSuccess) return -1;
  if (clear && v != 0) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(kv4::hadq_kv4_fault, &z, sizeof(z)) != cudaSuccess) return -1;
  }
  return static_cast<int>(v);
}

}  // namespace launch
}  // namespace hadq
