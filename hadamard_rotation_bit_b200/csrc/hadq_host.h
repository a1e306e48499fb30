// Host helpers shared by the translation units of the C ABI: error reporting,
// pointer checks, per-device launch caches and launches.
#pragma once

#include "hadq.h"

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <string>

namespace hadq {
namespace host {

// Records the calling thread's error line (hadq_last_error) and returns st.
hadq_status fail(hadq_status st, const std::string& msg);
void clear_error();

inline int64_t esize(hadq_dtype d) { return d == HADQ_F32 ? 4 : 2; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  uintptr_t lo = 0, hi = 0;
};

inline Span span(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + static_cast<uintptr_t>(bytes)};
}

inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// SM count of the current device (cached) and its number.
hadq_status device_sms(int* sms, int* dev_out);

// Resident CTAs per SM for `fn` at this block/smem size.  Also raises the
// dynamic shared memory limit of `fn` on this device when it needs more than
// 48 KB; the limit only ever grows (a kernel whose shared memory depends on
// the call must keep the largest size any earlier call of it needed).
hadq_status occupancy(const void* fn, int dev, int block, int smem, int* occ);

hadq_status check_launch(const char* what);
hadq_status launch_result(cudaError_t e, const char* what);

// The driver's tensor-map encoder; nullptr when it is not available.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Launch with programmatic stream serialization: the kernel may be scheduled
// while the previous kernel in the stream drains; it waits for that kernel's
// completion (griddepcontrol.wait) before touching global memory.  cluster:
// CTAs of a cluster along x (1: none).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl3(void (*fn)(KArgs...), dim3 grid, int cluster, int block, int smem, cudaStream_t stream,
                        Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*fn)(KArgs...), int64_t grid, int block, int smem, cudaStream_t stream, Args... args) {
  return launch_pdl3(fn, dim3(static_cast<unsigned>(grid)), 1, block, smem, stream, args...);
}

}  // namespace host
}  // namespace hadq
