// common.cuh -- host-side helpers shared by the entry points: error words, tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/blink.h"

namespace blink {

// Layout of the first 256 bytes of every workspace: the device error word, then reserved space.
struct WorkspaceHeader {
    int32_t error;      // 0 = fine, else a blink_status latched by a kernel
    int32_t reserved[63];
};
static_assert(sizeof(WorkspaceHeader) == 256, "workspace header is 256 bytes");

constexpr size_t kHeaderBytes = sizeof(WorkspaceHeader);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Encodes a rank-3 tiled tensor map over a bf16 tensor with dims {d0 (contiguous), d1, d2},
// byte strides {stride1, stride2}, box {b0, b1, b2}, 128-byte swizzle, zero fill out of bounds.
// Returns false if the driver entry point is missing or the driver rejects the map.
bool encode_tmap_3d_bf16(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2,
                         uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t b0, uint32_t b1, uint32_t b2);

// The same over bytes, with `swizzle` (128 or 64) bytes of swizzle.
bool encode_tmap_3d_bytes(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1_bytes,
                          uint64_t stride2_bytes, uint32_t b0, uint32_t b1, uint32_t b2, int swizzle);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether rows of `width` bytes, `na` of them `sa` bytes apart from `a`, share a byte with those of `b`.  Rows of
// one stride may interleave (slices of one wider row); with other strides touching extents count as shared.
bool strided_overlap(const void *a, int64_t sa, int64_t na, const void *b, int64_t sb, int64_t nb, int64_t width_a,
                     int64_t width_b);

// Launches `kern` with programmatic stream serialization: it may be scheduled while the kernel before it in the stream drains
// (where that one allows it) and has to wait (griddepcontrol.wait) before it touches memory.
template <class Kernel, class... Args>
cudaError_t launch_programmatic(Kernel kern, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

int current_sm_count();  // of the current device; 0 if it cannot be asked

}  // namespace blink
