// Host helpers shared by the entry points (gge_api.cu defines them).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/gge.h"

namespace gge {

constexpr int kMaxSmemOptin = 232448;  // 227 KiB per block on sm_100 / sm_103
constexpr int kCtrlBytesHost = 1024;
constexpr int kEpiWarpsHost = 8;  // epilogue warps of the TMA variants (4 with gathers)
constexpr size_t kWorkspaceBytes = 256;
// the split last wave's tickets (one int32 per tail tile, CTA, epilogue warp and chunk)
// follow the status words in a region of their own: no other call writes there,
// so a ticket is never mistaken for another call's data
constexpr size_t kTicketBytes = 16384;
constexpr size_t kTailBase = kWorkspaceBytes + kTicketBytes;
constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 1;

int sm_count();  // of the current device, or -1
int elem_bytes(int32_t dt);
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
gge_status check_view(const gge_tensor& t);
// an output / C view: [M, N, L] N-major with 16-byte aligned rows and batches
gge_status check_mn(const gge_tensor* t, int64_t M, int64_t N, int64_t L);
gge_status check_workspace(void* ws, size_t bytes);
// a tensor map of `es`-byte elements, box b0 x b1 x b2, with or without the
// 128-byte swizzle; encoded maps are cached
gge_status encode_3d(CUtensorMap* m, void* ptr, int es, uint64_t d0, uint64_t d1, uint64_t d2,
                     uint64_t s1_bytes, uint64_t s2_bytes, uint32_t b0, uint32_t b1,
                     uint32_t b2 = 1, bool swizzle = true);

}  // namespace gge
