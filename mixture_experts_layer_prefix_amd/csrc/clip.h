// Gradient norm and clipping: tables of tensors and launchers (see clip.hip).
#pragma once
#include "common.h"

namespace moe {

constexpr int kChunk = 16384;               // elements a workgroup takes at a time
constexpr int kClipGroups = 1024;           // workgroups at most, four per compute unit
constexpr int64_t kEntryMax = 1ll << 30;    // elements of one table entry at most (a multiple of kChunk)
constexpr uint32_t kF32Entry = 0x80000000u; // flag in numel: fp32 elements (bf16 otherwise)

// Kernel arguments may take 4 KiB.
struct NormTable {
  static constexpr int kEntries = 240;
  const void* src[kEntries];
  uint32_t numel[kEntries];
  uint32_t first[kEntries + 1];  // chunk number each entry starts at; first[n]: all chunks
  int n;
};
struct ClipTable {
  static constexpr int kEntries = 160;
  const void* src[kEntries];
  void* dst[kEntries];
  uint32_t numel[kEntries];
  uint32_t first[kEntries + 1];
  int n;
};
static_assert(sizeof(NormTable) + 16 <= 4096 && sizeof(ClipTable) + 48 <= 4096, "tables exceed the kernel arguments");

size_t grad_norm_scratch_bytes(int n, const int64_t* numel);
hipError_t launch_grad_norm(int n, const void* const* grads, const int64_t* numel, const int32_t* types, float* norm,
                            void* scratch, hipStream_t s);
// norm_in null: the norm of these tensors, left in *norm.
hipError_t launch_clip_grads(int n, const void* const* grads, void* const* out, const int64_t* numel,
                             const int32_t* types, float max_norm, const float* norm_in, float* norm, void* scratch,
                             hipStream_t s);

}  // namespace moe
