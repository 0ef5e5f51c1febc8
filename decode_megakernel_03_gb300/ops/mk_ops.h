// Host-side declarations shared by the operators over a KV cache: the checks of
// mk_cache, the error slot of calls without a handle, and the cache as the
// kernels see it.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

#include "mk.h"

namespace mk {

constexpr int kMaxSeqs = 1024;        // sequences per call
constexpr int kMaxOpLayers = 64;      // layers per call (their pointers travel in the parameters)
constexpr uint32_t kNoRow = 0xffffffffu;

// Records the message for mk_last_error(NULL) and returns code. Never throws.
int op_fail(int code, const char* msg) noexcept;
// the same for a CUDA error code (a cudaError_t); 0 gives MK_OK
int op_cuda(int cuda_error, const char* what) noexcept;

// One layer of a cache, by value in the kernel parameters. Rows are numbered
// (block * n_kv_heads + head) * block_size + row; check_cache makes sure that
// the number fits 32 bits below kNoRow.
struct CacheView {
  const int32_t* table;  // nullptr: contiguous
  int entries, n_blocks, block_size, n_kv, capacity;
};

// Checks a cache for a call over `batch` sequences (need_table: false for the
// calls that address blocks directly) and fills the view. MK_OK or the code.
int check_cache(const mk_cache* c, int batch, bool need_table, CacheView* out) noexcept;

inline bool aligned(const void* p, size_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

#if defined(__CUDACC__)
// Row number of slot `slot` of sequence b at kv-head 0 (kNoRow: the page is not
// there); head h's row is h * block_size behind it. slot is in [0, capacity).
__device__ __forceinline__ uint32_t cache_row(const CacheView& c, int b, int slot) {
  if (c.table == nullptr) return (uint32_t)b * c.n_kv * c.block_size + slot;
  const int e = slot / c.block_size;
  const int blk = __ldg(c.table + (size_t)b * c.entries + e);
  if ((unsigned)blk >= (unsigned)c.n_blocks) return kNoRow;
  return (uint32_t)blk * c.n_kv * c.block_size + (slot - e * c.block_size);
}

// starts[b] and counts[b] at their nearest bounds
__device__ __forceinline__ int clamped(const int32_t* p, int b, int hi) {
  return p == nullptr ? hi : min(max(__ldg(p + b), 0), hi);
}

// The launch that depends on this one may be scheduled; its griddep_wait still
// waits until this grid has completed and its writes are visible.
__device__ __forceinline__ void griddep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void griddep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

}  // namespace mk
