// Attention of a tree of drafted tokens (include/mk.h, mk_tree_attention): what its
// kernels share -- the parameters, the line of work and its shares.
//
// For kv-head g of sequence b the rows are (node, query head of the group):
// row r = t * G + i, i < G = n_heads / n_kv_heads. All rows of a (b, g) read the
// same keys, so a key tile is fetched once for a tile of rows. The tiles of all
// (b, g) form one line of work that is cut into equal shares, one per group
// of blocks, wherever the cuts fall; the lengths are read on the device, so the
// grid does not depend on them and a captured call stays valid. A share that
// covers a (b, g) whole writes its rows; shares that cover a part write
// (o, m, l) to the workspace and a second kernel joins them. A share also costs
// what its beginning and its end take: each (b, g) counts that many tiles more
// on the line, or a block with many short sequences would be the last to finish.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "mk_ops.h"
#include "mk_ptx.cuh"

namespace mk {

struct AttnParams {
  CacheView cache;
  const uint16_t *k, *v;
  const void* q;
  void* out;
  int64_t qs, os;
  const int32_t *starts, *parents, *counts;
  int B, T, nh, G;
  int tile_log2;               // keys of a tile
  int extra;                   // tiles that a share's beginning and end are worth
  int row_tile;                // rows of a row tile
  int row_tiles, groups;       // grid = groups x row_tiles, row tiles fastest
  uint32_t inv_groups;         // floor(2^32 / groups) + 1, at most 2^32 - 1
  float scale_log2;            // scale * log2(e)
  float* part_o;               // [groups][2][row_tiles][row_tile][D]
  float* part_ml;              // [groups][2][row_tiles][row_tile][2]: (max, sum)
};

// ---- the line of work -----------------------------------------------------------
// Sequence b has nt(b) tiles for each kv-head; items are ordered (b, g), each is
// `extra` places and then its tiles in order. A block finds its part of the line
// before it can fetch anything, so that this part has one division left (with five a
// block's start took 1000 cycles longer).

// The line in shared memory: the places of the sequences before b, and the
// sequences' starts and counts (at their bounds).
struct Line {
  int prefix[kMaxSeqs + 1];
  int start[kMaxSeqs];
  uint8_t count[kMaxSeqs];
};

// places of an item with `keys` keys
__device__ __forceinline__ int places_of(const AttnParams& p, int keys) {
  return ((keys + (1 << p.tile_log2) - 1) >> p.tile_log2) + p.extra;
}

// Fills it with one warp. (The host makes sure that the line has fewer than 2^31
// places.)
__device__ __forceinline__ void work_line(const AttnParams& p, Line& line) {
  const int lane = threadIdx.x % 32;
  int sum = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int x = 0;
    if (b < p.B) {
      const int start = clamped(p.starts, b, p.cache.capacity), count = clamped(p.counts, b, p.T);
      line.start[b] = start;
      line.count[b] = (uint8_t)count;
      const int keys = count > 0 ? min(start + count, p.cache.capacity) : 0;
      if (keys > 0) x = places_of(p, keys) * p.cache.n_kv;
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (b < p.B) line.prefix[b + 1] = sum + x;
    sum += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) line.prefix[0] = 0;
  __syncwarp();
}

// The cut of a line of W places: group s has the places [begin(s), begin(s + 1)),
// begin(s) = floor(s W / groups) = s q + floor(s r / groups).
struct Cut {
  int W, groups, q, r;
  uint32_t inv;
  __device__ __forceinline__ Cut(int W_, const AttnParams& p)
      : W(W_), groups(p.groups), inv(p.inv_groups) {
    q = (int)__umulhi((uint32_t)W, inv);  // at most one off, as W < 2^31
    r = W - q * groups;
    if (r < 0) --q, r += groups;
    if (r >= groups) ++q, r -= groups;
  }
  __device__ __forceinline__ int begin(int s) const {
    return s * q + (int)__umulhi((uint32_t)(s * r), inv);  // exact: s r groups < 2^32
  }
  // the group that has place u
  __device__ __forceinline__ int group_of(int u) const {
    int s = min(groups - 1, (int)(((float)u + 1.f) * (float)groups / (float)W));  // at most one off
    if (begin(s) > u) --s;
    else if (begin(s + 1) <= u) ++s;
    return s;
  }
};

// A share of the line that lies in one item: tiles [k0, k0 + n) of the nt tiles of
// kv-head g of sequence b.
struct Share {
  int b, g, k0, n, nt;
  bool begins;  // it begins where the group's part of the line begins
  int count, start, len, rows;
};

// The next share from place u on, which moves behind it. False at the end of the
// part [u_begin, u_end).
__device__ __forceinline__ bool next_share(const AttnParams& p, const Line& line, int u_begin,
                                           int u_end, int& u, Share& s) {
  do {
    if (u >= u_end) return false;
    int lo = 0, hi = p.B;  // the last sequence whose prefix is <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (line.prefix[mid] <= u) lo = mid;
      else hi = mid;
    }
    s.b = lo;
    const int places = (line.prefix[lo + 1] - line.prefix[lo]) / p.cache.n_kv, at = u - line.prefix[lo];
    s.nt = places - p.extra;
    // floor(at / places), which is below 4096: the rounded quotient is at most one off
    s.g = (int)__fdividef((float)at, (float)places);
    if (s.g * places > at) --s.g;
    else if ((s.g + 1) * places <= at) ++s.g;
    const int tile0 = line.prefix[lo] + s.g * places + p.extra;  // place of the item's tile 0
    s.k0 = max(u - tile0, 0);
    s.n = min(u_end - tile0, s.nt) - s.k0;
    s.begins = u == u_begin;
    u = tile0 + s.nt;
  } while (s.n <= 0);  // a part that ends before the item's first tile
  s.count = line.count[s.b];
  s.start = line.start[s.b];
  s.len = min(s.start + s.count, p.cache.capacity);
  s.rows = s.count * p.G;
  return true;
}

// the number of a row tile of a share in the workspace
__device__ __forceinline__ size_t part_slot(const AttnParams& p, int group, bool begins, int rt) {
  return ((size_t)group * 2 + (begins ? 0 : 1)) * p.row_tiles + rt;
}

// offset of a row (of kv-head g of sequence b) in q or out
__device__ __forceinline__ int64_t row_offset(const AttnParams& p, int b, int g, int row, int D,
                                              int64_t stride) {
  return ((int64_t)b * p.T + row / p.G) * stride + (g * p.G + row % p.G) * D;
}

// ---- asynchronous 16-byte copies ---------------------------------------------------
// (bytes 0: the destination is zeroed)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// P bf16 parts of a pair whose sum is the value to 2^-8P of it, each part the
// rounded rest of the ones before (an infinite part has no rest).
template <int P>
__device__ __forceinline__ void split(float a, float b, uint32_t (&part)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    part[i] = bf16x2_rn(a, b);
    if (i + 1 < P) {
      const float ha = bf_lo(part[i]), hb = bf_hi(part[i]);
      a = isinf(ha) ? 0.f : a - ha;
      b = isinf(hb) ? 0.f : b - hb;
    }
  }
}

// Allows a kernel its dynamic shared memory, once on each device (ready: a bit per
// device; doing it twice does no harm).
inline int allow_shared(std::atomic<uint64_t>& ready, const void* fn, int bytes) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return op_cuda(e, "mk_tree_attention");
  const uint64_t bit = 1ull << (device & 63);
  if (device < 64 && (ready.load(std::memory_order_acquire) & bit)) return MK_OK;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return op_cuda(e, "mk_tree_attention");
  ready.fetch_or(bit, std::memory_order_release);
  return MK_OK;
}

// Launch of the kernel for many rows (mk_tree_attention_tc.cu).
int launch_tree_attention_tc(const AttnParams& p, int head_dim, int type, cudaStream_t st);

}  // namespace mk
