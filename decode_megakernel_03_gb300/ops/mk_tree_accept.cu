// Greedy acceptance of a drafted tree (include/mk.h, mk_tree_accept): each
// node's largest logit, then the walk from node 0 to the last accepted node.
#include <cuda_runtime.h>

#include <algorithm>

#include "mk_ops.h"
#include "mk_ptx.cuh"

namespace mk {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

// Comparable key of (value, index): the larger value wins, the lower index
// among equal ones. NaN is below everything, -0 equals +0.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t index) {
  uint32_t u = __float_as_uint(v + 0.f);
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  if (v != v) u = 0;
  return (uint64_t)u << 32 | (0xffffffffu - index);
}

struct ArgmaxParams {
  const void* logits;
  int64_t stride;
  const int32_t* counts;
  int T, V, splits, span;  // span: values of a split
  uint64_t* keys;          // [rows][splits]
};

// Block (split, row) finds the largest of `span` values of a row. Each thread
// keeps its largest so far and where it was: it meets its values in ascending
// order, so a strictly larger one replaces it. One pass, bound by the bytes of
// the logits (512 rows of 128256 fp32 values, 263 MB, in 42.2 us: 6.2 TB/s; in bf16
// 25.3 us, 5.2 TB/s, where the comparisons weigh twice as much); kUnroll 16-byte
// loads per thread are in flight (8: no faster).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) argmax_kernel(const __grid_constant__ ArgmaxParams p) {
  griddep_launch();
  const int row = blockIdx.y, b = row / p.T;
  if (row - b * p.T >= clamped(p.counts, b, p.T)) return;
  const T* x = (const T*)p.logits + (int64_t)row * p.stride;
  const int lo = blockIdx.x * p.span, hi = min(p.V, lo + p.span);
  float best = -INFINITY;
  int at = -1;  // none above -inf yet
  int first_low = -1;  // the first value that is -inf (not NaN)
  auto see = [&](float v, int i) {
    if (v > best) best = v, at = i;
  };
  if constexpr (VEC) {
    constexpr int E = 16 / sizeof(T);
    // lo is a multiple of E; the row's last values may fill a vector partly
    const int whole = hi / E * E;
    for (int i0 = lo + threadIdx.x * E; i0 < whole; i0 += kThreads * E * kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kThreads * E;
        if (i < whole) w[u] = __ldcs(reinterpret_cast<const uint4*>(x + i));
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * kThreads * E;
        if (i < whole) {
          const uint32_t a[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
              see(__uint_as_float(a[j]), i + j);
            } else {
              see(bf_lo(a[j]), i + 2 * j);
              see(bf_hi(a[j]), i + 2 * j + 1);
            }
          }
        }
      }
    }
    for (int i = max(whole, lo) + threadIdx.x; i < hi; i += kThreads) {
      if constexpr (sizeof(T) == 4) see(__ldcs(reinterpret_cast<const float*>(x) + i), i);
      else see(bf16f(__ldcs(reinterpret_cast<const uint16_t*>(x) + i)), i);
    }
  } else {
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
      if constexpr (sizeof(T) == 4) see(__ldcs(reinterpret_cast<const float*>(x) + i), i);
      else see(bf16f(__ldcs(reinterpret_cast<const uint16_t*>(x) + i)), i);
    }
  }
  // Nothing above -inf in this thread: a second look for the first -inf, so that
  // NaN stays below it (rows of this kind are rare and short of sense).
  if (at < 0 && lo < hi) {
    for (int i = lo + threadIdx.x; i < hi && first_low < 0; i += kThreads) {
      float v;
      if constexpr (sizeof(T) == 4) v = reinterpret_cast<const float*>(x)[i];
      else v = bf16f(reinterpret_cast<const uint16_t*>(x)[i]);
      if (v == -INFINITY) first_low = i;
    }
  }
  uint64_t key = at >= 0 ? key_of(best, at)
                 : first_low >= 0 ? key_of(-INFINITY, first_low)
                 : lo + (int)threadIdx.x < hi ? key_of(NAN, lo + threadIdx.x) : 0;
#pragma unroll
  for (int d = 16; d; d /= 2) key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
  __shared__ uint64_t s_key[kThreads / 32];
  if (threadIdx.x % 32 == 0) s_key[threadIdx.x / 32] = key;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) key = max(key, s_key[w]);
    p.keys[(int64_t)row * p.splits + blockIdx.x] = key;
  }
}

struct WalkParams {
  const uint64_t* keys;
  const int32_t *tokens, *parents, *counts;
  int32_t *choices, *path, *accepted, *next;
  int T, splits;
};

// One block per sequence: the splits' keys joined, one of 32 warps per node at a
// time, then one warp walks. A chain (no parents) may have any length: its nodes are
// taken 32 at a time. In a tree, lane l holds nodes l and l + 32; the children
// whose token fits are found by a ballot, the lowest one first.
constexpr int kWalkThreads = 1024;

__global__ void __launch_bounds__(kWalkThreads) walk_kernel(const __grid_constant__ WalkParams p) {
  __shared__ int s_choice[MK_MAX_TREE];
  const int b = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n = clamped(p.counts, b, p.T);
  const int64_t base = (int64_t)b * p.T;
  // of a tree, lane l of the walking warp holds nodes l and l + 32
  const bool tree = p.parents != nullptr, has0 = lane < n, has1 = lane + 32 < n;
  int par0 = -1, par1 = -1, tok0 = 0, tok1 = 0;
  if (warp == 0 && tree) {
    if (has0) par0 = __ldg(p.parents + base + lane), tok0 = __ldg(p.tokens + base + lane);
    if (has1) par1 = __ldg(p.parents + base + lane + 32), tok1 = __ldg(p.tokens + base + lane + 32);
  }
  griddep_wait();
  for (int t = warp; t < p.T; t += kWalkThreads / 32) {
    uint64_t key = 0;
    if (t < n)
      for (int s = lane; s < p.splits; s += 32)
        key = max(key, p.keys[(base + t) * p.splits + s]);
#pragma unroll
    for (int d = 16; d; d /= 2) key = max(key, __shfl_xor_sync(0xffffffffu, key, d));
    if (lane == 0) {
      const int c = t < n ? (int)(0xffffffffu - (uint32_t)key) : -1;
      p.choices[base + t] = c;
      if (tree) s_choice[t] = c;  // a tree has at most MK_MAX_TREE nodes
      p.path[base + t] = -1;
    }
  }
  __syncthreads();  // the block's choices and path entries are visible to it
  if (warp != 0) return;
  const int32_t *tok = p.tokens + base, *choice = p.choices + base;
  int taken = 0, cur = -1;
  if (n > 0) {
    cur = 0;
    taken = 1;
    if (tree) {
      if (lane == 0) p.path[base] = 0;
      for (;;) {
        const int want = s_choice[cur];
        const unsigned f0 = __ballot_sync(0xffffffffu, has0 && lane > cur && par0 == cur && tok0 == want);
        const unsigned f1 = __ballot_sync(0xffffffffu, has1 && lane + 32 > cur && par1 == cur && tok1 == want);
        if (!(f0 | f1)) break;
        cur = f0 ? __ffs(f0) - 1 : 31 + __ffs(f1);
        if (lane == 0) p.path[base + taken] = cur;
        ++taken;
      }
    } else {
      // node t + 1 is accepted while its token is node t's choice
      for (;;) {
        const int t = cur + 1 + lane;
        const bool fits = t < n && tok[t] == choice[t - 1];
        const unsigned f = __ballot_sync(0xffffffffu, fits);
        const int more = f == 0xffffffffu ? 32 : __ffs(~f) - 1;
        cur += more;
        if (more < 32) break;
      }
      taken = cur + 1;
      for (int t = lane; t < taken; t += 32) p.path[base + t] = t;
    }
  }
  if (lane == 0) {
    p.accepted[b] = taken;
    p.next[b] = n > 0 ? choice[cur] : -1;
  }
}

// Splits of a row: as many as make 8 blocks per SM of a 152-SM machine, what is
// resident at once (512 rows of 128256 values, fp32 / bf16: 42.2 / 25.3 us; 4 per
// SM 43.7 / 26.7, 16 43.4 / 26.0, 32 43.7 / 27.8), none shorter than 4096 values
// (16 rows, fp32 / bf16: 5.2 / 5.2 us; with 2048 values 6.2 / 7.2).
int splits_of(int rows, int V) {
  const int want = std::max(1, 8 * 152 / std::max(1, rows));
  return std::min(want, std::max(1, V / 4096));
}

int check_accept(int batch, int n_tokens, int vocab) {
  if (batch < 1 || batch > kMaxSeqs || n_tokens < 1 || (int64_t)batch * n_tokens > 65535)
    return op_fail(MK_ERR_INVALID,
                   "batch must be 1 to 1024, n_tokens at least 1, their product at most 65535");
  if (vocab < 1 || vocab > (1 << 30))
    return op_fail(MK_ERR_INVALID, "vocab must be 1 to 2^30");
  return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

int mk_tree_accept_workspace(int batch, int n_tokens, int vocab, size_t* bytes) {
  if (!bytes) return op_fail(MK_ERR_INVALID, "bytes is NULL");
  if (int rc = check_accept(batch, n_tokens, vocab)) return rc;
  const size_t rows = (size_t)batch * n_tokens;
  *bytes = rows * splits_of((int)rows, vocab) * sizeof(uint64_t);
  return MK_OK;
}

int mk_tree_accept(int batch, int n_tokens, int vocab, int type, const void* logits,
                   int64_t logits_stride, const int32_t* tokens, const int32_t* parents,
                   const int32_t* counts, int32_t* choices, int32_t* path, int32_t* accepted,
                   int32_t* next, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  if (int rc = mk_tree_accept_workspace(batch, n_tokens, vocab, &need)) return rc;
  if (!logits || !tokens || !choices || !path || !accepted || !next || !workspace)
    return op_fail(MK_ERR_INVALID, "mk_tree_accept: a NULL argument");
  if (type != MK_TYPE_BF16 && type != MK_TYPE_FP32)
    return op_fail(MK_ERR_INVALID, "type must be MK_TYPE_BF16 or MK_TYPE_FP32");
  if (parents && n_tokens > MK_MAX_TREE)
    return op_fail(MK_ERR_INVALID, "a tree has at most MK_MAX_TREE nodes");
  const size_t size = type == MK_TYPE_FP32 ? 4 : 2;
  if (logits_stride < vocab || !aligned(logits, size))
    return op_fail(MK_ERR_INVALID, "logits: aligned to its type, a stride of at least vocab");
  if (!aligned(workspace, 256) || workspace_bytes < need)
    return op_fail(MK_ERR_INVALID, "workspace: 256-byte aligned and as large as its query says");
  const int rows = batch * n_tokens;
  ArgmaxParams a;
  a.logits = logits;
  a.stride = logits_stride;
  a.counts = counts;
  a.T = n_tokens;
  a.V = vocab;
  a.splits = splits_of(rows, vocab);
  a.span = (int)(((int64_t)vocab + a.splits - 1) / a.splits);
  a.span = (a.span + 7) / 8 * 8;  // whole 16-byte vectors
  a.keys = (uint64_t*)workspace;
  const bool vec = aligned(logits, 16) && logits_stride * size % 16 == 0;
  const dim3 grid(a.splits, rows);
  cudaStream_t st = (cudaStream_t)stream;
  if (type == MK_TYPE_FP32) {
    if (vec) argmax_kernel<float, true><<<grid, kThreads, 0, st>>>(a);
    else argmax_kernel<float, false><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (vec) argmax_kernel<uint16_t, true><<<grid, kThreads, 0, st>>>(a);
    else argmax_kernel<uint16_t, false><<<grid, kThreads, 0, st>>>(a);
  }
  if (int rc = op_cuda(cudaGetLastError(), "mk_tree_accept")) return rc;
  const WalkParams w{a.keys, tokens, parents, counts, choices, path, accepted, next,
                     n_tokens, a.splits};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(batch);
  cfg.blockDim = dim3(kWalkThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return op_cuda(cudaLaunchKernelEx(&cfg, walk_kernel, w), "mk_tree_accept");
}

}  // extern "C"
