// Verification of drafted nodes by rejection sampling (include/mk.h,
// mk_tree_verify).
//
// At a node with the target's probabilities p and the drafter's q, the rejection of j
// children leaves the distribution r_j = norm(max(r_{j-1} - q, 0)), r_0 = p. With
// c_0 = 0, N_0 = 1 and c_{j+1} = c_j + N_j, N_j = sum max(p - c_j q, 0), that is
// r_j = max(p - c_j q, 0) / N_j: subtracting q from max(p - c q, 0) / N is subtracting
// (c + N) q from p, as what was cut off before is cut off again. So a node needs its
// row's maximum and sum, one more sum for each rejection, and nothing is written to
// memory between.
#include <cuda_runtime.h>

#include "mk_ops.h"
#include "mk_ptx.cuh"

namespace mk {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

struct VerifyParams {
  const void *logits, *draft;
  int64_t logits_stride, draft_stride, noise_stride;
  const float *temperature, *uniform, *noise;
  const int32_t *tokens, *parents, *counts;
  int32_t *path, *accepted, *next;
  int T, V;
};

template <typename T>
__device__ __forceinline__ float value(const T* p) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float*>(p);
  else return bf16f(*reinterpret_cast<const uint16_t*>(p));
}

// A row's softmax at a temperature: weights relative to the largest logit. A NaN or
// -inf has none; the largest has 1, also where it is infinite or the temperature tiny.
struct Softmax {
  float top, k, inv;  // largest logit; log2(e) / temperature; 1 / sum
  int only;           // temperature not above 0: the one index that has a weight (else -1)
  __device__ __forceinline__ float weight(float l, int i) const {
    if (only >= 0) return i == only ? 1.f : 0.f;
    return l == top ? 1.f : l > -INFINITY ? fast_exp2((l - top) * k) : 0.f;
  }
};

template <typename Op>
__device__ __forceinline__ float block_reduce(float x, float* s, Op op) {
#pragma unroll
  for (int d = 16; d; d /= 2) x = op(x, __shfl_xor_sync(0xffffffffu, x, d));
  __syncthreads();  // s is free
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = x;
  __syncthreads();
  x = s[threadIdx.x % 32];
#pragma unroll
  for (int d = 16; d; d /= 2) x = op(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Sum {
  __device__ float operator()(float a, float b) const { return a + b; }
};
__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t* s) {
#pragma unroll
  for (int d = 16; d; d /= 2) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
  __syncthreads();
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = x;
  __syncthreads();
  x = s[threadIdx.x % 32];
#pragma unroll
  for (int d = 16; d; d /= 2) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}

// One block per sequence walks its tree; every thread keeps the walk's state.
template <typename L, typename Q>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ float s_f[32];
  __shared__ uint64_t s_k[32];
  __shared__ int s_gone[MK_MAX_TREE];  // tokens taken out (drafts without probabilities)
  const int b = blockIdx.x, tid = threadIdx.x;
  const int n = clamped(p.counts, b, p.T);
  const int64_t base = (int64_t)b * p.T;
  for (int t = tid; t < p.T; t += kThreads) p.path[base + t] = t == 0 && n > 0 ? 0 : -1;
  if (n == 0) {
    if (tid == 0) p.accepted[b] = 0, p.next[b] = -1;
    return;
  }
  const float heat = p.temperature ? p.temperature[b] : 1.f;
  const bool has_draft = p.draft != nullptr;
  const float* noise = p.noise + (int64_t)b * p.noise_stride;

  auto row_of = [&](int t) { return (const L*)p.logits + (base + t) * p.logits_stride; };
  auto draft_of = [&](int t) { return (const Q*)p.draft + (base + t) * p.draft_stride; };
  auto share = [&](const Q* q, int i) {  // a drafter's probability; NaN and negative ones are 0
    const float x = value(q + i);
    return x > 0.f ? x : 0.f;
  };
  // false: no value above -inf
  auto softmax_of = [&](const L* x, Softmax& f) {
    float top = -INFINITY;
    for (int i = tid; i < p.V; i += kThreads) top = fmaxf(top, value(x + i));
    f.top = block_reduce(top, s_f, Max());
    f.only = -1;
    f.inv = 1.f;
    if (f.top == -INFINITY) return false;
    if (!(heat > 0.f)) {
      uint64_t key = 0;
      for (int i = tid; i < p.V; i += kThreads)
        if (value(x + i) == f.top) key = max(key, (uint64_t)(p.V - i));
      f.only = p.V - (int)block_max(key, s_k);
      return true;
    }
    f.k = 1.4426950408889634f / heat;
    float sum = 0.f;
    for (int i = tid; i < p.V; i += kThreads) sum += f.weight(value(x + i), i);
    f.inv = 1.f / block_reduce(sum, s_f, Sum());
    return true;
  };

  int cur = 0, taken = 1, gone = 0;
  float c = 0.f, mass = 1.f;  // c_j, N_j
  Softmax f;
  bool some = softmax_of(row_of(0), f);
  // a node's children come behind it, in ascending order: one look at each node
  for (int t = 1; some && t < n; ++t) {
    int up = t - 1;
    if (p.parents) up = p.parents[base + t];
    if (up != cur) {
      if (!p.parents) break;  // a chain ends with its first rejected node
      continue;
    }
    const int x = p.tokens[base + t];
    if ((unsigned)x >= (unsigned)p.V) continue;
    const float px = f.weight(value(row_of(cur) + x), x) * f.inv;
    float u = p.uniform[base + t], left = px, chance = 1.f;
    u = u > 0.f ? fminf(u, 1.f) : 0.f;
    if (has_draft) {
      chance = share(draft_of(cur), x);
      left = fmaxf(px - c * chance, 0.f);
    } else {
      for (int i = 0; i < gone; ++i)
        if (s_gone[i] == x) left = 0.f;
    }
    if (u * chance * mass < left) {
      cur = t;
      if (tid == 0) p.path[base + taken] = t;
      ++taken;
      c = 0.f, mass = 1.f, gone = 0;
      some = softmax_of(row_of(t), f);
    } else if (has_draft) {
      c += mass;
      const L* row = row_of(cur);
      const Q* q = draft_of(cur);
      float sum = 0.f;
      for (int i = tid; i < p.V; i += kThreads)
        sum += fmaxf(f.weight(value(row + i), i) * f.inv - c * share(q, i), 0.f);
      mass = block_reduce(sum, s_f, Sum());
    } else if (left > 0.f) {
      __syncthreads();  // everybody has looked at the list
      if (tid == 0) s_gone[gone] = x;
      __syncthreads();
      ++gone;
      mass = fmaxf(mass - left, 0.f);
    }
  }
  // ---- the race over what is left
  int next = -1;
  if (some) {
    const L* row = row_of(cur);
    const Q* q = draft_of(cur);
    uint64_t best = 0;
    for (int again = 0; again < 2 && best == 0; ++again) {  // nothing left (by rounding): over p itself
      for (int i = tid; i < p.V; i += kThreads) {
        float r = f.weight(value(row + i), i) * f.inv;
        if (!again) {
          if (has_draft && c > 0.f) r -= c * share(q, i);
          for (int j = 0; j < gone; ++j)
            if (s_gone[j] == i) r = 0.f;
        }
        if (!(r > 0.f)) continue;
        const float e = noise[i];
        const float score = __fdividef(r, e > 1e-30f ? fminf(e, 1e30f) : 1e-30f);
        best = max(best, (uint64_t)__float_as_uint(score) << 32 | (0xffffffffu - (uint32_t)i));
      }
      best = block_max(best, s_k);
    }
    if (best) next = (int)(0xffffffffu - (uint32_t)best);
  }
  if (tid == 0) {
    p.accepted[b] = taken;
    p.next[b] = next;
  }
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_tree_verify(int batch, int n_tokens, int vocab, int type, const void* logits,
                              int64_t logits_stride, int draft_type, const void* draft,
                              int64_t draft_stride, const float* temperature,
                              const int32_t* tokens, const int32_t* parents, const int32_t* counts,
                              const float* uniform, const float* noise, int64_t noise_stride,
                              int32_t* path, int32_t* accepted, int32_t* next, void* stream) {
  if (batch < 1 || batch > kMaxSeqs || n_tokens < 1 || (int64_t)batch * n_tokens > 65535)
    return op_fail(MK_ERR_INVALID,
                   "batch must be 1 to 1024, n_tokens at least 1, their product at most 65535");
  if (vocab < 1 || vocab > (1 << 30))
    return op_fail(MK_ERR_INVALID, "vocab must be 1 to 2^30");
  if (!logits || !tokens || !uniform || !noise || !path || !accepted || !next)
    return op_fail(MK_ERR_INVALID, "mk_tree_verify: a NULL argument");
  if ((type != MK_TYPE_BF16 && type != MK_TYPE_FP32) ||
      (draft && draft_type != MK_TYPE_BF16 && draft_type != MK_TYPE_FP32))
    return op_fail(MK_ERR_INVALID, "type, draft_type must be MK_TYPE_BF16 or MK_TYPE_FP32");
  if (parents && n_tokens > MK_MAX_TREE)
    return op_fail(MK_ERR_INVALID, "a tree has at most MK_MAX_TREE nodes");
  const size_t size = type == MK_TYPE_FP32 ? 4 : 2, draft_size = draft_type == MK_TYPE_FP32 ? 4 : 2;
  if (logits_stride < vocab || !aligned(logits, size))
    return op_fail(MK_ERR_INVALID, "logits: aligned to its type, a stride of at least vocab");
  if (draft && (draft_stride < vocab || !aligned(draft, draft_size)))
    return op_fail(MK_ERR_INVALID, "draft: aligned to its type, a stride of at least vocab");
  if (noise_stride < vocab || !aligned(noise, 4) || !aligned(uniform, 4) ||
      !aligned(temperature, 4))
    return op_fail(MK_ERR_INVALID,
                   "noise: a stride of at least vocab; noise, uniform, temperature: aligned to 4 bytes");
  VerifyParams p{logits, draft, logits_stride, draft_stride, noise_stride, temperature, uniform,
                 noise, tokens, parents, counts, path, accepted, next, n_tokens, vocab};
  cudaStream_t st = (cudaStream_t)stream;
  const bool narrow = draft && draft_type == MK_TYPE_BF16;
  if (type == MK_TYPE_FP32) {
    if (narrow) verify_kernel<float, uint16_t><<<batch, kThreads, 0, st>>>(p);
    else verify_kernel<float, float><<<batch, kThreads, 0, st>>>(p);
  } else {
    if (narrow) verify_kernel<uint16_t, uint16_t><<<batch, kThreads, 0, st>>>(p);
    else verify_kernel<uint16_t, float><<<batch, kThreads, 0, st>>>(p);
  }
  return op_cuda(cudaGetLastError(), "mk_tree_verify");
}
