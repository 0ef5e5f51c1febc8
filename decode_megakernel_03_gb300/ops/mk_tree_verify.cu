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

#include <atomic>
#include <climits>

#include "mk_ops.h"
#include "mk_ptx.cuh"

namespace mk {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;  // that take values; one more warp decides
constexpr int kMaxCluster = 16;
constexpr int E = 8;  // a thread takes values by eight
constexpr float kSlack = 8.f;  // log2 of how far a weight may exceed 1 while a thread adds up

struct VerifyParams {
  const void *logits, *draft;
  int64_t logits_stride, draft_stride, noise_stride;
  const float *temperature, *uniform, *noise;
  const int32_t *tokens, *parents, *counts;
  int32_t *path, *accepted, *next;
  int T, V, span;  // span: values of a block's part of a row
};

// ---- the cluster -------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// to the same place of block `rank`'s shared memory
__device__ __forceinline__ uint32_t remote(const void* at, uint32_t rank) {
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(at)), "r"(rank));
  return to;
}
__device__ __forceinline__ void put_remote(const void* at, uint32_t rank, uint2 v) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(remote(at, rank)), "r"(v.x), "r"(v.y)
               : "memory");
}
__device__ __forceinline__ void put_remote(const void* at, uint32_t rank, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(remote(at, rank)), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// n bytes from `at` on will be read; whole 16-byte units
__device__ __forceinline__ void prefetch(const void* at, uint32_t n) {
  if (n) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(n) : "memory");
}

// A drafted child of the node that the walk is at: the target's logit and the drafter's
// probability of its token, its random number.
struct Child {
  float l, q, u;
  int token, node;
};

// What the blocks of a cluster hand to one another, each kind twice: one is written
// while a block may still read the one before.
struct Shared {
  uint2 part[2][kMaxCluster * kWarps];  // each warp's share of a sum
  uint4 child[2][MK_MAX_TREE];          // from block 0: l, q, u, token
  uint2 child_node[2][MK_MAX_TREE];     // its node
  uint2 head[2];                        // from block 0: the number of children (-1: no node at
                                        // all), the temperature
  Child kid[MK_MAX_TREE];               // of block 0's deciding warp
  int gone[MK_MAX_TREE];                // tokens taken out (drafts without probabilities)
};

// ---- values --------------------------------------------------------------------------

// eight values of a row
template <typename T>
struct Eight {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return e & 1 ? bf_hi(w[e / 2]) : bf_lo(w[e / 2]);
  }
};
// values i to i + 7 (those from `end` on: `fill`)
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int i, int end, float fill, Eight<T>& v) {
  if (VEC && i + E <= end) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + i) + h);
      v.w[4 * h] = a.x, v.w[4 * h + 1] = a.y, v.w[4 * h + 2] = a.z, v.w[4 * h + 3] = a.w;
    }
    return;
  }
  const uint32_t f = __float_as_uint(fill);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const bool there = i + e < end;
    if constexpr (sizeof(T) == 4) {
      v.w[e] = there ? __ldg(reinterpret_cast<const uint32_t*>(row) + i + e) : f;
    } else {
      const uint32_t x = there ? __ldg(reinterpret_cast<const uint16_t*>(row) + i + e) : f >> 16;
      v.w[e / 2] = e & 1 ? v.w[e / 2] | x << 16 : x;
    }
  }
}
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const float*>(p));
  else return bf16f(__ldg(reinterpret_cast<const uint16_t*>(p)));
}
// a drafter's probability: NaN and negative ones are 0
__device__ __forceinline__ float probability(float q) { return fmaxf(q, 0.f); }

// A row's softmax at a temperature: weights relative to the largest logit. A NaN or
// -inf has none; the largest has 1, also where it is infinite or the temperature tiny.
struct Softmax {
  float top, k, inv;  // largest logit; log2(e) / temperature; 1 / sum
  int only;           // temperature not above 0: the one index that has a weight (else -1)
  bool plain;         // top and k are finite, no `only`: weight is `quick`
  __device__ __forceinline__ void set_plain() { plain = only < 0 && fabsf(top) < INFINITY && k < INFINITY; }
  __device__ __forceinline__ float weight(float l, int i) const {
    if (only >= 0) return i == only ? 1.f : 0.f;
    return l == top ? 1.f : l > -INFINITY ? fast_exp2((l - top) * k) : 0.f;
  }
  // of two values, neither of them NaN
  __device__ __forceinline__ float2 quick(float a, float b) const {
    const unsigned long long z = mul2(sum2(pack2(a, b), pack2(-top, -top)), pack2(k, k));
    float2 w = unpack2(z);
    w.x = fast_exp2(w.x);
    w.y = fast_exp2(w.y);
    return w;
  }
  // of eight; the sum of them
  template <typename L>
  __device__ __forceinline__ float weights(const Eight<L>& v, int i, float (&w)[E]) const {
    if (plain) {
      unsigned long long sum = 0;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 x = quick(v[e], v[e + 1]);
        w[e] = x.x, w[e + 1] = x.y;
        sum = sum2(sum, pack2(x.x, x.y));
      }
      const float2 z = unpack2(sum);
      if (z.x + z.y < INFINITY) return z.x + z.y;  // else one is NaN
    }
    return slow_weights(v, i, w);
  }
  template <typename L>
  __device__ __noinline__ float slow_weights(const Eight<L> v, int i, float (&w)[E]) const {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sum += w[e] = weight(v[e], i + e);
    return sum;
  }
  // of U groups: their sum
  template <int U, typename G>
  __device__ __forceinline__ float sum_of(const G (&x)[U]) const {
    if (plain) {
      unsigned long long sum[2] = {0, 0};
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 w = quick(x[u].v[e], x[u].v[e + 1]);
          sum[e / 2 % 2] = sum2(sum[e / 2 % 2], pack2(w.x, w.y));
        }
      const float2 z = unpack2(sum2(sum[0], sum[1]));
      if (z.x + z.y < INFINITY) return z.x + z.y;
    }
    float sum = 0.f, w[E];
#pragma unroll
    for (int u = 0; u < U; ++u) sum += slow_weights(x[u].v, 0, w);
    return sum;
  }
};

// the largest of eight values (-inf where all are NaN)
__device__ __forceinline__ float largest(const Eight<float>& v) {
  const float a = fmaxf(fmaxf(fmaxf(v[0], v[1]), v[2]), fmaxf(fmaxf(v[3], v[4]), v[5]));
  return fmaxf(fmaxf(fmaxf(a, v[6]), v[7]), -INFINITY);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float largest(const Eight<uint16_t>& v) {
  const uint32_t a = max_bf16x2(max_bf16x2(v.w[0], v.w[1]), max_bf16x2(v.w[2], v.w[3]));
  return fmaxf(fmaxf(bf_lo(a), bf_hi(a)), -INFINITY);
}

// (a NaN loses)
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
// the smallest index among the lanes that have the largest value
__device__ __forceinline__ int warp_first(float x, float top, int at) {
  return __reduce_min_sync(0xffffffffu, x == top ? at : INT_MAX);
}

// A thread's sum of weights, of groups of them. What an add rounds off goes into the next one: a
// block that has a row to itself adds up vocab / 2048 groups a thread, which without that could all
// be rounded the same way (2^-15 of a sum of 2^19 equal values).
// In units of 2^-24 a row's sum is then off by 46 at most (10 adds of 32 weights, 2 here, 5 for the
// lane's, the warp's and the block's reference each, 14 adds of lanes and parts, the reciprocal and
// its product 5), and by what its weights are off by: of a weight 2^-z four for the exponential and
// 4 ln 2 z for the difference, log2(e) / temperature and their product; z up to log2 vocab matters,
// at 2^30 88. A probability e^-28 of the largest: 46 + 88 + 4 + 112 = 250 < 256.
struct Sum {
  float total = 0.f, over = 0.f;  // over: what total is too large by
  __device__ __forceinline__ void add(float x) {
    const float y = x - over, t = total + y;
    over = (t - total) - y;
    total = t;
  }
  __device__ __forceinline__ void scale(float f) { total *= f, over *= f; }
};

// ---- the kernel --------------------------------------------------------------------------

// The rows that a pass goes over, and a group of eight values of each.
template <typename T, typename... R>
struct Rows {
  struct Group {
    Eight<T> v;
    typename Rows<R...>::Group rest;
  };
  const T* row;
  float fill;
  Rows<R...> rest;
  template <bool VEC>
  __device__ __forceinline__ void load(int i, int end, Group& to) const {
    load8<T, VEC>(row, i, end, fill, to.v);
    rest.template load<VEC>(i, end, to.rest);
  }
};
template <typename T>
struct Rows<T> {
  struct Group {
    Eight<T> v;
  };
  const T* row;
  float fill;
  template <bool VEC>
  __device__ __forceinline__ void load(int i, int end, Group& to) const {
    load8<T, VEC>(row, i, end, fill, to.v);
  }
};

// The thread's groups of eight values in ascending order, U at a time, kStride apart:
// take(i, groups). The next U are loaded while the ones before are taken; what lies behind
// the end is `fill`.
constexpr int kStride = kThreads * E;
template <bool VEC, int U, typename R, typename Take>
__device__ __forceinline__ void over_values(int first, int hi, const R& rows, Take take) {
  typename R::Group next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) rows.template load<VEC>(first + u * kStride, hi, next[u]);
#pragma unroll 1
  for (int i = first; i < hi; i += U * kStride) {
    typename R::Group now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      now[u] = next[u];
      if (i + U * kStride < hi) rows.template load<VEC>(i + (U + u) * kStride, hi, next[u]);
    }
    take(i, now);
  }
}

// One cluster walks a sequence's tree, each block with its part of the vocabulary. A step
// is a sum over a row: a node's softmax, what a rejection leaves (only where another
// child follows it), the race. Each warp's part of it goes to every block's shared memory,
// and after one barrier each warp adds all of them up in the same order. One warp of
// block 0 alone reads what decides the walk beside the sums (the tree, the random numbers,
// the children's logits, the temperature) and hands it on, beside the others' work, so that all
// blocks take the same way to the same barriers whatever the inputs are.
// Bound by latency. Few sequences: by the chain of a step, about 5000 cycles with 16 blocks on a
// row of 128256 values: 1900 until the part's sum is there (memory, then eight values at a
// time), 500 to hand it on, 1300 at the barrier, 1000 to add up the parts, 500 to decide; 8
// trees of 64, 1 to 6 nodes accepted, take 26 us. Many: by the sequences with the longest
// chains, whose four blocks have 5700 cycles of a step to read and sum 32064 values each; 64
// chains of 8, 132 MB of rows, take 52 us, 2.5 TB/s. Measured and slower: copies to shared
// memory ahead of the sums, 16 bytes a thread each (4300 cycles for the 1900); two groups of
// values at a time in the race or the residual's sum (registers; 59 us); 512 threads a block
// (clusters of 16 of which fewer are resident: 46 us for 8 sampled trees instead of 35).
template <typename L, typename Q, bool VEC>
__global__ void __launch_bounds__(kThreads + 32, 2) verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ Shared sm;
  cluster_arrive();  // waited for before the first look at another block's memory
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = cluster_rank(), blocks = cluster_size(), b = blockIdx.x / blocks;
  const int64_t base = (int64_t)b * p.T;
  // the deciding warps take no values
  const int lo = min(p.V, rank * p.span), hi = warp == kWarps ? lo : min(p.V, lo + p.span);
  const int first = lo + tid * E;
  const bool decides = rank == 0 && warp == kWarps;
  const bool has_draft = p.draft != nullptr;
  float heat = p.temperature ? __ldg(p.temperature + b) : 1.f;
  const float* noise = p.noise + (int64_t)b * p.noise_stride;

  // lane l of the deciding warp holds nodes l and l + 32 of a tree
  int n = 0;
  int par[2] = {-1, -1}, tok[2] = {-1, -1};
  float uni[2] = {0.f, 0.f};
  if (decides) {
    n = clamped(p.counts, b, p.T);
    if (p.parents) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = lane + 32 * h;
        if (t < n) {
          par[h] = __ldg(p.parents + base + t);
          tok[h] = __ldg(p.tokens + base + t);
          uni[h] = __ldg(p.uniform + base + t);
        }
      }
    }
    for (int t = lane; t < p.T; t += 32) p.path[base + t] = t == 0 && n > 0 ? 0 : -1;
    __syncwarp();  // before the path's entries
  }
  // the block's part of a row of `size`-byte values, into the L2 cache
  auto fetch_part = [&](const void* row, int size) {
    if (VEC && warp == kWarps && lane == 0)
      prefetch((const uint8_t*)row + (size_t)lo * size, (uint32_t)(min(p.V, lo + p.span) - lo) * size / 16 * 16);
  };
  fetch_part((const L*)p.logits + base * p.logits_stride, sizeof(L));
  fetch_part(noise, 4);

  int step = 0, node_step = 0, cur = 0, taken = 1, gone = 0;
  float c = 0.f, mass = 1.f;  // c_j, N_j
  Softmax f;
  bool some = true;
  const L* row = nullptr;
  const Q* draft = nullptr;

  // hands the warp's part (the same in all lanes) to every block; the barrier
  auto exchange = [&](uint2 x) {
    if (warp < kWarps && lane < blocks) put_remote(&sm.part[step & 1][rank * kWarps + warp], lane, x);
    cluster_arrive();
    cluster_wait();
  };
  // part i of the lane's of the exchange's
  auto part = [&](int i, uint2 none) {
    const int at = lane + 32 * i;
    return at < blocks * kWarps ? sm.part[step & 1][at] : none;
  };
  constexpr int kParts = kMaxCluster * kWarps / 32;

  f.k = fmaxf(1.4426950408889634f / heat, 1e-38f);
  for (;;) {
    // ---- the node's softmax, and its children
    row = (const L*)p.logits + (base + cur) * p.logits_stride;
    draft = (const Q*)p.draft + (base + cur) * p.draft_stride;
    // (more than two rounds of loads: into the L2 cache at once: 5300 to 5700 cycles, else 6900 to 7700)
    if (step > 0 && p.span > 16 / (int)sizeof(L) * kStride) fetch_part(row, sizeof(L));
    f.only = -1;
    f.top = -INFINITY;
    Sum all_of;
    int at = INT_MAX;  // heat not above 0: the first index of the largest
    const Rows<L> values{row, -INFINITY};
    if (heat > 0.f) {
      // (the reference moves only where it has to, by 2^kSlack: what its moves round falls off
      // with what they scale, however often a row's largest value changes)
      constexpr int U = 8 / sizeof(L);
      float high = -INFINITY;
      over_values<VEC, U>(first, hi, values, [&](int, const auto& x) {
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, largest(x[u].v));
        high = fmaxf(high, top);
        if ((top - f.top) * f.k > kSlack) {
          all_of.scale(fast_exp2((f.top - top) * f.k));
          f.top = top;
          f.set_plain();
        }
        if (f.top > -INFINITY) all_of.add(f.sum_of(x));
      });
      if (high > f.top) {
        all_of.scale(fast_exp2((f.top - high) * f.k));
        f.top = high;
      }
    } else {
      over_values<VEC, 1>(first, hi, values, [&](int i, const auto& x) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (x[0].v[e] > f.top) f.top = x[0].v[e], at = i + e;
      });
      if (f.top == -INFINITY) at = INT_MAX;
    }
    if (step == 0) cluster_wait();
    if (decides) {
      // (a child comes behind its parent)
      Child kid[2];
      bool is_kid[2] = {false, false};
      auto look = [&](int h, int t, int x, float u) {
        if ((unsigned)x >= (unsigned)p.V) return;
        is_kid[h] = true;
        kid[h].l = load1(row + x);
        kid[h].q = has_draft ? probability(load1(draft + x)) : 1.f;
        kid[h].u = u > 0.f ? fminf(u, 1.f) : 0.f;
        kid[h].token = x;
        kid[h].node = t;
      };
      if (p.parents) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (par[h] == cur && lane + 32 * h > cur) look(h, lane + 32 * h, tok[h], uni[h]);
      } else if (lane == 0 && cur + 1 < n) {
        look(0, cur + 1, __ldg(p.tokens + base + cur + 1), __ldg(p.uniform + base + cur + 1));
      }
      const unsigned k0 = __ballot_sync(0xffffffffu, is_kid[0]), k1 = __ballot_sync(0xffffffffu, is_kid[1]);
      const unsigned below = (1u << lane) - 1;
      const int place[2] = {__popc(k0 & below), __popc(k0) + __popc(k1 & below)};
      const int kids = n == 0 ? -1 : __popc(k0) + __popc(k1), to = node_step & 1;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (is_kid[h]) sm.kid[place[h]] = kid[h];
      __syncwarp();
      if (lane < blocks) put_remote(&sm.head[to], lane, make_uint2(kids, __float_as_uint(heat)));
      for (int i = lane; i < kids * blocks; i += 32) {
        const int j = i / blocks, r = i - j * blocks;
        const Child k = sm.kid[j];
        put_remote(&sm.child[to][j], r, make_uint4(__float_as_uint(k.l), __float_as_uint(k.q), __float_as_uint(k.u), k.token));
        put_remote(&sm.child_node[to][j], r, make_uint2(k.node, 0));
      }
      __syncwarp();
    }
    {
      const float top = warp_max(f.top);
      if (heat > 0.f) {
        float sum = all_of.total;
        sum = warp_sum(f.top == top ? sum : sum > 0.f ? sum * fast_exp2((f.top - top) * f.k) : 0.f);
        exchange(make_uint2(__float_as_uint(top), __float_as_uint(sum)));
      } else {
        exchange(make_uint2(__float_as_uint(top), (uint32_t)warp_first(f.top, top, at)));
      }
    }
    const int here = node_step++ & 1;
    const uint2 head = sm.head[here];
    const int kids = (int)head.x;
    if (step == 0 && heat != __uint_as_float(head.y)) {  // (what decides the walk comes from block 0 alone)
      heat = __uint_as_float(head.y);
      f.k = fmaxf(1.4426950408889634f / heat, 1e-38f);
    }
    {
      uint2 x[kParts];
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        x[i] = part(i, make_uint2(0xff800000u, 0));
        top = fmaxf(top, __uint_as_float(x[i].x));
      }
      f.top = top = warp_max(top);
      if (heat > 0.f) {
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const float t = __uint_as_float(x[i].x), s = __uint_as_float(x[i].y);
          all += t == top ? s : s > 0.f ? s * fast_exp2((t - top) * f.k) : 0.f;
        }
        f.inv = __fdividef(1.f, warp_sum(all));  // (a sum of 1 to 2^30 weights of at most 1)
      } else {
        int least = INT_MAX;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          if (__uint_as_float(x[i].x) == top && lane + 32 * i < blocks * kWarps) least = min(least, (int)x[i].y);
        f.only = __reduce_min_sync(0xffffffffu, least);
        f.inv = 1.f;
      }
      f.set_plain();
    }
    ++step;
    some = kids >= 0 && f.top > -INFINITY;
    if (kids < 0) taken = 0;
    if (!some) break;
    // ---- its children in turn
    int took = -1;
    c = 0.f, mass = 1.f, gone = 0;
    for (int j = 0; j < kids; ++j) {
      const uint4 x = sm.child[here][j];
      const Child kid{__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), (int)x.w,
                      (int)sm.child_node[here][j].x};
      const float px = f.weight(kid.l, kid.token) * f.inv;
      float left = px;
      if (has_draft) {
        left = fmaxf(px - c * kid.q, 0.f);
      } else {
        for (int i = 0; i < gone; ++i)
          if (sm.gone[i] == kid.token) left = 0.f;
      }
      if (kid.u * kid.q * mass < left) {
        took = kid.node;
        break;
      }
      if (has_draft) {
        c += mass;
        if (j + 1 == kids) break;  // nobody asks for what is left
        if (j == 0) fetch_part(draft, sizeof(Q));
        Sum sum;
        over_values<VEC, 1>(first, hi, Rows<L, Q>{row, -INFINITY, {draft, 0.f}}, [&](int i, const auto& x) {
          float w[E];
          f.weights(x[0].v, i, w);
#pragma unroll
          for (int e = 0; e < E; ++e) w[e] = fmaxf(w[e] * f.inv - c * probability(x[0].rest.v[e]), 0.f);
          sum.add(((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7])));
        });
        exchange(make_uint2(__float_as_uint(warp_sum(sum.total)), 0));
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) all += __uint_as_float(part(i, make_uint2(0, 0)).x);
        mass = warp_sum(all);
        ++step;
      } else if (left > 0.f) {
        __syncthreads();  // everybody has looked at the list
        if (tid == 0) sm.gone[gone] = kid.token;
        __syncthreads();
        ++gone;
        mass = fmaxf(mass - left, 0.f);
      }
    }
    if (took < 0) break;
    cur = took;
    if (decides && lane == 0) p.path[base + taken] = cur;
    ++taken;
  }

  // ---- the race over what is left; where rounding leaves nothing, over p itself
  int next = -1;
  for (int again = 0; some && again < 2; ++again) {
    const bool all = again || !has_draft || c == 0.f;
    if (!all) fetch_part(draft, sizeof(Q));
    float best = 0.f;
    int at = -1;
    // (the first of the largest scores: a thread meets its values in ascending order)
    auto race = [&](int i, float(&w)[E], const Eight<float>& e) {
#pragma unroll
      for (int j = 0; j < E; ++j) w[j] = __fdividef(w[j], fminf(fmaxf(e[j], 1e-30f), 1e30f));
      const float top = fmaxf(fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])), fmaxf(fmaxf(w[4], w[5]), fmaxf(w[6], w[7])));
      if (top > best) {
        best = top;
#pragma unroll
        for (int j = E - 1; j >= 0; --j)
          if (w[j] == top) at = i + j;
      }
    };
    if (all) {
      over_values<VEC, 1>(first, hi, Rows<L, float>{row, -INFINITY, {noise, 1.f}}, [&](int i, const auto& x) {
        float w[E];
        f.weights(x[0].v, i, w);
        if (!again)
          for (int j = 0; j < gone; ++j) {
            const int d = sm.gone[j] - i;
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (d == e) w[e] = 0.f;
          }
        race(i, w, x[0].rest.v);
      });
    } else {
      const float by = c * __fdividef(1.f, f.inv);  // in units of the weights
      over_values<VEC, 1>(first, hi, Rows<L, Q, float>{row, -INFINITY, {draft, 0.f, {noise, 1.f}}}, [&](int i, const auto& x) {
        float w[E];
        f.weights(x[0].v, i, w);
#pragma unroll
        for (int j = 0; j < E; ++j) w[j] = fmaf(-by, probability(x[0].rest.v[j]), w[j]);
        race(i, w, x[0].rest.rest.v);
      });
    }
    {
      const float top = warp_max(best);
      exchange(make_uint2(__float_as_uint(top), (uint32_t)warp_first(best, top, at)));
    }
    uint2 x[kParts];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      x[i] = part(i, make_uint2(0, 0));
      top = fmaxf(top, __uint_as_float(x[i].x));
    }
    top = warp_max(top);
    ++step;
    if (top > 0.f) {
      int least = INT_MAX;
#pragma unroll
      for (int i = 0; i < kParts; ++i)
        if (__uint_as_float(x[i].x) == top) least = min(least, (int)x[i].y);
      next = __reduce_min_sync(0xffffffffu, least);
      break;
    }
  }
  if (decides && lane == 0) {
    p.accepted[b] = taken;
    p.next[b] = next;
  }
}

// Launches with clusters of the largest power of two that gives each thread of a block eight values
// and leaves every cluster of the call resident at once, as the device says for this kernel: a
// cluster lies in one GPC, so that 14 or 15 of 16 blocks (by the chip), 36 of 8 and 74 of 4 are
// resident where two blocks to each of 152 SMs would be 19, 38 and 76. One more than fit would wait
// for a whole walk: chains of 4 over 128256 values, 16 sequences with clusters of 16 29.6 us, of 8
// 18.8; 38 with 8 40.9, with 4 32.8; 76 with 4 59.7, with 2 52.6.
template <typename L, typename Q, bool VEC>
int launch(VerifyParams p, int batch, cudaStream_t st) {
  constexpr int kSizes = 4, kDevices = 64;  // of 16, 8, 4 and 2 blocks
  static std::atomic<int> resident[kDevices][kSizes];  // 1 + how many; 0: not asked yet
  auto* fn = verify_kernel<L, Q, VEC>;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return op_cuda(e, "mk_tree_verify");
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads + 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int blocks = 1;
  for (int i = 0; i < kSizes && blocks == 1; ++i) {
    const int size = kMaxCluster >> i;
    if (p.V < size * kThreads * E) continue;
    int fit = device < kDevices ? resident[device][i].load(std::memory_order_acquire) : 0;
    if (fit == 0) {
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return op_cuda(e, "mk_tree_verify");
      attr.val.clusterDim.x = size;
      cfg.gridDim = dim3(size);
      e = cudaOccupancyMaxActiveClusters(&fit, fn, &cfg);
      if (e != cudaSuccess) return op_cuda(e, "mk_tree_verify");
      ++fit;
      if (device < kDevices) resident[device][i].store(fit, std::memory_order_release);
    }
    if (batch < fit) blocks = size;
  }
  p.span = (int)(((int64_t)p.V + blocks - 1) / blocks + E - 1) / E * E;
  attr.val.clusterDim.x = blocks;
  cfg.gridDim = dim3((unsigned)batch * blocks);
  return op_cuda(cudaLaunchKernelEx(&cfg, fn, p), "mk_tree_verify");
}

template <bool VEC>
int launch_types(const VerifyParams& p, int type, bool narrow, int batch, cudaStream_t st) {
  if (type == MK_TYPE_FP32)
    return narrow ? launch<float, uint16_t, VEC>(p, batch, st)
                  : launch<float, float, VEC>(p, batch, st);
  return narrow ? launch<uint16_t, uint16_t, VEC>(p, batch, st)
                : launch<uint16_t, float, VEC>(p, batch, st);
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
  const VerifyParams p{logits, draft, logits_stride, draft_stride, noise_stride, temperature, uniform,
                       noise, tokens, parents, counts, path, accepted, next, n_tokens, vocab, 0};
  cudaStream_t st = (cudaStream_t)stream;
  const bool narrow = draft && draft_type == MK_TYPE_BF16;
  auto by16 = [](const void* at, int64_t stride, size_t size) {
    return aligned(at, 16) && stride * size % 16 == 0;
  };
  const bool vec = by16(logits, logits_stride, size) && by16(noise, noise_stride, 4) &&
                   (!draft || by16(draft, draft_stride, draft_size));
  return vec ? launch_types<true>(p, type, narrow, batch, st)
             : launch_types<false>(p, type, narrow, batch, st);
}
