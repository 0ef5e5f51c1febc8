// Attention of a batch whose groups share a prefix (include/mk.h,
// mk_prefix_attention): its line of work over the kernel for many rows
// (mk_tree_attention_tc.cuh), the kernel that joins a row's shares, the entry point.
//
// The line of work has two kinds of entry. A group's prefix: the rows of all its
// sequences (sequence, node, query head of the kv-head's group) against the prefix's
// keys, which are therefore fetched once for up to 128 or 256 rows, nothing masked. A
// sequence's own keys behind the prefix: its nodes' rows, masked by the tree. Each is,
// for every kv-head and row tile, an item of tiles of 128 keys; the items of all form
// one line that is cut into equal shares, one per block. A row's result is joined
// from the shares of both items by a second kernel (an item that was not cut leaves
// its sums in a place of its row's own), but where there is no prefix a whole item
// writes its rows.
#include <algorithm>
#include <type_traits>

#include "mk_tree_attention_tc.cuh"

namespace mk {

struct PrefixLine;
struct PrefixShare;

struct PrefixParams : AttnParams {
  using Line = PrefixLine;
  using Share = PrefixShare;
  int n_groups;
  const int32_t *first, *shared;   // DEVICE [n_groups]
  int64_t cut_rows;                // rows of the workspace before the uncut items'
};

// The line in shared memory: places before entry e (the groups, then the sequences),
// the sequences' starts, counts (at their bounds) and groups, the groups' first
// sequences and the lengths of their prefixes.
struct PrefixLine {
  static constexpr int kNone = 0xffff;
  int prefix[2 * kMaxSeqs + 1];
  int start[kMaxSeqs], shared[kMaxSeqs];
  uint16_t group[kMaxSeqs], first[kMaxSeqs];
  uint8_t count[kMaxSeqs];
  // slots of sequence b that are its group's
  __device__ __forceinline__ int from(int b) const { return group[b] == kNone ? 0 : shared[group[b]]; }
  // sequences of group j
  __device__ __forceinline__ int size(int j, int n_groups, int B) const {
    return (j + 1 < n_groups ? first[j + 1] : B) - first[j];
  }
};

__device__ __forceinline__ int row_tiles_of(const PrefixParams& p, int rows) {
  return (rows + p.row_tile - 1) / p.row_tile;
}

// Fills it with one warp. A group's prefix is at most the shortest context of its
// sequences (those that have nodes; 0 without one).
__device__ __forceinline__ void work_line(const PrefixParams& p, PrefixLine& line) {
  const int lane = threadIdx.x % 32;
  int last = 0;
  for (int j0 = 0; j0 < p.n_groups; j0 += 32) {
    const int j = j0 + lane;
    int x = j < p.n_groups ? min(max(__ldg(p.first + j), 0), p.B) : 0;
    // not before the groups before it
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x = max(x, y);
    }
    x = max(x, last);
    last = __shfl_sync(0xffffffffu, x, 31);
    if (j < p.n_groups) {
      line.first[j] = (uint16_t)x;
      line.shared[j] = INT_MAX;
    }
  }
  __syncwarp();
  for (int b = lane; b < p.B; b += 32) {
    const int start = clamped(p.starts, b, p.cache.capacity), count = clamped(p.counts, b, p.T);
    line.start[b] = start;
    line.count[b] = (uint8_t)count;
    int lo = -1, hi = p.n_groups;  // the last group that begins at b or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (line.first[mid] <= b) lo = mid;
      else hi = mid;
    }
    line.group[b] = lo < 0 ? PrefixLine::kNone : (uint16_t)lo;
    if (lo >= 0 && count > 0) atomicMin(&line.shared[lo], min(start, max(__ldg(p.shared + lo), 0)));
  }
  __syncwarp();
  int sum = 0;
  const int entries = p.n_groups + p.B;
  for (int e0 = 0; e0 < entries; e0 += 32) {
    const int e = e0 + lane;
    int keys = 0, rows = 0;
    if (e < p.n_groups) {
      keys = line.shared[e];
      if (keys == INT_MAX) line.shared[e] = keys = 0;
      rows = line.size(e, p.n_groups, p.B) * p.T * p.G;
    }
    __syncwarp();
    if (e >= p.n_groups && e < entries) {
      const int b = e - p.n_groups;
      if (line.count[b] > 0) keys = min(line.start[b] + line.count[b], p.cache.capacity) - line.from(b);
      rows = line.count[b] * p.G;
    }
    int x = keys > 0 ? places_of(p, keys) * row_tiles_of(p, rows) * p.cache.n_kv : 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (e < entries) line.prefix[e + 1] = sum + x;
    sum += __shfl_sync(0xffffffffu, x, 31);
  }
  if (lane == 0) line.prefix[0] = 0;
  __syncwarp();
}

__device__ __forceinline__ int all_places(const PrefixParams& p, const PrefixLine& line) {
  return line.prefix[p.n_groups + p.B];
}

// A share of the line that lies in one item. Of a prefix b is the group's first
// sequence, whose rows are read, and no key is a node (start = len, no count).
struct PrefixShare {
  int b, g, k0, n, nt;
  bool begins, is_prefix;
  int count, start, len, rows;
  int first;  // slot of the item's first key
  int row0;   // first row of the item's row tile
};

__device__ __forceinline__ bool next_share(const PrefixParams& p, const PrefixLine& line, int u_begin,
                                           int u_end, int& u, PrefixShare& s) {
  do {
    if (u >= u_end) return false;
    int lo = 0, hi = p.n_groups + p.B;  // the last entry whose prefix is <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (line.prefix[mid] <= u) lo = mid;
      else hi = mid;
    }
    s.is_prefix = lo < p.n_groups;
    if (s.is_prefix) {
      s.b = line.first[lo];
      s.count = s.first = 0;
      s.start = s.len = line.shared[lo];
      s.rows = line.size(lo, p.n_groups, p.B) * p.T * p.G;
    } else {
      s.b = lo - p.n_groups;
      s.count = line.count[s.b];
      s.start = line.start[s.b];
      s.first = line.from(s.b);
      s.len = min(s.start + s.count, p.cache.capacity);
      s.rows = s.count * p.G;
    }
    const int tiles = row_tiles_of(p, s.rows), places = places_of(p, s.len - s.first);
    const int at = u - line.prefix[lo];
    s.nt = places - p.extra;
    // floor(at / places), which is below 2^21: the rounded quotient is at most one off
    int item = (int)__fdividef((float)at, (float)places);
    if (item * places > at) --item;
    else if ((item + 1) * places <= at) ++item;
    s.g = tiles == 1 ? item : item / tiles;
    s.row0 = (item - s.g * tiles) * p.row_tile;
    const int tile0 = line.prefix[lo] + item * places + p.extra;  // place of the item's tile 0
    s.k0 = max(u - tile0, 0);
    s.n = min(u_end - tile0, s.nt) - s.k0;
    s.begins = u == u_begin;
    u = tile0 + s.nt;
  } while (s.n <= 0);  // a part that ends before the item's first tile
  return true;
}

__device__ __forceinline__ int first_slot(const PrefixShare& s) { return s.first; }
__device__ __forceinline__ int first_row(const PrefixShare& s) { return s.row0; }
__device__ __forceinline__ bool row_there(const PrefixParams& p, const PrefixLine& line,
                                          const PrefixShare& s, int row) {
  if (row >= s.rows) return false;
  if (!s.is_prefix) return true;
  const int node = row / p.G, seq = node / p.T;
  return node - seq * p.T < line.count[s.b + seq];
}
// (of a prefix no row has a node among the keys)
__device__ __forceinline__ int row_node(const PrefixParams& p, const PrefixShare& s, int row) {
  return s.is_prefix ? -1 : row / p.G;
}
// (rows of a prefix are those of its first sequence and on)
__device__ __forceinline__ int64_t row_offset(const PrefixParams& p, const PrefixShare& s, int row,
                                              int D, int64_t stride) {
  return row_offset(p, s.b, s.g, row, D, stride);
}
__device__ __forceinline__ bool is_final(const PrefixShare& s) {
  return !s.is_prefix && s.first == 0 && s.n == s.nt;
}
// The workspace's rows: two row tiles for each group of blocks, then each row's sums
// over an uncut prefix, each row's over uncut own keys.
__device__ __forceinline__ size_t uncut_slot(const PrefixParams& p, bool is_prefix, int b, int g,
                                             int row) {
  const int64_t at = ((int64_t)b * p.T + row / p.G) * p.nh + g * p.G + row % p.G;
  return p.cut_rows + (is_prefix ? 0 : (int64_t)p.B * p.T * p.nh) + at;
}
__device__ __forceinline__ size_t share_slot(const PrefixParams& p, int group, const PrefixShare& s,
                                             int, int local, int row) {
  if (s.n == s.nt) return uncut_slot(p, s.is_prefix, s.b, s.g, row);
  return part_slot(p, group, s.begins, 0) * p.row_tile + local;
}

namespace {

// Joins a row's shares, of its group's prefix and of its own keys, a warp to a row
// (FEW: a block's four warps, every fourth share each). The lanes read the shares'
// maxima and sums 32 at a time, so that every share's factor is known before its
// columns are read; the order is fixed.
template <int D, bool FEW, typename T>
__global__ void __launch_bounds__(128) prefix_attention_join(const __grid_constant__ PrefixParams p) {
  constexpr int E = D / 32, TURNS = FEW ? 4 : 1, U = FEW ? 8 : 2;  // U: loads in flight
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ PrefixLine line;
  __shared__ Vec other[4][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, turn = FEW ? warp : 0;
  const int b = blockIdx.y / p.cache.n_kv, g = blockIdx.y % p.cache.n_kv;
  if (warp == 0) work_line(p, line);
  __syncthreads();
  const int row = FEW ? blockIdx.x : blockIdx.x * 4 + warp;
  const Cut cut(all_places(p, line), p);
  // Of both items: the places where it begins, the blocks that have a part of it (n of them
  // from g0 on), the row's number in its row tile.
  int item0[2], g0[2], n[2] = {0, 0}, local[2];
  const bool there = row < line.count[b] * p.G;
  if (there) {
    const int from = line.from(b);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const bool pre = which == 0;
      const int keys = pre ? from : min(line.start[b] + line.count[b], p.cache.capacity) - from;
      if (keys == 0) continue;
      const int j = line.group[b];
      const int r = pre ? (b - line.first[j]) * p.T * p.G + row : row;
      const int rows = pre ? line.size(j, p.n_groups, p.B) * p.T * p.G : line.count[b] * p.G;
      const int places = places_of(p, keys), rt = r / p.row_tile;
      local[which] = r - rt * p.row_tile;
      item0[which] = line.prefix[pre ? j : p.n_groups + b] + (g * row_tiles_of(p, rows) + rt) * places;
      g0[which] = cut.group_of(item0[which] + p.extra);
      n[which] = cut.group_of(item0[which] + places - 1) - g0[which] + 1;
    }
  }
  const int all = n[0] + n[1];
  const bool joins = all > 1 || n[0] == 1;  // else it was written whole
  griddep_wait();
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (joins) {
    // lane i: where share s0 + i keeps the row (-1: no share, or no key seen in
    // it), its maximum and sum
    int64_t at;
    float ms, ls;
    auto look = [&](int s0) {
      const int s = s0 + lane;
      at = -1, ms = -INFINITY, ls = 0.f;
      if (s < all) {
        const int which = s < n[0] ? 0 : 1;
        const int group = (which ? g0[1] - n[0] : g0[0]) + s;
        int64_t x;
        if ((which ? n[1] : n[0]) == 1) {
          x = (int64_t)uncut_slot(p, which == 0, b, g, row);
        } else {
          const int u0 = cut.begin(group);
          if (u0 == cut.begin(group + 1)) return;  // one of more groups than places
          x = (int64_t)part_slot(p, group, u0 >= (which ? item0[1] : item0[0]), 0) * p.row_tile +
              (which ? local[1] : local[0]);
        }
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + x);
        if (ml.y != 0.f) at = x, ms = ml.x, ls = ml.y;
      }
    };
    float m = -INFINITY;
    for (int s0 = 0; s0 < all; s0 += 32) {
      look(s0);
      m = fmaxf(m, ms);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int s0 = 0; s0 < all; s0 += 32) {
      if (all > 32) look(s0);  // else the lanes still have it
      const float f = at < 0 ? 0.f : fast_exp2(ms - m);
      l += ls * f;
      const int here = min(32, all - s0);
      for (int k0 = turn; k0 < here; k0 += U * TURNS) {
        Vec v[U];
        float w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int k = k0 + i * TURNS;
          const int64_t x = __shfl_sync(0xffffffffu, at, k & 31);
          w[i] = __shfl_sync(0xffffffffu, f, k & 31);
          v[i] = Vec{};
          if (k < here && x >= 0) v[i] = __ldcg(reinterpret_cast<const Vec*>(p.part_o + x * D) + lane);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float* c = reinterpret_cast<const float*>(&v[i]);
          const bool has = k0 + i * TURNS < here;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += has ? c[e] * w[i] : 0.f;
        }
      }
    }
#pragma unroll
    for (int d = 16; d; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
  }
  if constexpr (FEW) {
    Vec v;
#pragma unroll
    for (int e = 0; e < E; ++e) reinterpret_cast<float*>(&v)[e] = o[e];
    other[warp][lane] = v;
    __syncthreads();
    if (turn != 0) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const Vec x = other[w][lane];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += reinterpret_cast<const float*>(&x)[e];
    }
  }
  if (!joins) return;
  const float f = 1.f / l;
  const int64_t off = row_offset(p, b, g, row, D, p.os) + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float x = l == 0.f ? 0.f : o[e] * f, y = l == 0.f ? 0.f : o[e + 1] * f;  // 0: no key seen
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>((float*)p.out + off + e) = make_float2(x, y);
    else
      *reinterpret_cast<uint32_t*>((uint16_t*)p.out + off + e) = bf16x2_rn(x, y);
  }
}

constexpr char kName[] = "mk_prefix_attention";

struct PrefixPlan {
  int row_tile, groups;
  int64_t cut_rows, rows;  // rows of the workspace: of cut items, all
};

// The row tile by the rows of a group, were all alike.
int row_tile_of(int B, int T, int G, int type, int n_groups) {
  const int64_t each = ((int64_t)B * T * G + n_groups - 1) / n_groups;
  if (type == MK_TYPE_FP32) return each <= 32 ? 32 : 128;
  return each <= 128 ? 128 : 256;
}

int check_prefix(const mk_cache* cache, int batch, int n_tokens, int n_heads, int type, int n_groups,
                 CacheView* view) {
  if (int rc = check_cache(cache, batch, true, view)) return rc;
  if (n_tokens < 1 || n_tokens > MK_MAX_TREE)
    return op_fail(MK_ERR_INVALID, "n_tokens must be 1 to MK_MAX_TREE");
  if (n_groups < 1 || n_groups > batch)
    return op_fail(MK_ERR_INVALID, "n_groups must be 1 to batch");
  if (type != MK_TYPE_BF16 && type != MK_TYPE_FP32)
    return op_fail(MK_ERR_INVALID, "type must be MK_TYPE_BF16 or MK_TYPE_FP32");
  if (cache->n_kv_heads > 4096 || (int64_t)batch * cache->n_kv_heads > 65535)
    return op_fail(MK_ERR_INVALID, "batch x n_kv_heads must be at most 65535");
  if (n_heads < 1 || n_heads % cache->n_kv_heads || n_heads / cache->n_kv_heads > 8)
    return op_fail(MK_ERR_INVALID,
                   "n_heads must be a multiple of n_kv_heads, at most 8 heads per kv-head");
  // the line's places: row tiles of own rows and of the groups' (each may have one begun)
  const int G = n_heads / cache->n_kv_heads, tile = row_tile_of(batch, n_tokens, G, type, n_groups);
  const int64_t rows = (int64_t)n_tokens * G;
  const int64_t tiles = batch * ((rows + tile - 1) / tile) + batch * rows / tile + n_groups;
  if (tiles * cache->n_kv_heads * (view->capacity / kKeys + 8) > INT32_MAX)
    return op_fail(MK_ERR_INVALID, "batch x n_tokens x n_heads x capacity: more than 2^31 tiles");
  return MK_OK;
}

int make_plan(int B, int T, int nh, int G, int type, int n_groups, PrefixPlan* pl) {
  int device = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return op_cuda(e, kName);
  pl->row_tile = row_tile_of(B, T, G, type, n_groups);
  pl->groups = n_sm;
  pl->cut_rows = (int64_t)2 * pl->groups * pl->row_tile;
  pl->rows = pl->cut_rows + 2 * (int64_t)B * T * nh;
  return MK_OK;
}

template <int D>
int launch_join(const PrefixParams& p, int type, cudaStream_t st) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const bool few = (int64_t)p.T * p.G * p.B * p.cache.n_kv <= 1024;
  cfg.gridDim = dim3(few ? p.T * p.G : (p.T * p.G + 3) / 4, p.B * p.cache.n_kv);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto* fn = type == MK_TYPE_FP32
                 ? (few ? prefix_attention_join<D, true, float> : prefix_attention_join<D, false, float>)
                 : (few ? prefix_attention_join<D, true, uint16_t> : prefix_attention_join<D, false, uint16_t>);
  return op_cuda(cudaLaunchKernelEx(&cfg, fn, p), kName);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

int mk_prefix_attention_workspace(const mk_cache* cache, int batch, int n_tokens, int n_heads,
                                  int type, int n_groups, size_t* bytes) {
  if (!bytes) return op_fail(MK_ERR_INVALID, "bytes is NULL");
  CacheView view;
  PrefixPlan pl;
  if (int rc = check_prefix(cache, batch, n_tokens, n_heads, type, n_groups, &view)) return rc;
  if (int rc = make_plan(batch, n_tokens, n_heads, n_heads / cache->n_kv_heads, type, n_groups, &pl))
    return rc;
  *bytes = (size_t)pl.rows * (cache->head_dim + 2) * sizeof(float);
  return MK_OK;
}

int mk_prefix_attention(const mk_cache* cache, int layer, int batch, int n_tokens, int n_heads,
                        int type, float scale, const void* q, int64_t q_stride, int n_groups,
                        const int32_t* first, const int32_t* prefix, const int32_t* starts,
                        const int32_t* parents, const int32_t* counts, void* out,
                        int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  PrefixParams p;
  PrefixPlan pl;
  if (int rc = check_prefix(cache, batch, n_tokens, n_heads, type, n_groups, &p.cache)) return rc;
  if (layer < 0 || layer >= cache->n_layers)
    return op_fail(MK_ERR_INVALID, "layer out of range [0, n_layers)");
  if (!q || !out || !first || !prefix || !starts || !workspace)
    return op_fail(MK_ERR_INVALID, "mk_prefix_attention: a NULL argument");
  if (!(scale > 0.f) || scale > 1e30f)
    return op_fail(MK_ERR_INVALID, "scale must be positive and finite");
  const int unit = type == MK_TYPE_FP32 ? 4 : 8;
  const int64_t row = (int64_t)n_heads * cache->head_dim;
  if (!aligned(q, 16) || !aligned(out, 16) || q_stride % unit || out_stride % unit ||
      q_stride < row || out_stride < row)
    return op_fail(MK_ERR_INVALID,
                   "q, out: 16-byte aligned rows, strides at least a row, are needed");
  if (!aligned(workspace, 256)) return op_fail(MK_ERR_INVALID, "workspace: not 256-byte aligned");
  if (int rc = make_plan(batch, n_tokens, n_heads, n_heads / cache->n_kv_heads, type, n_groups, &pl))
    return rc;
  if (workspace_bytes < (size_t)pl.rows * (cache->head_dim + 2) * sizeof(float))
    return op_fail(MK_ERR_INVALID, "workspace: smaller than its query says");
  p.k = (const uint16_t*)cache->k[layer];
  p.v = (const uint16_t*)cache->v[layer];
  p.q = q, p.out = out, p.qs = q_stride, p.os = out_stride;
  p.starts = starts, p.parents = parents, p.counts = counts;
  p.B = batch, p.T = n_tokens, p.nh = n_heads, p.G = n_heads / cache->n_kv_heads;
  p.tile_log2 = 7;
  p.extra = 4, p.row_tile = pl.row_tile, p.row_tiles = 1, p.groups = pl.groups;
  p.inv_groups = (uint32_t)std::min<uint64_t>((1ull << 32) / pl.groups + 1, UINT32_MAX);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.n_groups = n_groups, p.first = first, p.shared = prefix;
  p.cut_rows = pl.cut_rows;
  p.part_o = (float*)workspace;
  p.part_ml = p.part_o + (size_t)pl.rows * cache->head_dim;
  cudaStream_t st = (cudaStream_t)stream;
  if (int rc = launch_tc(p, p.groups, cache->head_dim, type, kName, st)) return rc;
  return cache->head_dim == 64 ? launch_join<64>(p, type, st) : launch_join<128>(p, type, st);
}

}  // extern "C"
