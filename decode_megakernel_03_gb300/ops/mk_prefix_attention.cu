// Attention of a batch whose groups share a prefix (include/mk.h,
// mk_prefix_attention): its line of work over the kernel for many rows
// (mk_tree_attention_tc.cuh), the kernel that joins a row's shares, the entry point.
//
// The line of work has two kinds of entry. A group's prefix: the rows of all its
// sequences (sequence, node, query head of the kv-head's group) against the prefix's
// keys, which are therefore fetched once for up to 128 or 256 rows, nothing masked. A
// sequence's own keys behind the prefix: its nodes' rows, masked by the tree. Each is,
// for every kv-head and row tile, an item of tiles of 128 keys; the items of all form
// one line that is cut into equal shares, one per block, so that blocks with long
// prefixes and blocks with many short sequences end together. A row's result is joined
// from the shares of both items by a second kernel (an item that was not cut leaves
// its sums in a place of its row's own), but where there is no prefix a whole item
// writes its rows.
//
// Measured on the 8B shape, bf16: 64 samples of two documents (32768 and 26215 keys, 256
// to 2048 own keys, 4 nodes each; 531 MB, 123 GFLOP) 222 us (211 without the code of kRun): the prefixes' tiles are
// bound by the products, which both parts of the weights go through (4400 cycles for two
// blocks of rows, 3072 of them products), the own keys' by the beginnings and ends of 512
// items (9000 cycles each) and their tiles (2000). 32 samples behind 8192 keys, 16 to 512
// own ones (68 MB) 37 us: 4 until a block has its line, 13 to 27 for its shares, 5 for
// the join. (The own keys by a kernel at warp level that also joins
// them with the prefix's sums, started early, took 252 and 47 us, this one then 234 and 41: it has the
// memory to itself only when the products are done.)
#include <algorithm>
#include <type_traits>

#include "mk_tree_attention_tc.cuh"

namespace mk {

struct PrefixLine;
struct PrefixShare;

// Where a sequence's two items are, for the kernel that joins its rows: the place where the
// entry begins, its tiles of keys (0: no item), its rows; the row of the sequence's
// first node in the prefix's item; the sequence's nodes.
struct alignas(16) RowPlan {
  int pre_base, pre_tiles, pre_rows, pre_row;
  int own_base, own_tiles, own_rows, pad;
};

struct PrefixParams : AttnParams {
  using Line = PrefixLine;
  using Share = PrefixShare;
  static constexpr bool kMixed = true;
  int n_groups;
  const int32_t *first, *shared;   // DEVICE [n_groups]
  int row_log2;                    // of row_tile
  uint32_t inv_G, inv_T;           // for div_by
  // The workspace: part_o, part_ml with two row tiles for each group of blocks (cut items), then
  // every row twice (uncut items, of a prefix and own); the runs; for each sequence its plan; the
  // line's length. A cut item's part_o holds eight columns of all rows of its tile and then the next
  // eight, so that neighbouring rows' threads store to neighbouring places (row after row 128
  // rows took 5900 cycles) and the join's lanes read whole sectors.
  int64_t cut_rows;
  RowPlan* plans;                  // [B]
  int* length;
};

// n / d for n * d < 2^32, inv = floor(2^32 / d) + 1 (d = 1: not used)
__device__ __forceinline__ int div_by(int n, int d, uint32_t inv) {
  return d == 1 ? n : (int)__umulhi((uint32_t)n, inv);
}

// ---- the line ------------------------------------------------------------------------

// The line in shared memory: places before entry e (the groups, then the sequences),
// the sequences' starts, counts (at their bounds) and groups, the groups' first
// sequences and the lengths of their prefixes.
struct PrefixLine {
  static constexpr int kNone = 0xffff;
  int prefix[2 * kMaxSeqs + 1];
  int start[kMaxSeqs], shared[kMaxSeqs];
  uint16_t group[kMaxSeqs], first[kMaxSeqs + 1];
  uint8_t count[kMaxSeqs];
  // slots of sequence b that are its group's
  __device__ __forceinline__ int from(int b) const { return group[b] == kNone ? 0 : shared[group[b]]; }
  // sequences of group j
  __device__ __forceinline__ int size(int j) const { return first[j + 1] - first[j]; }
};

// An entry's items: kv-heads, and for each its row tiles. A tile of keys of two blocks of 128
// rows is worth two places of the line (4400 cycles against 1750 to 2000 for one block's), a
// row tile's beginning and end p.extra.
struct Entry {
  int rows, tiles, row_tiles;  // tiles: of keys
  int places0, places;         // of a row tile that is not the last; of all row tiles of a kv-head
  __device__ __forceinline__ Entry(const PrefixParams& p, int rows_, int tiles_)
      : rows(rows_), tiles(tiles_), row_tiles((rows_ + p.row_tile - 1) >> p.row_log2) {
    places0 = (tiles << cost_log2(p, 0)) + p.extra;
    places = (row_tiles - 1) * places0 + (tiles << cost_log2(p, row_tiles - 1)) + p.extra;
  }
  __device__ __forceinline__ int cost_log2(const PrefixParams& p, int rt) const {
    return p.row_tile == 256 && rows - (rt << 8) > 128 ? 1 : 0;
  }
};
__device__ __forceinline__ int key_tiles(int keys) { return (keys + kKeys - 1) / kKeys; }

// Fills it with one warp. A group's prefix is at most the shortest context of its
// sequences (those that have nodes; 0 without one).
__device__ __forceinline__ void work_line(const PrefixParams& p, PrefixLine& line) {
  const int lane = threadIdx.x % 32;
  // (the first ones of everything are loaded at once)
  auto first_of = [&](int j) { return j < p.n_groups ? min(max(__ldg(p.first + j), 0), p.B) : 0; };
  auto start_of = [&](int b) { return b < p.B ? clamped(p.starts, b, p.cache.capacity) : 0; };
  auto count_of = [&](int b) { return b < p.B ? clamped(p.counts, b, p.T) : 0; };
  auto shared_of = [&](int j) { return j < p.n_groups ? max(__ldg(p.shared + j), 0) : 0; };
  int next_first = first_of(lane), start0 = start_of(lane), count0 = count_of(lane);
  const int shared0 = shared_of(lane);
  int last = 0;
  for (int j0 = 0; j0 < p.n_groups; j0 += 32) {
    const int j = j0 + lane;
    int x = next_first;
    next_first = first_of(j + 32);
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
  if (lane == 0) line.first[p.n_groups] = (uint16_t)p.B;
  __syncwarp();
  for (int b = lane; b < p.B; b += 32) {
    const int start = start0, count = count0;
    start0 = start_of(b + 32), count0 = count_of(b + 32);
    line.start[b] = start;
    line.count[b] = (uint8_t)count;
    int lo = -1, hi = p.n_groups;  // the last group that begins at b or before
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (line.first[mid] <= b) lo = mid;
      else hi = mid;
    }
    line.group[b] = lo < 0 ? PrefixLine::kNone : (uint16_t)lo;
    if (lo >= 0 && count > 0) atomicMin(&line.shared[lo], start);
  }
  __syncwarp();
  for (int j = lane; j < p.n_groups; j += 32) {
    const int least = line.shared[j];
    line.shared[j] = least == INT_MAX ? 0 : min(least, j == lane ? shared0 : shared_of(j));
  }
  __syncwarp();
  int sum = 0;
  const int entries = p.n_groups + p.B;
  for (int e0 = 0; e0 < entries; e0 += 32) {
    const int e = e0 + lane;
    int keys = 0, rows = 0;
    if (e < p.n_groups) {
      keys = line.shared[e];
      rows = line.size(e) * p.T * p.G;
    } else if (e < entries) {
      const int b = e - p.n_groups;
      if (line.count[b] > 0) keys = min(line.start[b] + line.count[b], p.cache.capacity) - line.from(b);
      rows = line.count[b] * p.G;
    }
    int x = keys > 0 ? Entry(p, rows, key_tiles(keys)).places * p.cache.n_kv : 0;
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

// What the joining kernel asks for, by a warp of every block.
__device__ __forceinline__ void put_plans(const PrefixParams& p, const PrefixLine& line) {
  for (int b = blockIdx.x * 32 + threadIdx.x % 32; b < p.B; b += gridDim.x * 32) {
    const int from = line.from(b), count = line.count[b];
    RowPlan x = {0, 0, 0, 0, 0, 0, count * p.G, 0};
    if (from > 0) {
      const int j = line.group[b];
      x.pre_base = line.prefix[j];
      x.pre_tiles = key_tiles(from);
      x.pre_rows = line.size(j) * p.T * p.G;
      x.pre_row = (b - line.first[j]) * p.T * p.G;
    }
    if (const int keys = min(line.start[b] + count, p.cache.capacity) - from; count > 0 && keys > 0) {
      x.own_base = line.prefix[p.n_groups + b];
      x.own_tiles = key_tiles(keys);
    }
    p.plans[b] = x;
  }
  if (blockIdx.x == 0 && threadIdx.x % 32 == 0) *p.length = all_places(p, line);
}

// ---- shares ------------------------------------------------------------------------------

// A share of the line that lies in one item. Of a prefix b is the group's first
// sequence, whose rows are read, and no key is a node (start = len, no count).
struct PrefixShare {
  int entry = -1;  // of the line
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
    int lo = s.entry;  // the last entry whose prefix is <= u: this one or a later one
    if (lo < 0) {
      int hi = p.n_groups + p.B;
      lo = 0;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (line.prefix[mid] <= u) lo = mid;
        else hi = mid;
      }
    } else {
      while (line.prefix[lo + 1] <= u) ++lo;
    }
    s.entry = lo;
    s.is_prefix = lo < p.n_groups;
    if (s.is_prefix) {
      s.b = line.first[lo];
      s.count = s.first = 0;
      s.start = s.len = line.shared[lo];
      s.rows = line.size(lo) * p.T * p.G;
    } else {
      s.b = lo - p.n_groups;
      s.count = line.count[s.b];
      s.start = line.start[s.b];
      s.first = line.from(s.b);
      s.len = min(s.start + s.count, p.cache.capacity);
      s.rows = s.count * p.G;
    }
    const Entry e(p, s.rows, key_tiles(s.len - s.first));
    const int at = u - line.prefix[lo];
    // floor(at / places), which is below 2^12: the rounded quotient is at most one off
    s.g = (int)__fdividef((float)at, (float)e.places);
    if (s.g * e.places > at) --s.g;
    else if ((s.g + 1) * e.places <= at) ++s.g;
    int rt = 0;
    if (e.row_tiles > 1) {  // (below 2^15)
      const int in = at - s.g * e.places;
      rt = (int)__fdividef((float)in, (float)e.places0);
      if (rt * e.places0 > in) --rt;
      else if ((rt + 1) * e.places0 <= in) ++rt;
      rt = min(rt, e.row_tiles - 1);
    }
    s.row0 = rt << p.row_log2;
    const int cost = e.cost_log2(p, rt), round = (1 << cost) - 1;
    s.nt = e.tiles;
    const int tile0 = line.prefix[lo] + s.g * e.places + rt * e.places0 + p.extra;  // place of the item's tile 0
    // (a tile belongs to the block that has its first place)
    s.k0 = (max(u - tile0, 0) + round) >> cost;
    s.n = min((max(u_end - tile0, 0) + round) >> cost, s.nt) - s.k0;
    s.begins = u == u_begin;
    u = tile0 + (s.nt << cost);
  } while (s.n <= 0);  // a part that has no tile of the item
  return true;
}

__device__ __forceinline__ int first_slot(const PrefixShare& s) { return s.first; }
__device__ __forceinline__ int first_row(const PrefixShare& s) { return s.row0; }
__device__ __forceinline__ bool row_there(const PrefixParams& p, const PrefixLine& line,
                                          const PrefixShare& s, int row) {
  if (row >= s.rows) return false;
  if (!s.is_prefix) return true;
  const int node = div_by(row, p.G, p.inv_G), seq = div_by(node, p.T, p.inv_T);
  return node - seq * p.T < line.count[s.b + seq];
}
// (of a prefix no row has a node among the keys)
__device__ __forceinline__ int row_node(const PrefixParams& p, const PrefixShare& s, int row) {
  return s.is_prefix ? -1 : div_by(row, p.G, p.inv_G);
}
// (rows of a prefix are those of its first sequence and on)
__device__ __forceinline__ int64_t row_offset(const PrefixParams& p, const PrefixShare& s, int row,
                                              int D, int64_t stride) {
  const int node = div_by(row, p.G, p.inv_G);
  return ((int64_t)s.b * p.T + node) * stride + (s.g * p.G + row - node * p.G) * D;
}
__device__ __forceinline__ bool is_final(const PrefixShare& s) {
  return !s.is_prefix && s.first == 0 && s.n == s.nt;
}
// The workspace's row of row `row` of kv-head g, counted from sequence b on, of an uncut item.
__device__ __forceinline__ size_t uncut_slot(const PrefixParams& p, bool is_prefix, int b, int g,
                                             int row) {
  const int node = div_by(row, p.G, p.inv_G);
  const int64_t at = ((int64_t)b * p.T + node) * p.nh + g * p.G + row - node * p.G;
  return p.cut_rows + (is_prefix ? 0 : (int64_t)p.B * p.T * p.nh) + at;
}
__device__ __forceinline__ size_t share_slot(const PrefixParams& p, int group, const PrefixShare& s,
                                             int, int local, int row) {
  if (s.n == s.nt) return uncut_slot(p, s.is_prefix, s.b, s.g, row);
  return part_slot(p, group, s.begins, 0) * p.row_tile + local;
}
// columns c to c + 3 and, behind them, c + 4 to c + 7 of a row of the workspace; `step` vectors on
// the next eight
__device__ __forceinline__ float4* part_place(const PrefixParams& p, size_t slot, int D, int c, int& step) {
  if ((int64_t)slot >= p.cut_rows) {
    step = 2;
    return reinterpret_cast<float4*>(p.part_o + slot * D + c);
  }
  step = 2 * p.row_tile;
  const size_t local = slot & (p.row_tile - 1), tile = slot - local;
  return reinterpret_cast<float4*>(p.part_o + tile * D) + (c / 8) * step + 2 * local;
}

namespace {

// ---- the join ------------------------------------------------------------------------------

// Joins a row's shares, of its group's prefix and of its own keys, a warp to a row
// (FEW: a block's four warps, every fourth share each). The lanes read the shares'
// maxima and sums 32 at a time, so that every share's factor is known before its
// columns are read; the order is fixed. Bound by latency: three reads in a row, each of
// 0.7 to 0.9 us, with the plan first.
template <int D, bool FEW, typename T>
__global__ void __launch_bounds__(128) prefix_attention_join(const __grid_constant__ PrefixParams p) {
  constexpr int E = D / 32, TURNS = FEW ? 4 : 1, U = FEW ? 8 : 4;  // U: loads in flight
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ Vec other[4][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, turn = FEW ? warp : 0;
  const int b = blockIdx.y / p.cache.n_kv, g = blockIdx.y % p.cache.n_kv;
  const int row = FEW ? blockIdx.x : blockIdx.x * 4 + warp;
  griddep_wait();
  const int4* at_plan = reinterpret_cast<const int4*>(p.plans + b);
  const int4 plan[2] = {__ldcg(at_plan), __ldcg(at_plan + 1)};
  const Cut cut(__ldcg(p.length), p);
  // Of both items: the place of its tile 0, its tiles, their cost, the blocks that may have a part
  // of it (n of them from g0 on), the row's number in its row tile.
  int tile0[2], nt[2], cost[2], g0[2], n[2] = {0, 0}, local[2];
  if (row < plan[1].z) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      nt[which] = plan[which].y;
      if (nt[which] == 0) continue;
      const Entry e(p, plan[which].z, nt[which]);
      const int r = which ? row : plan[0].w + row, rt = r >> p.row_log2;
      local[which] = r - (rt << p.row_log2);
      cost[which] = e.cost_log2(p, rt);
      tile0[which] = plan[which].x + g * e.places + rt * e.places0 + p.extra;
      g0[which] = cut.group_of(tile0[which]);
      n[which] = cut.group_of(tile0[which] + ((nt[which] - 1) << cost[which])) - g0[which] + 1;
    }
  }
  const int all = n[0] + n[1];
  const bool joins = all > 1 || n[0] == 1;  // else it was written whole
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (joins) {
    // lane i: where share s0 + i keeps the row's first columns (a vector of part_o, fewer than
    // 2^32 of them; kNoRow: no share, or no key seen in it), its maximum and sum
    uint32_t at;
    float ms, ls;
    auto look = [&](int s0) {
      const int s = s0 + lane;
      at = kNoRow, ms = -INFINITY, ls = 0.f;
      if (s < all) {
        const int which = s < n[0] ? 0 : 1;
        const int group = (which ? g0[1] - n[0] : g0[0]) + s;
        int64_t x;
        if ((which ? n[1] : n[0]) == 1) {
          x = (int64_t)uncut_slot(p, which == 0, b, g, row);
        } else {
          // (a block between may have no tile's first place)
          const int t0 = which ? tile0[1] : tile0[0], c = which ? cost[1] : cost[0];
          const int u0 = cut.begin(group), round = (1 << c) - 1;
          if ((max(u0 - t0, 0) + round) >> c >= min((max(cut.begin(group + 1) - t0, 0) + round) >> c, which ? nt[1] : nt[0]))
            return;
          x = (int64_t)part_slot(p, group, u0 >= t0 - p.extra, 0) * p.row_tile + (which ? local[1] : local[0]);
        }
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + x);
        int step;
        const float4* place = part_place(p, (size_t)x, D, 0, step);
        if (ml.y != 0.f) at = (uint32_t)(place - reinterpret_cast<const float4*>(p.part_o)), ms = ml.x, ls = ml.y;
      }
    };
    // the lane's columns of a share whose next eight columns are `step` vectors on
    const int step0 = n[0] == 1 ? 2 : 2 * p.row_tile, step1 = n[1] == 1 ? 2 : 2 * p.row_tile;
    const Vec* base = reinterpret_cast<const Vec*>(p.part_o) + lane % (8 / E);
    const int near0 = lane / (8 / E) * step0, near1 = lane / (8 / E) * step1;
    float m = -INFINITY;
    for (int s0 = 0; s0 < all; s0 += 32) {
      look(s0);
      m = fmaxf(m, ms);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int s0 = 0; s0 < all; s0 += 32) {
      if (all > 32) look(s0);  // else the lanes still have it
      const float f = at == kNoRow ? 0.f : fast_exp2(ms - m);
      l += ls * f;
      const int here = min(32, all - s0);
      for (int k0 = turn; k0 < here; k0 += U * TURNS) {
        Vec v[U];
        float w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int k = k0 + i * TURNS;
          const uint32_t x = __shfl_sync(0xffffffffu, at, k & 31);
          w[i] = __shfl_sync(0xffffffffu, f, k & 31);
          v[i] = Vec{};
          if (k < here && x != kNoRow) v[i] = __ldcg(base + (size_t)(x + (s0 + k < n[0] ? near0 : near1)) * (4 / E));
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
  size_t runs;             // float4
  size_t sums(int D) const { return ((size_t)rows * (D + 2) * sizeof(float) + 31) / 32 * 32; }
  size_t bytes(int D, int B) const {
    return sums(D) + runs * sizeof(float4) + (size_t)B * sizeof(RowPlan) + sizeof(int);
  }
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
  if (tiles * cache->n_kv_heads * (view->capacity / kKeys + 8) * 2 > INT32_MAX)
    return op_fail(MK_ERR_INVALID, "batch x n_tokens x n_heads x capacity: more than 2^31 tiles");
  return MK_OK;
}

int make_plan(const CacheView& cache, int D, int B, int T, int nh, int type, int n_groups,
              PrefixPlan* pl) {
  int device = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return op_cuda(e, kName);
  pl->row_tile = row_tile_of(B, T, nh / cache.n_kv, type, n_groups);
  pl->groups = n_sm;
  pl->cut_rows = (int64_t)2 * pl->groups * pl->row_tile;
  pl->rows = pl->cut_rows + 2 * (int64_t)B * T * nh;
  pl->runs = run_vectors(type, pl->row_tile, ((int64_t)cache.capacity + kKeys - 1) / kKeys, pl->groups, D);
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
  if (int rc = make_plan(view, cache->head_dim, batch, n_tokens, n_heads, type, n_groups, &pl)) return rc;
  *bytes = pl.bytes(cache->head_dim, batch);
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
  if (int rc = make_plan(p.cache, cache->head_dim, batch, n_tokens, n_heads, type, n_groups, &pl)) return rc;
  if (workspace_bytes < pl.bytes(cache->head_dim, batch))
    return op_fail(MK_ERR_INVALID, "workspace: smaller than its query says");
  p.k = (const uint16_t*)cache->k[layer];
  p.v = (const uint16_t*)cache->v[layer];
  p.q = q, p.out = out, p.qs = q_stride, p.os = out_stride;
  p.starts = starts, p.parents = parents, p.counts = counts;
  p.B = batch, p.T = n_tokens, p.nh = n_heads, p.G = n_heads / cache->n_kv_heads;
  p.tile_log2 = 7;
  // What an item's beginning and end are worth, in tiles (32 samples behind 8192 keys, bf16, one
  // block of rows: 2, 3, 4, 5 39.3, 37.4, 38.4, 40.6 us; 64 samples of two prompts of up to 32768
  // keys, two blocks: 4, 5, 6, 7, 8 236, 224, 221, 223, 225; 24 samples in fp32: 2, 3, 4 50.8, 53.7, 55.6)
  p.extra = type == MK_TYPE_FP32 ? 2 : pl.row_tile > 128 ? 6 : 3;
  p.row_tile = pl.row_tile, p.row_tiles = 1,
  p.row_log2 = pl.row_tile == 32 ? 5 : pl.row_tile == 128 ? 7 : 8, p.groups = pl.groups;
  p.inv_groups = (uint32_t)std::min<uint64_t>((1ull << 32) / pl.groups + 1, UINT32_MAX);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.n_groups = n_groups, p.first = first, p.shared = prefix;
  p.cut_rows = pl.cut_rows;
  p.part_o = (float*)workspace;
  p.part_ml = p.part_o + (size_t)pl.rows * cache->head_dim;
  float4* runs = (float4*)((uint8_t*)workspace + pl.sums(cache->head_dim));
  p.runs = pl.runs ? runs : nullptr;
  p.plans = (RowPlan*)(runs + pl.runs);
  p.length = (int*)(p.plans + batch);
  auto inverse = [](int d) { return (uint32_t)std::min<uint64_t>((1ull << 32) / d + 1, UINT32_MAX); };
  p.inv_G = inverse(p.G), p.inv_T = inverse(p.T);
  cudaStream_t st = (cudaStream_t)stream;
  if (int rc = launch_tc(p, p.groups, cache->head_dim, type, kName, st)) return rc;
  return cache->head_dim == 64 ? launch_join<64>(p, type, st) : launch_join<128>(p, type, st);
}

}  // extern "C"
