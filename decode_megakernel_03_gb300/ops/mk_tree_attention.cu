// Attention of a tree of drafted tokens over a KV cache (include/mk.h,
// mk_tree_attention): the entry point, the kernel for few rows (warp-level
// products) and the kernel that joins shares. The one for many rows is in
// mk_tree_attention_tc.cu.
#include <algorithm>
#include <type_traits>

#include "mk_tree_attention.cuh"

namespace mk {
namespace {

constexpr int kStages = 3;       // tiles in shared memory
constexpr int kThreads = 128;    // four warps, each a quarter of a tile's keys
constexpr int kRows = 16;        // rows of a row tile
constexpr int kCtasPerSm = 2;
constexpr int kMaxG = 8;

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// ---- the kernel ------------------------------------------------------------------------
// One m16 block of rows. P = 1: bf16 activations; P = 3: fp32 ones, queries and
// weights as three bf16 parts (2^-24 of the value: fp32's own step; the cache is
// bf16, so products of parts are exact). Weights of bf16 calls are two bf16 parts
// (2^-17, as the decode step holds its own); sums, maxima and the output accumulate
// in fp32. A tile is 16 KB of keys and 16 KB of values whatever the head's size: 64-key tiles of 64 dimensions spent their time on the
// barriers between them. Three tiles per block and two blocks per SM keep 192 KB
// per SM in flight. Bound by the bytes of the keys and values: a single bf16 token of
// 8 sequences over 16384 keys each (8B shape, 537 MB) takes 89 us, 6.0 TB/s; fp32 in
// heads of 64 (1B shape, 268 MB) 70 us, bound by its six products and the
// splitting. Short contexts are bound by
// latency: 512 keys of one sequence 9.2 us, two launches of which the second
// waits for the first inside.
constexpr int tile_keys(int D) { return 8192 / D; }
// How the weights times the values are added up, as the matrix unit truncates when it
// accumulates (kRun): in heads of 64 and in fp32 by rounded adds of each product; in bf16 heads of
// 128 in the unit, and the sums of so many tiles to the workspace (a warp takes a quarter of a
// tile's keys, so that these are as many products as a run of the other kernel). 8 tokens over
// 16384 keys each, 8B shape: 84.1 us with runs, 83.9 without, 90.3 with rounded adds, which spill
// there; 4 tokens over 131072 keys, 1B shape: 160.9 with rounded adds, 159.3 without, 166.6 with runs.
constexpr int run_tiles(int D) { return 4 * kRun * 128 / tile_keys(D); }

template <int D, int P>
struct Layout {
  static constexpr int kTile = tile_keys(D), kRunTiles = run_tiles(D);
  static constexpr bool kRuns = P == 1 && D == 128;
  static constexpr int kStageBytes = 2 * kTile * D * 2;
  static constexpr int kRing = kStages * kStageBytes;
  // joined warps: o [4][kRows][D] fp32 over the ring
  static_assert(4 * kRows * D * 4 <= kRing, "the warps' shares fit the ring");
  static constexpr int kRowTab = (kStages + 1) * kTile * 4;
  static constexpr int kBytes = kRing + kRowTab;
};

template <int D, int P>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
tree_attention_kernel(const __grid_constant__ AttnParams p) {
  using Lay = Layout<D, P>;
  constexpr int kTile = Lay::kTile, RT = kRows, KB = D / 16, NB = D / 8;
  constexpr int W = P == 1 ? 2 : P;  // parts of the weights
  constexpr int NK = kTile / 64;  // blocks of 16 keys that a warp takes of a tile
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* rowtab = reinterpret_cast<uint32_t*>(smem + Lay::kRing);  // [kStages + 1][kTile]
  __shared__ Line line;
  __shared__ uint64_t s_seen[MK_MAX_TREE];   // node -> the nodes it sees
  __shared__ int s_up[MK_MAX_TREE];
  // non-finite values of the nodes' v rows: bit d % 32 of word d / 32, +inf in
  // [0], -inf in [1], NaN in both
  __shared__ uint32_t s_odd[MK_MAX_TREE][2][D / 32];
  __shared__ float s_ml[4][RT][2];
  __shared__ float s_run[kThreads][2];  // the reference of the thread's earlier runs
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int grp = lane / 4, tig = lane % 4;
  const int rt = blockIdx.x % p.row_tiles, group = blockIdx.x / p.row_tiles;
  const uint32_t ring = smem_u32(smem);

  griddep_launch();
  if (warp == 0) work_line(p, line);
  __syncthreads();
  const Cut cut(line.prefix[p.B], p);
  const int u_begin = cut.begin(group), u_end = cut.begin(group + 1);
  int u = u_begin;

  Share sh;
  while (next_share(p, line, u_begin, u_end, u, sh)) {
    const int b = sh.b, g = sh.g, k0 = sh.k0, n = sh.n;
    const int count = sh.count, start = sh.start, len = sh.len, rows = sh.rows;
    if (rt * RT >= rows) continue;  // no row of this tile is there

    // ---- key rows of tile `it` of the share into rowtab, its copies
    auto row_of = [&](int it) -> uint32_t {  // threads 0..kTile-1
      const int slot = (k0 + it) * kTile + tid;
      if (it >= n || slot >= len) return kNoRow;
      const uint32_t r = cache_row(p.cache, b, slot);
      return r == kNoRow ? r : r + (uint32_t)g * p.cache.block_size;
    };
    auto fetch = [&](int it) {
      if (it < n) {
        constexpr int CPR = D / 8, RPP = kThreads / CPR;
        const uint32_t* tab = rowtab + it % (kStages + 1) * kTile;
        const uint32_t base = ring + it % kStages * Lay::kStageBytes;
        const int c = tid % CPR;
#pragma unroll
        for (int i = 0; i < kTile / RPP; ++i) {
          const int r = tid / CPR + i * RPP;
          const uint32_t row = tab[r];
          const uint32_t bytes = row == kNoRow ? 0 : 16;
          const size_t off = row == kNoRow ? 0 : (size_t)row * D + 8 * c;
          const uint32_t dst = base + r * (D * 2) + ((c ^ (r & 7)) * 16);
          cp_async16(dst, p.k + off, bytes);
          cp_async16(dst + kTile * D * 2, p.v + off, bytes);
        }
      }
      cp_async_commit();
    };

    __syncthreads();  // the share before this one is done with shared memory
    if (tid < kTile) {
#pragma unroll
      for (int it = 0; it < kStages; ++it) rowtab[it * kTile + tid] = row_of(it);
    }
    if (tid < MK_MAX_TREE) {
      // The nodes each node sees, by doubling: seen covers the nearest 2^i
      // ancestors, up is the next one behind them.
      int up = -1;
      if (tid < count) {
        up = p.parents ? __ldg(p.parents + (size_t)b * p.T + tid) : tid - 1;
        if (up < 0 || up >= tid) up = -1;
      }
      s_up[tid] = up;
      s_seen[tid] = 1ull << tid;
      for (int w = 0; w < 2 * (D / 32); ++w) (&s_odd[tid][0][0])[w] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < kStages - 1; ++it) fetch(it);
    // ---- the rows' queries as A fragments, and what the rows see
    uint4 qf[P][KB];
    {
      const void* src[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = rt * RT + h * 8 + grp;
        const int64_t off = row_offset(p, b, g, r, D, p.qs);
        src[h] = r >= rows ? nullptr
                 : P > 1    ? (const void*)((const float*)p.q + off)
                           : (const void*)((const uint16_t*)p.q + off);
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        uint32_t w[P][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (grp, 2tig), (grp + 8, 2tig), (grp, 2tig + 8), (grp + 8, 2tig + 8)
          const int c = kb * 16 + 2 * tig + (j / 2) * 8;
          const void* s = src[j % 2];
          if constexpr (P > 1) {
            const float2 x = s ? __ldg((const float2*)((const float*)s + c)) : make_float2(0.f, 0.f);
            uint32_t part[P];
            split(x.x, x.y, part);
#pragma unroll
            for (int q = 0; q < P; ++q) w[q][j] = part[q];
          } else {
            w[0][j] = s ? __ldg((const uint32_t*)((const uint16_t*)s + c)) : 0u;
          }
        }
#pragma unroll
        for (int q = 0; q < P; ++q) qf[q][kb] = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
      }
    }
    for (int i = 1; i < count; i *= 2) {
      uint64_t seen = 0;
      int up = -1;
      if (tid < MK_MAX_TREE) {
        up = s_up[tid];
        seen = s_seen[tid];
        if (up >= 0) {
          seen |= s_seen[up];
          up = s_up[up];
        }
      }
      __syncthreads();
      if (tid < MK_MAX_TREE) {
        s_up[tid] = up;
        s_seen[tid] = seen;
      }
      __syncthreads();
    }

    uint64_t seen[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = rt * RT + h * 8 + grp;
      seen[h] = r < rows ? s_seen[r / p.G] : 0;
    }

    float o[NB][4], mx[2], sum[2];
#pragma unroll
    for (int d = 0; d < NB; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    mx[0] = mx[1] = -INFINITY;
    sum[0] = sum[1] = 0.f;

    // adds the sums of the runs before this one (some) to o
    auto add_runs = [&](const float4* runs) {
      float back[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float from = s_run[tid][h];
        back[h] = from == mx[h] ? 1.f : fast_exp2(from - mx[h]);
      }
#pragma unroll
      for (int d = 0; d < NB; ++d) {
        const float4 x = runs[d * kThreads];
        o[d][0] = fmaf(x.x, back[0], o[d][0]), o[d][1] = fmaf(x.y, back[0], o[d][1]);
        o[d][2] = fmaf(x.z, back[1], o[d][2]), o[d][3] = fmaf(x.w, back[1], o[d][3]);
      }
    };
    float4* runs = p.runs + (size_t)blockIdx.x * NB * kThreads + tid;

    // ---- the tiles
    for (int it = 0; it < n; ++it) {
      if (Lay::kRuns && it % Lay::kRunTiles == 0 && it > 0) {  // a run ends
        if (it > Lay::kRunTiles) add_runs(runs);
#pragma unroll
        for (int d = 0; d < NB; ++d) {
          runs[d * kThreads] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
          o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
        }
        s_run[tid][0] = mx[0], s_run[tid][1] = mx[1];
      }
      cp_async_wait<kStages - 2>();
      __syncthreads();  // tile `it` is there; everybody is done with tile it - 1
      fetch(it + kStages - 1);
      uint32_t next_row = kNoRow;
      if (tid < kTile) next_row = row_of(it + kStages);
      const uint32_t ks = ring + it % kStages * Lay::kStageBytes, vs = ks + kTile * D * 2;
      const uint32_t* tab = rowtab + it % (kStages + 1) * kTile;
      const int slot0 = (k0 + it) * kTile;

      bool odd = false;  // the tile holds a node with a non-finite v value
      if (slot0 + kTile > start) {
        // nodes of the tile: a value that some rows must not see cannot be
        // cancelled by a zero weight if it is not finite, so it is taken out
        // here and added to the rows that see it
        constexpr int CPR = D / 8;
        bool bad = false;
        for (int i = tid; i < kTile * CPR; i += kThreads) {
          const int r = i / CPR, c = i % CPR, node = slot0 + r - start;
          if (node < 0 || node >= count || tab[r] == kNoRow) continue;
          uint8_t* at = smem + (vs - ring) + r * (D * 2) + ((c ^ (r & 7)) * 16);
          uint16_t* x = reinterpret_cast<uint16_t*>(at);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint16_t v = x[e];
            if ((v & 0x7f80) == 0x7f80) {
              const int d = c * 8 + e;
              const bool nan = v & 0x7f;
              if (nan || !(v & 0x8000)) atomicOr(&s_odd[node][0][d / 32], 1u << (d % 32));
              if (nan || (v & 0x8000)) atomicOr(&s_odd[node][1][d / 32], 1u << (d % 32));
              x[e] = 0;
              bad = true;
            }
          }
        }
        odd = __syncthreads_or(bad);
      }

      // scores of the warp's keys
      float s[NK][2][4];
#pragma unroll
      for (int nk = 0; nk < NK; ++nk)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nk][j][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int nk = 0; nk < NK; ++nk) {
          // blocks: keys 0-7 dims 0-7, keys 0-7 dims 8-15, keys 8-15 dims 0-7, ...
          const int r = (warp * NK + nk) * 16 + (lane / 16) * 8 + lane % 8, c = kb * 2 + (lane / 8) % 2;
          uint32_t kf[4];
          ldsm_x4(kf, ks + r * (D * 2) + ((c ^ (r & 7)) * 16));
          if constexpr (P == 1) {
            mma_bf16_16816(s[nk][0], qf[0][kb], kf[0], kf[1]);
            mma_bf16_16816(s[nk][1], qf[0][kb], kf[2], kf[3]);
          } else {
            // the matrix unit may truncate as it accumulates: the smallest parts
            // first, and the sums over the dimensions by rounded adds
            float x[2][4] = {};
#pragma unroll
            for (int q = P - 1; q >= 0; --q) {
              mma_bf16_16816(x[0], qf[q][kb], kf[0], kf[1]);
              mma_bf16_16816(x[1], qf[q][kb], kf[2], kf[3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nk][0][e] += x[0][e], s[nk][1][e] += x[1][e];
          }
        }
      // what is not seen: keys behind the length, pages that are not there,
      // nodes that are no ancestors
      const uint32_t mine = lane < 16 * NK ? tab[warp * 16 * NK + lane] : 0;
      const bool plain = slot0 + kTile <= start && !__any_sync(0xffffffffu, mine == kNoRow);
#pragma unroll
      for (int nk = 0; nk < NK; ++nk)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nk][j][e] *= p.scale_log2;
            if (!plain) {
              const int key = (warp * NK + nk) * 16 + j * 8 + 2 * tig + (e & 1);
              const int node = slot0 + key - start;
              const bool see = tab[key] != kNoRow && (node < 0 || (seen[e / 2] >> node & 1));
              if (!see) s[nk][j][e] = -INFINITY;
            }
          }

      // running maximum and sum
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float t = -INFINITY;
#pragma unroll
        for (int nk = 0; nk < NK; ++nk)
          t = fmaxf(t, fmaxf(fmaxf(s[nk][0][2 * h], s[nk][0][2 * h + 1]),
                             fmaxf(s[nk][1][2 * h], s[nk][1][2 * h + 1])));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        const float now = fmaxf(mx[h], t);
        const float from = now == -INFINITY ? 0.f : now;  // nothing seen yet: weights 0
        const float keep = fast_exp2(mx[h] - from);
        mx[h] = now;
        float add = 0.f;
#pragma unroll
        for (int nk = 0; nk < NK; ++nk)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w = fast_exp2(s[nk][j][2 * h + e] - from);
              s[nk][j][2 * h + e] = w;
              add += w;
            }
        sum[h] = sum[h] * keep + add;
        if (__any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll
          for (int d = 0; d < NB; ++d) {
            o[d][2 * h] *= keep;
            o[d][2 * h + 1] *= keep;
          }
        }
      }

      // o += weights x v
#pragma unroll
      for (int nk = 0; nk < NK; ++nk) {
        uint4 w[W];
        uint32_t part[4][W];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          split(s[nk][j / 2][j % 2 * 2], s[nk][j / 2][j % 2 * 2 + 1], part[j]);
#pragma unroll
        for (int q = 0; q < W; ++q) w[q] = make_uint4(part[0][q], part[1][q], part[2][q], part[3][q]);
#pragma unroll
        for (int d = 0; d < NB; d += 2) {
          const int r = (warp * NK + nk) * 16 + (lane / 8) % 2 * 8 + lane % 8, c = d + lane / 16;
          uint32_t vf[4];
          ldsm_x4_t(vf, vs + r * (D * 2) + ((c ^ (r & 7)) * 16));
          if constexpr (Lay::kRuns) {
#pragma unroll
            for (int q = W - 1; q >= 0; --q) {
              mma_bf16_16816(o[d], w[q], vf[0], vf[1]);
              mma_bf16_16816(o[d + 1], w[q], vf[2], vf[3]);
            }
          } else {
            float x[2][4] = {};
#pragma unroll
            for (int q = W - 1; q >= 0; --q) {
              mma_bf16_16816(x[0], w[q], vf[0], vf[1]);
              mma_bf16_16816(x[1], w[q], vf[2], vf[3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] += x[0][e], o[d + 1][e] += x[1][e];
          }
        }
      }
      if (odd) {
#pragma unroll 1
        for (int key = warp * 16 * NK; key < (warp + 1) * 16 * NK; ++key) {
          const int node = slot0 + key - start;
          if (node < 0 || node >= count || tab[key] == kNoRow) continue;
#pragma unroll
          for (int d = 0; d < NB; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = d * 8 + 2 * tig + (e & 1);
              if (!(seen[e / 2] >> node & 1)) continue;
              if (s_odd[node][0][c / 32] >> (c % 32) & 1) o[d][e] += INFINITY;
              if (s_odd[node][1][c / 32] >> (c % 32) & 1) o[d][e] -= INFINITY;
            }
        }
      }
      if (tid < kTile) rowtab[(it + kStages) % (kStages + 1) * kTile + tid] = next_row;
    }

    if (Lay::kRuns && n > Lay::kRunTiles) add_runs(runs);

    // ---- the warps' shares joined: sums within a quad, maxima across warps
    cp_async_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
      if (tig == 0) {
        s_ml[warp][h * 8 + grp][0] = mx[h];
        s_ml[warp][h * 8 + grp][1] = sum[h];
      }
    }
    __syncthreads();  // also: everybody is done with the ring
    float* so = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = h * 8 + grp;
      const float top = fmaxf(fmaxf(s_ml[0][r][0], s_ml[1][r][0]), fmaxf(s_ml[2][r][0], s_ml[3][r][0]));
      const float f = fast_exp2(mx[h] - top);
      const bool none = sum[h] == 0.f;  // a seen key's largest weight is 1 (or NaN)
#pragma unroll
      for (int d = 0; d < NB; ++d)
        *reinterpret_cast<float2*>(so + (warp * RT + r) * D + d * 8 + 2 * tig) =
            none ? make_float2(0.f, 0.f) : make_float2(o[d][2 * h] * f, o[d][2 * h + 1] * f);
    }
    __syncthreads();
    const bool whole = n == sh.nt;
    const size_t slot = part_slot(p, group, sh.begins, rt);
    for (int i = tid; i < RT * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4, row = rt * RT + r;
      if (row >= rows) break;
      const float top = fmaxf(fmaxf(s_ml[0][r][0], s_ml[1][r][0]), fmaxf(s_ml[2][r][0], s_ml[3][r][0]));
      float l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w4 = 0; w4 < 4; ++w4) {
        if (s_ml[w4][r][1] != 0.f) l += s_ml[w4][r][1] * fast_exp2(s_ml[w4][r][0] - top);
        const float4 x = *reinterpret_cast<const float4*>(so + (w4 * RT + r) * D + c);
        a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
      }
      if (whole) {
        const float f = l == 0.f ? 0.f : 1.f / l;  // no key seen: 0
        if (l == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);
        a.x *= f, a.y *= f, a.z *= f, a.w *= f;
        const int64_t off = row_offset(p, b, g, row, D, p.os) + c;
        if constexpr (P > 1)
          *reinterpret_cast<float4*>((float*)p.out + off) = a;
        else
          *reinterpret_cast<uint2*>((uint16_t*)p.out + off) =
              make_uint2(bf16x2_rn(a.x, a.y), bf16x2_rn(a.z, a.w));
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot * RT + r) * D + c) = a;
        if (c == 0) {
          p.part_ml[(slot * RT + r) * 2] = top;
          p.part_ml[(slot * RT + r) * 2 + 1] = l;
        }
      }
    }
  }
}

// Joins the shares of the items that were cut. Few rows: the four warps of a block
// take one row, every fourth share each, and add up in shared memory in a
// fixed order. Many: a warp takes a row (four one after another took 6 us longer
// on 6400 rows). A lane has D / 32 of the row's columns; the lanes read the
// shares' maxima and sums 32 at a time, so that every share's factor is known
// before its columns are read. Bound by latency: it starts while the other kernel
// runs, has its line of work by the time that ends, and then reads twice in a row
// (the factors, the columns), about 4 us.
template <int D, bool FEW, typename T>
__global__ void __launch_bounds__(128) tree_attention_join(const __grid_constant__ AttnParams p) {
  constexpr int E = D / 32, TURNS = FEW ? 4 : 1, U = FEW ? 8 : 2;  // U: loads in flight
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ Line line;
  __shared__ Vec other[4][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, turn = FEW ? warp : 0;
  const int b = blockIdx.y / p.cache.n_kv, g = blockIdx.y % p.cache.n_kv;
  if (warp == 0) work_line(p, line);
  __syncthreads();
  const int row = FEW ? blockIdx.x : blockIdx.x * 4 + warp;
  const int places = line.prefix[b + 1] == line.prefix[b] ? 0 : places_of(p, min(line.start[b] + line.count[b], p.cache.capacity));
  const int rt = row / p.row_tile, r = row - rt * p.row_tile;
  bool cut_up = places > 0 && row < line.count[b] * p.G;
  int g0 = 0, g1 = 0, item0 = 0;
  const Cut cut(line.prefix[p.B], p);
  if (cut_up) {
    item0 = line.prefix[b] + g * places;
    g0 = cut.group_of(item0 + p.extra);
    g1 = cut.group_of(item0 + places - 1);
    cut_up = g0 != g1;  // else it was written whole
  }
  griddep_wait();
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  if (cut_up) {
    // lane i: where share s0 + i keeps the row (-1: no share, or no key seen in
    // it), its maximum and sum
    int64_t at;
    float ms, ls;
    auto look = [&](int s0) {
      const int s = s0 + lane;
      at = -1, ms = -INFINITY, ls = 0.f;
      if (s <= g1) {
        const int u0 = cut.begin(s);
        if (u0 != cut.begin(s + 1)) {  // not one of more groups than places
          const int64_t x = (int64_t)part_slot(p, s, u0 >= item0, rt) * p.row_tile + r;
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + x);
          if (ml.y != 0.f) at = x, ms = ml.x, ls = ml.y;
        }
      }
    };
    float m = -INFINITY;
    for (int s0 = g0; s0 <= g1; s0 += 32) {
      look(s0);
      m = fmaxf(m, ms);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int s0 = g0; s0 <= g1; s0 += 32) {
      if (g1 - g0 >= 32) look(s0);  // else the lanes still have it
      const float f = at < 0 ? 0.f : fast_exp2(ms - m);
      l += ls * f;
      const int n = min(32, g1 - s0 + 1);
      for (int k0 = turn; k0 < n; k0 += U * TURNS) {
        Vec v[U];
        float w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int k = k0 + i * TURNS;
          const int64_t x = __shfl_sync(0xffffffffu, at, k & 31);
          w[i] = __shfl_sync(0xffffffffu, f, k & 31);
          v[i] = Vec{};
          if (k < n && x >= 0) v[i] = __ldcg(reinterpret_cast<const Vec*>(p.part_o + x * D) + lane);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float* c = reinterpret_cast<const float*>(&v[i]);
          const bool has = k0 + i * TURNS < n;
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
  if (!cut_up) return;
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

struct Plan {
  bool tc;  // the kernel for many rows
  int tile, extra, row_tile, row_tiles, groups;
  size_t o_floats, ml_floats, runs;  // runs: float4
  size_t bytes() const { return (o_floats + ml_floats) * sizeof(float) + runs * sizeof(float4); }
};

// Which kernel, and its tiles. Up to 16 rows go to the warp-level kernel, whose
// products are that size, but for fp32 with heads of 128, whose six products are
// too much for it; the others to the tensor-memory kernel: bf16 activations in two
// streams of up to 128 rows each (up to 128 rows: two streams over the same rows
// that take turns at the key tiles), fp32 ones in tiles of 128 rows, or, up to 32
// rows, with the parts of the weights stacked.
// Warp-level against tensor-memory kernel, us:
//   8 sequences over 16384 keys, 8B shape, bf16   4 nodes (16 rows)  93.2    93.4
//                                                 5 nodes (20 rows) 159.6    92.7
//                                          fp32   1 node            129.9   103.3
//                                                 4 nodes           136.9   107.6
//                                1B shape, fp32   4 nodes            70.8    82.0
//   8 sequences over 1024 keys,  8B shape, fp32   1 node             22.0    23.9
//                                                 4 nodes            26.3    26.8
//   one sequence over 1024 keys, 8B shape, bf16   1 node             10.6    12.7
//                                                 5 nodes            13.7    13.6
//   4 sequences over 4096 keys,  1B shape, fp32   4 nodes            18.9    21.9
// fp32 parts stacked against one after another (8 sequences over 16384 keys, 8 nodes): 8B
// shape 111 us against 129, 1B shape 84 against 94.
// Two blocks of up to 128 rows in a pass over the keys against a pass for each (bf16,
// 8 sequences, 8B shape), 132 / 256 rows: over 16384 keys 154 / 168 us against 165 /
// 170, over 32768 285 / 315 against 308 / 325, over 4096 59 / 68 against 62 / 65; the
// lengths are not known here, and one sequence over 2048 keys, where the second
// block's share only adds to the first's, takes 27 / 30 us against 23 / 24.
Plan plan_of(const CacheView& cache, int B, int T, int G, int D, int type, int n_sm) {
  Plan pl;
  const int rows = T * G;
  pl.tc = rows > kRows || (type == MK_TYPE_FP32 && D == 128);
  // measured at 0, 2, 4 and 8: 25 nodes over 128 to 4096 keys (1B shape, 8 sequences)
  // 32.4, 24.1, 22.9, 24.0 us; 6 fp32 nodes over 2048 to 16384 keys (8B shape, 4
  // sequences) 51.3, 49.5, 46.6, 45.4; one token of 64 sequences over 1024 keys (1B
  // shape) 39.6, 40.4, 42.5, 43.4; one sequence over 4096 keys alike within 5 %
  pl.extra = 4;
  if (pl.tc && type == MK_TYPE_FP32) {
    pl.tile = 128;
    pl.row_tile = rows <= 32 ? 32 : 128;
    pl.row_tiles = (rows + 127) / 128;
    pl.groups = std::max(1, n_sm / pl.row_tiles);
  } else if (pl.tc) {
    pl.tile = 128;
    pl.row_tiles = (rows + 255) / 256;
    const int each = (rows + pl.row_tiles - 1) / pl.row_tiles;
    pl.row_tile = each <= 128 ? 128 : (each + 63) / 64 * 64;
    pl.groups = std::max(1, n_sm / pl.row_tiles);
  } else {
    pl.tile = tile_keys(D);
    pl.row_tile = kRows;
    pl.row_tiles = (rows + pl.row_tile - 1) / pl.row_tile;
    pl.groups = std::max(1, kCtasPerSm * n_sm / pl.row_tiles);
  }
  const size_t slots = (size_t)pl.groups * 2 * pl.row_tiles * pl.row_tile;
  pl.o_floats = slots * D;
  pl.ml_floats = slots * 2;
  // a share has no more tiles than a context, or than a block's part of the longest line
  const int64_t tiles = ((int64_t)cache.capacity + pl.tile - 1) / pl.tile, line = (int64_t)B * cache.n_kv * (tiles + pl.extra);
  const int64_t most = std::min(tiles, line / pl.groups + 1);
  if (pl.tc) pl.runs = run_vectors(type, pl.row_tile, most, pl.groups * pl.row_tiles, D);
  else pl.runs = D == 128 && most > run_tiles(D) ? (size_t)pl.groups * pl.row_tiles * (D / 8) * kThreads : 0;
  return pl;
}

int check_attention(const mk_cache* cache, int batch, int n_tokens, int n_heads, int type,
                    CacheView* view) {
  if (int rc = check_cache(cache, batch, true, view)) return rc;
  if (n_tokens < 1 || n_tokens > MK_MAX_TREE)
    return op_fail(MK_ERR_INVALID, "n_tokens must be 1 to MK_MAX_TREE");
  if (type != MK_TYPE_BF16 && type != MK_TYPE_FP32)
    return op_fail(MK_ERR_INVALID, "type must be MK_TYPE_BF16 or MK_TYPE_FP32");
  if (cache->n_kv_heads > 4096 || (int64_t)batch * cache->n_kv_heads > 65535)
    return op_fail(MK_ERR_INVALID, "batch x n_kv_heads must be at most 65535");
  if (n_heads < 1 || n_heads % cache->n_kv_heads || n_heads / cache->n_kv_heads > kMaxG)
    return op_fail(MK_ERR_INVALID,
                   "n_heads must be a multiple of n_kv_heads, at most 8 heads per kv-head");
  if ((int64_t)batch * cache->n_kv_heads * (view->capacity / 64 + 8) > INT32_MAX)
    return op_fail(MK_ERR_INVALID, "batch x n_kv_heads x capacity above 2^37");
  return MK_OK;
}

int make_plan(const CacheView& view, int D, int batch, int n_tokens, int n_heads, int type, Plan* pl) {
  int device = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return op_cuda(e, "mk_tree_attention");
  *pl = plan_of(view, batch, n_tokens, n_heads / view.n_kv, D, type, n_sm);
  return MK_OK;
}

template <int D, int P>
int launch(const AttnParams& p, cudaStream_t st) {
  using Lay = Layout<D, P>;
  auto* fn = tree_attention_kernel<D, P>;
  static std::atomic<uint64_t> ready{0};
  if (int rc = allow_shared(ready, (const void*)fn, Lay::kBytes, "mk_tree_attention")) return rc;
  fn<<<p.groups * p.row_tiles, kThreads, Lay::kBytes, st>>>(p);
  return op_cuda(cudaGetLastError(), "mk_tree_attention");
}

template <int D>
int launch_all(const AttnParams& p, const Plan& pl, int type, cudaStream_t st) {
  int rc;
  if (pl.tc) rc = launch_tree_attention_tc(p, D, type, st);
  else if (D == 64 && type == MK_TYPE_FP32) rc = launch<64, 3>(p, st);
  else rc = launch<D, 1>(p, st);
  if (rc) return rc;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // A block for a row where that still leaves few blocks per SM (1B shape over
  // 4096 keys, rows of all kv-heads: 32 rows 13.3 us against 20.3, 512 13.8 against
  // 18.3, 1024 15.6 against 20.0; 2048 21.7 against 22.8, but 4096 29.7 against 23.8)
  const bool few = (int64_t)p.T * p.G * p.B * p.cache.n_kv <= 1024;
  cfg.gridDim = dim3(few ? p.T * p.G : (p.T * p.G + 3) / 4, p.B * p.cache.n_kv);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto* fn = type == MK_TYPE_FP32
                 ? (few ? tree_attention_join<D, true, float> : tree_attention_join<D, false, float>)
                 : (few ? tree_attention_join<D, true, uint16_t> : tree_attention_join<D, false, uint16_t>);
  return op_cuda(cudaLaunchKernelEx(&cfg, fn, p), "mk_tree_attention");
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

int mk_tree_attention_workspace(const mk_cache* cache, int batch, int n_tokens, int n_heads,
                                int type, size_t* bytes) {
  if (!bytes) return op_fail(MK_ERR_INVALID, "bytes is NULL");
  CacheView view;
  Plan pl;
  if (int rc = check_attention(cache, batch, n_tokens, n_heads, type, &view)) return rc;
  if (int rc = make_plan(view, cache->head_dim, batch, n_tokens, n_heads, type, &pl)) return rc;
  *bytes = pl.bytes();
  return MK_OK;
}

int mk_tree_attention(const mk_cache* cache, int layer, int batch, int n_tokens, int n_heads,
                      int type, float scale, const void* q, int64_t q_stride,
                      const int32_t* starts, const int32_t* parents, const int32_t* counts,
                      void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                      void* stream) {
  AttnParams p;
  Plan pl;
  if (int rc = check_attention(cache, batch, n_tokens, n_heads, type, &p.cache)) return rc;
  if (layer < 0 || layer >= cache->n_layers)
    return op_fail(MK_ERR_INVALID, "layer out of range [0, n_layers)");
  if (!q || !out || !starts || !workspace)
    return op_fail(MK_ERR_INVALID, "mk_tree_attention: a NULL argument");
  if (!(scale > 0.f) || scale > 1e30f)
    return op_fail(MK_ERR_INVALID, "scale must be positive and finite");
  const int unit = type == MK_TYPE_FP32 ? 4 : 8;
  const int64_t row = (int64_t)n_heads * cache->head_dim;
  if (!aligned(q, 16) || !aligned(out, 16) || q_stride % unit || out_stride % unit ||
      q_stride < row || out_stride < row)
    return op_fail(MK_ERR_INVALID,
                   "q, out: 16-byte aligned rows, strides at least a row, are needed");
  if (!aligned(workspace, 256)) return op_fail(MK_ERR_INVALID, "workspace: not 256-byte aligned");
  if (int rc = make_plan(p.cache, cache->head_dim, batch, n_tokens, n_heads, type, &pl)) return rc;
  if (workspace_bytes < pl.bytes())
    return op_fail(MK_ERR_INVALID, "workspace: smaller than its query says");
  p.k = (const uint16_t*)cache->k[layer];
  p.v = (const uint16_t*)cache->v[layer];
  p.q = q, p.out = out, p.qs = q_stride, p.os = out_stride;
  p.starts = starts, p.parents = parents, p.counts = counts;
  p.B = batch, p.T = n_tokens, p.nh = n_heads, p.G = n_heads / cache->n_kv_heads;
  p.tile_log2 = pl.tile == 128 ? 7 : 6;
  p.extra = pl.extra, p.row_tile = pl.row_tile, p.row_tiles = pl.row_tiles, p.groups = pl.groups;
  p.inv_groups = (uint32_t)std::min<uint64_t>((1ull << 32) / pl.groups + 1, UINT32_MAX);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.part_o = (float*)workspace;
  p.part_ml = p.part_o + pl.o_floats;
  p.runs = pl.runs ? (float4*)(p.part_ml + pl.ml_floats) : nullptr;
  cudaStream_t st = (cudaStream_t)stream;
  return cache->head_dim == 64 ? launch_all<64>(p, pl, type, st) : launch_all<128>(p, pl, type, st);
}

}  // extern "C"
