// Operators that write a KV cache (include/mk.h): rotary positions with the
// append of the new rows, the accepted rows moved down, pages copied. All are
// bound by the bytes they move.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "mk_ops.h"
#include "mk_ptx.cuh"

namespace mk {

int check_cache(const mk_cache* c, int batch, bool need_table, CacheView* out) noexcept {
  if (!c) return op_fail(MK_ERR_INVALID, "cache is NULL");
  if (c->head_dim != 64 && c->head_dim != 128)
    return op_fail(MK_ERR_INVALID, "cache: head_dim must be 64 or 128");
  if (c->n_layers < 1 || c->n_layers > kMaxOpLayers)
    return op_fail(MK_ERR_INVALID, "cache: n_layers must be 1 to 64");
  if (c->n_kv_heads < 1 || c->n_blocks < 1 || c->block_size < 1)
    return op_fail(MK_ERR_INVALID,
                   "cache: n_kv_heads, n_blocks and block_size must be at least 1");
  if ((double)c->n_kv_heads * c->n_blocks * c->block_size >= (double)kNoRow)
    return op_fail(MK_ERR_INVALID, "cache: more than 2^32 - 2 rows in a layer");
  if (!c->k || !c->v) return op_fail(MK_ERR_INVALID, "cache: k / v is NULL");
  for (int l = 0; l < c->n_layers; ++l)
    if (!c->k[l] || !c->v[l] || !aligned(c->k[l], 16) || !aligned(c->v[l], 16))
      return op_fail(MK_ERR_INVALID, "cache: a layer's pointer is NULL or not 16-byte aligned");
  int64_t capacity = c->block_size;
  if (need_table) {
    if (batch < 1 || batch > kMaxSeqs || batch > c->batch)
      return op_fail(MK_ERR_INVALID, "batch must be 1 to 1024 and at most the cache's");
    if (c->block_table) {
      if (c->table_entries < 1 || !aligned(c->block_table, 4))
        return op_fail(MK_ERR_INVALID, "cache: table_entries must be at least 1");
      capacity = (int64_t)c->table_entries * c->block_size;
    } else if (c->table_entries != 0 || c->batch > c->n_blocks) {
      return op_fail(MK_ERR_INVALID,
                     "cache: a contiguous cache has table_entries 0 and a block per sequence");
    }
    if (capacity > (1 << 30)) return op_fail(MK_ERR_INVALID, "cache: capacity above 2^30 slots");
  }
  if (out)
    *out = CacheView{c->block_table, c->block_table ? c->table_entries : 0, c->n_blocks,
                     c->block_size, c->n_kv_heads, (int)capacity};
  return MK_OK;
}

namespace {

// ---- element access: N = 1, 2, 4 or 8 consecutive elements, aligned to N elements ------

// raw elements, in 32-bit words (bf16: two to a word; `at` is even unless N = 1)
template <int N>
__device__ __forceinline__ void load(const float* p, uint32_t* w, int at) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(p + i);
      w[at + i] = a.x, w[at + i + 1] = a.y, w[at + i + 2] = a.z, w[at + i + 3] = a.w;
    }
  } else if constexpr (N == 2) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[at] = a.x, w[at + 1] = a.y;
  } else {
    w[at] = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <int N>
__device__ __forceinline__ void load(const uint16_t* p, uint32_t* w, int at) {
  if constexpr (N == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[at / 2] = a.x, w[at / 2 + 1] = a.y, w[at / 2 + 2] = a.z, w[at / 2 + 3] = a.w;
  } else if constexpr (N == 4) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    w[at / 2] = a.x, w[at / 2 + 1] = a.y;
  } else if constexpr (N == 2) {
    w[at / 2] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    w[at / 2] = at & 1 ? w[at / 2] | (uint32_t)*p << 16 : *p;
  }
}
template <typename T>
__device__ __forceinline__ float elem(const uint32_t* w, int j) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
  else return (j & 1) ? bf_hi(w[j >> 1]) : bf_lo(w[j >> 1]);
}
template <int N>
__device__ __forceinline__ void store(float* p, const float* x) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else {
    *p = x[0];
  }
}
template <int N>
__device__ __forceinline__ void store(uint16_t* p, const float* x) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]),
                                              bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
  else if constexpr (N == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]));
  else if constexpr (N == 2)
    *reinterpret_cast<uint32_t*>(p) = bf16x2_rn(x[0], x[1]);
  else
    *p = (uint16_t)bf16x2_rn(x[0], 0.f);
}

// ---- rotary positions and append ------------------------------------------------

constexpr int kRopeThreads = 128, kRopeRowThreads = 256;  // of a block; of one with a single row
constexpr int kRopeTokens = 4;  // most tokens of a block

struct RopeParams {
  CacheView cache;
  mk_rope rope;
  uint16_t *k_cache, *v_cache;
  const void *q, *k, *v;
  void* q_out;
  int64_t qs, ks, vs, os;  // row strides in elements
  const int32_t *starts, *parents, *counts;
  int rows, T, nh, tokens;  // rows = batch * T; tokens per block
  // mk_norm_rope_append: the weights (nullptr: ones) and what is added to a mean square
  const uint16_t *q_norm, *k_norm;
  float eps;
};

// The block's rows: each token's position (-1: the row is not there), cache row and angles.
template <int D>
struct RopeRows {
  float2 cs[kRopeTokens][D / 2];
  int pos[kRopeTokens];
  uint32_t row[kRopeTokens];
};
template <int D, int THREADS>
__device__ __forceinline__ void find_rows(const RopeParams& p, RopeRows<D>& s) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int row0 = blockIdx.x * p.tokens;
  if (warp < p.tokens) {
    const int row = row0 + warp;
    int pos = -1;  // the row is not there
    uint32_t crow = kNoRow;
    if (row < p.rows) {
      const int b = row / p.T, t = row - b * p.T;
      if (t < clamped(p.counts, b, p.T)) {
        const int start = clamped(p.starts, b, p.cache.capacity);
        int depth = t;
        if (p.parents) {
          // lane l holds the parents of nodes l and l + 32
          const int32_t* par = p.parents + (size_t)b * p.T;
          const int lo = lane < p.T ? __ldg(par + lane) : -1;
          const int hi = lane + 32 < p.T ? __ldg(par + lane + 32) : -1;
          depth = 0;
          for (int n = t;;) {
            const int up = __shfl_sync(0xffffffffu, n < 32 ? lo : hi, n & 31);
            if (up < 0 || up >= n) break;
            n = up;
            ++depth;
          }
        }
        pos = start + depth;
        if (start + t < p.cache.capacity) crow = cache_row(p.cache, b, start + t);
      }
    }
    if (lane == 0) {
      s.pos[warp] = pos;
      s.row[warp] = crow;
    }
  }
  __syncthreads();
  for (int i = tid; i < p.tokens * (D / 2); i += THREADS) {
    const int tok = i / (D / 2), pair = i % (D / 2);
    float2 v = make_float2(1.f, 0.f);  // behind rotary_dim: passes through
    if (2 * pair < p.rope.rotary_dim) {
      const int64_t turn = (int64_t)(p.rope.turns[pair] * (uint64_t)max(s.pos[tok], 0));
      sincospif(2.f * ((float)turn * 0x1p-64f), &v.y, &v.x);
      v.x *= p.rope.magnitude;
      v.y *= p.rope.magnitude;
    }
    s.cs[tok][pair] = v;
  }
  __syncthreads();
}

// A block takes `tokens` rows: one angle per (token, pair), shared by all heads
// (sincospif of a fraction of a turn found by a 64-bit fixed-point product: position
// times the plan's own 2^-53 turns off, less than fp32's rounding up to position 2^27).
// Then a warp takes heads of q, k and v of one row, D / 8 lanes to a head. A lane
// has four pairs, both members of each, so that its sines and cosines stay in its
// registers and nothing is exchanged (q_out may be q). PIECE: elements that lie
// together for a lane, 8 when the pairs are neighbours, else the largest of 4, 2, 1
// that divides rotary_dim / 2; the elements behind rotary_dim are taken as
// neighbours.
// (Eight elements in a row per lane and the partners by shuffles: 218 us
// against 132 for the 32768 rows below in halves of 64, 450 against 138 in
// halves of 62, where the partners were loaded one by one.)
// Bound by the bytes of the rows: 32768 rows of the 8B shape, bf16, 805 MB, take
// 120 us as halves, 6.7 TB/s; U heads of a lane are in flight: 133 us with 2,
// 136 with 8 (neighbours, four rows in 256 threads, where 4 took 125). 200 rows take 4 to 5 us, a
// launch's latency; a block of a single row has 256 threads there, with 128 it took 0.2 us more.
template <typename T, int D, int PIECE, int THREADS>
__global__ void __launch_bounds__(THREADS) rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, U = 4;
  __shared__ RopeRows<D> s;
  constexpr int WARPS = THREADS / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row0 = blockIdx.x * p.tokens;
  find_rows<D, THREADS>(p, s);

  const int tok = warp % p.tokens;  // tokens divides WARPS
  if (s.pos[tok] < 0) return;
  const int n_kv = p.cache.n_kv, heads = p.nh + 2 * n_kv, step = WARPS / p.tokens * HPW;
  const int c = lane % LPH, half = p.rope.rotary_dim / 2;
  const int64_t row = row0 + tok;
  const uint32_t crow = s.row[tok];
  // piece i of the lane (elements N i to N i + N - 1 of its eight) starts at `at`;
  // elements j and j + 4 (neighbours: 2j and 2j + 1) are its pair j
  constexpr int N = PIECE, FIRST = N == 8 ? 1 : 4 / N;
  int at[8 / N];
  if constexpr (N == 8) {
    at[0] = 8 * c;
  } else {
#pragma unroll
    for (int i = 0; i < FIRST; ++i) {
      const int pair = 4 * c + N * i;
      at[i] = pair < half ? pair : 2 * pair;
      at[i + FIRST] = pair < half ? half + pair : 2 * pair + N;
    }
  }
  float2 w[4];
  bool turns[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    turns[j] = 4 * c + j < half;
    w[j] = s.cs[tok][4 * c + j];
  }
  for (int base = warp / p.tokens * HPW; base < heads; base += U * step) {
    uint32_t x[U][2 * sizeof(T)];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int head = base + u * step + lane / LPH;
      if (head >= heads) continue;
      const T* src;
      if (head < p.nh) src = (const T*)p.q + row * p.qs + head * D;
      else if (head < p.nh + n_kv) src = (const T*)p.k + row * p.ks + (head - p.nh) * D;
      else src = (const T*)p.v + row * p.vs + (head - p.nh - n_kv) * D;
#pragma unroll
      for (int i = 0; i < 8 / N; ++i) load<N>(src + at[i], x[u], N * i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int head = base + u * step + lane / LPH;
      if (head >= heads) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = elem<T>(x[u], j);
      if (head < p.nh + n_kv) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = N == 8 ? 2 * j : j, k = N == 8 ? 2 * j + 1 : j + 4;
          const float a = o[i], b = o[k];
          if (turns[j]) {
            o[i] = a * w[j].x - b * w[j].y;
            o[k] = a * w[j].y + b * w[j].x;
          }
        }
      }
      auto put = [&](auto* dst) {
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) store<N>(dst + at[i], o + N * i);
      };
      if (head < p.nh) {
        put((T*)p.q_out + row * p.os + head * D);
      } else if (crow != kNoRow) {
        const bool key = head < p.nh + n_kv;
        const int g = head - p.nh - (key ? 0 : n_kv);
        put((key ? p.k_cache : p.v_cache) + ((size_t)crow + (size_t)g * p.cache.block_size) * D);
      }
    }
  }
}

// The same of heads that are normalised first: a head x of q or k becomes x w f,
// f = 1 / sqrt(sum x^2 / D + eps), and then turns. What does not depend on the head is
// put together once for a row: a pair (a, b) with weights (v, w) becomes
//   f (a v cos - b w sin), f (a v sin + b w cos),
// four products of a weight and an angle that stay in a lane's registers while it goes
// through its heads (of q, then of k and v), pair by pair in two-wide arithmetic. A sum of
// squares is fp32, over the lane's eight elements and then the head's lanes by shuffles; one
// that leaves fp32's range is taken again from x 2^-70. Only the result is rounded.
// Bound by the bytes, with less room to wait for them than the rotation alone has: 32768 rows
// of the 8B shape, bf16 in halves, 805 MB, take 131 us, 6.1 TB/s. Weights and rotation one
// after another: 170. With one call to a graph, where this takes 133: blocks of 256 threads 144,
// and 155 with as many registers as it would like; sixteen elements a lane 157 to 174. 600 rows take 6 us, a launch's latency and
// that of a row's position, angle and queries.
template <typename T, int D, int PIECE>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 2 ? 7 : 4) norm_rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, WARPS = kRopeThreads / 32, U = 4;
  __shared__ RopeRows<D> s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row0 = blockIdx.x * p.tokens;
  const int tok = warp % p.tokens;  // tokens divides WARPS
  const int n_kv = p.cache.n_kv, step = WARPS / p.tokens * HPW;
  const int c = lane % LPH, half = p.rope.rotary_dim / 2;
  const int first = warp / p.tokens * HPW + lane / LPH;  // the lane's first head
  const int64_t row = row0 + tok;
  const unsigned mine = (LPH == 8 ? 0xffu : 0xffffu) << (lane / LPH * LPH);  // a head's lanes
  // pieces as above; the pairs behind rotary_dim turn by the angle 0
  constexpr int N = PIECE, FIRST = N == 8 ? 1 : 4 / N;
  int at[8 / N];
  if constexpr (N == 8) {
    at[0] = 8 * c;
  } else {
#pragma unroll
    for (int i = 0; i < FIRST; ++i) {
      const int pair = 4 * c + N * i;
      at[i] = pair < half ? pair : 2 * pair;
      at[i + FIRST] = pair < half ? half + pair : 2 * pair + N;
    }
  }
  constexpr auto left = [](int j) { return N == 8 ? 2 * j : j; };       // of the lane's pair j
  constexpr auto right = [](int j) { return N == 8 ? 2 * j + 1 : j + 4; };

  uint32_t x[U][2 * sizeof(T)];
  auto fetch = [&](uint32_t* x, const T* src) {
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) load<N>(src + at[i], x, N * i);
  };
  const T* q = (const T*)p.q + row * p.qs;
  auto fetch_queries = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * step < p.nh) fetch(x[u], q + (h + u * step) * D);
  };
  // the first queries are on their way while the row's position and angles are found, where
  // every row is there
  const bool early = p.counts == nullptr && row < p.rows;
  if (early) fetch_queries(first);
  find_rows<D, kRopeThreads>(p, s);
  if (s.pos[tok] < 0) return;
  const uint32_t crow = s.row[tok];

  unsigned long long turn[2][4];  // of pairs 0, 1 and 2, 3: v cos, -w sin, v sin, w cos
  auto put_together = [&](const uint16_t* weights) {
    uint32_t w[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};  // ones
    if (weights) {
#pragma unroll
      for (int i = 0; i < 8 / N; ++i) load<N>(weights + at[i], w, N * i);
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float2 x = s.cs[tok][4 * c + j], y = s.cs[tok][4 * c + j + 1];
      const float v0 = elem<uint16_t>(w, left(j)), v1 = elem<uint16_t>(w, left(j + 1));
      const float w0 = elem<uint16_t>(w, right(j)), w1 = elem<uint16_t>(w, right(j + 1));
      turn[j / 2][0] = pack2(v0 * x.x, v1 * y.x);
      turn[j / 2][1] = pack2(-w0 * x.y, -w1 * y.y);
      turn[j / 2][2] = pack2(v0 * x.y, v1 * y.y);
      turn[j / 2][3] = pack2(w0 * x.x, w1 * y.x);
    }
  };
  // the head in x, normalised and turned, to dst
  auto finish = [&](const uint32_t* x, auto* dst) {
    unsigned long long a[2], b[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      a[j] = pack2(elem<T>(x, left(2 * j)), elem<T>(x, left(2 * j + 1)));
      b[j] = pack2(elem<T>(x, right(2 * j)), elem<T>(x, right(2 * j + 1)));
    }
    auto squares = [&] {
      unsigned long long sum = mul2(a[0], a[0]);
      ffma2(sum, b[0], b[0]);
      ffma2(sum, a[1], a[1]);
      ffma2(sum, b[1], b[1]);
      const float2 z = unpack2(sum);
      float t = z.x + z.y;
#pragma unroll
      for (int d = 1; d < LPH; d *= 2) t += __shfl_xor_sync(mine, t, d);
      return t * (1.f / D);
    };
    float mean = squares(), eps = p.eps;
    if (!(mean < INFINITY)) {
      const unsigned long long small = pack2(0x1p-70f, 0x1p-70f);
#pragma unroll
      for (int j = 0; j < 2; ++j) a[j] = mul2(a[j], small), b[j] = mul2(b[j], small);
      mean = squares();
      eps = 0.f;  // below a rounding of a mean of 2^121 and more
    }
    const float f = rsqrtf(mean + eps);
    const unsigned long long f2 = pack2(f, f);
    float o[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      a[j] = mul2(a[j], f2), b[j] = mul2(b[j], f2);
      unsigned long long l = mul2(a[j], turn[j][0]), r = mul2(a[j], turn[j][2]);
      ffma2(l, b[j], turn[j][1]);
      ffma2(r, b[j], turn[j][3]);
      const float2 y = unpack2(l), z = unpack2(r);
      o[left(2 * j)] = y.x, o[left(2 * j + 1)] = y.y;
      o[right(2 * j)] = z.x, o[right(2 * j + 1)] = z.y;
    }
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) store<N>(dst + at[i], o + N * i);
  };
  put_together(p.q_norm);
  T* out = (T*)p.q_out + row * p.os;
  for (int h = first; h < p.nh; h += U * step) {
    if (!early || h != first) fetch_queries(h);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * step < p.nh) finish(x[u], out + (h + u * step) * D);
  }
  if (crow == kNoRow) return;
  put_together(p.k_norm);
  const T *k = (const T*)p.k + row * p.ks, *v = (const T*)p.v + row * p.vs;
  for (int h = first; h < n_kv; h += U / 2 * step) {
#pragma unroll
    for (int u = 0; u < U / 2; ++u) {
      const int g = h + u * step;
      if (g < n_kv) fetch(x[u], k + g * D), fetch(x[u + U / 2], v + g * D);
    }
#pragma unroll
    for (int u = 0; u < U / 2; ++u) {
      const int g = h + u * step;
      if (g >= n_kv) continue;
      const size_t to = ((size_t)crow + (size_t)g * p.cache.block_size) * D;
      finish(x[u], p.k_cache + to);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = elem<T>(x[u + U / 2], j);
#pragma unroll
      for (int i = 0; i < 8 / N; ++i) store<N>(p.v_cache + to + at[i], o + N * i);
    }
  }
}

template <typename T, int D, int PIECE, bool NORM>
void launch_rope(const RopeParams& p, cudaStream_t st) {
  const dim3 grid((p.rows + p.tokens - 1) / p.tokens);
  if constexpr (NORM) norm_rope_append_kernel<T, D, PIECE><<<grid, kRopeThreads, 0, st>>>(p);
  else if (p.tokens == 1) rope_append_kernel<T, D, PIECE, kRopeRowThreads><<<grid, kRopeRowThreads, 0, st>>>(p);
  else rope_append_kernel<T, D, PIECE, kRopeThreads><<<grid, kRopeThreads, 0, st>>>(p);
}
template <typename T, int D, bool NORM>
void launch_rope(const RopeParams& p, cudaStream_t st) {
  const int half = p.rope.rotary_dim / 2;
  if (p.rope.interleaved) launch_rope<T, D, 8, NORM>(p, st);
  else if (half % 4 == 0) launch_rope<T, D, 4, NORM>(p, st);
  else if (half % 2 == 0) launch_rope<T, D, 2, NORM>(p, st);
  else launch_rope<T, D, 1, NORM>(p, st);
}

// mk_rope_append and, with NORM, mk_norm_rope_append: the checks that they share, and
// the launch. p holds the weights and eps already.
template <bool NORM>
int rope_append(RopeParams& p, const char* name, const mk_rope* rope, const mk_cache* cache,
                int layer, int batch, int n_tokens, int n_heads, int type, const void* q,
                int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                void* q_out, int64_t q_out_stride, const int32_t* starts, const int32_t* parents,
                const int32_t* counts, void* stream) {
  if (int rc = check_cache(cache, batch, true, &p.cache)) return rc;
  if (!rope || !q || !k || !v || !q_out || !starts)
    return op_fail(MK_ERR_INVALID, NORM ? "mk_norm_rope_append: a NULL argument"
                                        : "mk_rope_append: a NULL argument");

  if (layer < 0 || layer >= cache->n_layers)
    return op_fail(MK_ERR_INVALID, "layer out of range [0, n_layers)");
  if (type != MK_TYPE_BF16 && type != MK_TYPE_FP32)
    return op_fail(MK_ERR_INVALID, "type must be MK_TYPE_BF16 or MK_TYPE_FP32");
  if (rope->head_dim != cache->head_dim || rope->rotary_dim < 2 ||
      rope->rotary_dim > rope->head_dim || rope->rotary_dim % 2)
    return op_fail(MK_ERR_INVALID, "rope is not a plan for this head_dim");
  if (n_tokens < 1 || (int64_t)batch * n_tokens > (1 << 30))
    return op_fail(MK_ERR_INVALID, "n_tokens must be at least 1 and batch x n_tokens at most 2^30");
  if (parents && n_tokens > MK_MAX_TREE)
    return op_fail(MK_ERR_INVALID, "a tree has at most MK_MAX_TREE nodes");
  if (n_heads < 1 || n_heads > 4096 || cache->n_kv_heads > 4096)
    return op_fail(MK_ERR_INVALID, "n_heads and n_kv_heads must be 1 to 4096");
  const int unit = type == MK_TYPE_FP32 ? 4 : 8;
  const int64_t need[4] = {n_heads, cache->n_kv_heads, cache->n_kv_heads, n_heads};
  const int64_t have[4] = {q_stride, k_stride, v_stride, q_out_stride};
  const void* at[4] = {q, k, v, q_out};
  for (int i = 0; i < 4; ++i)
    if (!aligned(at[i], 16) || have[i] % unit || have[i] < need[i] * cache->head_dim)
      return op_fail(MK_ERR_INVALID,
                     "q, k, v, q_out: 16-byte aligned rows, strides at least a row, are needed");
  p.rope = *rope;
  p.k_cache = (uint16_t*)cache->k[layer];
  p.v_cache = (uint16_t*)cache->v[layer];
  p.q = q, p.k = k, p.v = v, p.q_out = q_out;
  p.qs = q_stride, p.ks = k_stride, p.vs = v_stride, p.os = q_out_stride;
  p.starts = starts, p.parents = parents, p.counts = counts;
  p.rows = batch * n_tokens, p.T = n_tokens, p.nh = n_heads;
  // Rows of a block: one where the blocks are few (256 threads), from 1024 rows on two (128
  // threads), since a block's rows then find their angles together, from 4096 on four where a
  // row's heads are less than 8 KB. us for one, two, four rows, and four in 256 threads:
  //   8B shape, bf16 (12 KB)   512 rows   4.6    5.7    8.6    5.9
  //                           1024        6.7    6.4    9.2    6.6
  //                           2048       13.0   10.9   13.7   11.1
  //                           4096       23.1   19.1   19.5   20.4
  //                          32768        159  119.9  124.4  127.3
  //   1B shape, bf16 (6 KB)   1024        5.6    4.7    5.7    4.8
  //                           2048        9.3    5.8    6.6    6.2
  //                           4096       18.0   11.8   10.9   12.4
  //                          32768        128   67.6   63.2   74.0
  //   10 heads, fp32 (5 KB)   1024        6.4    3.9    4.6    4.0
  //                           4096       19.7    9.8    9.9   11.1
  //                          32768        138   52.6   52.0   59.8
  //   8B shape, fp32 (24 KB)  4096       32.0   31.6   33.7   31.9
  //                          32768        225  213.8  217.2  213.7
  // Normed, always 128 threads, two rows as long as all blocks are resident (7 per SM in bf16, 4
  // in fp32), then four up to 16 KB:
  //   8B shape, bf16 (12 KB)   512 rows   4.9    5.7    8.3
  //                           1024        6.2    6.7    9.1
  //                           2048       12.0   10.7   13.8
  //                           4096       21.6   19.5   19.3
  //                          32768        144  129.7  127.7
  //   1B shape, bf16 (6 KB)   2048        7.8    6.1    6.7
  //                           2560       10.5    8.5    7.7
  //                           4096       15.7   12.2   10.8
  //   10 heads, fp32 (5 KB)   1024        6.3    4.5    4.9
  //                           1536        8.2    6.7    5.3
  //   8B shape, fp32 (24 KB)  2048       17.4   17.7   17.7
  //                           4096       32.3   30.8   33.7
  //                          32768        221  212.5  215.3
  const int64_t row_bytes = (int64_t)(n_heads + 2 * cache->n_kv_heads) * cache->head_dim * (type == MK_TYPE_FP32 ? 4 : 2);
  const int most = NORM ? 2 * 152 * (type == MK_TYPE_FP32 ? 4 : 7) : 4095;  // rows in blocks of two
  const int64_t narrow = NORM ? 16384 : 8192;
  p.tokens = p.rows < 1024 ? 1 : p.rows > most && row_bytes < narrow ? kRopeTokens : 2;
  cudaStream_t st = (cudaStream_t)stream;
  if (type == MK_TYPE_FP32) {
    if (cache->head_dim == 64) launch_rope<float, 64, NORM>(p, st);
    else launch_rope<float, 128, NORM>(p, st);
  } else {
    if (cache->head_dim == 64) launch_rope<uint16_t, 64, NORM>(p, st);
    else launch_rope<uint16_t, 128, NORM>(p, st);
  }
  return op_cuda(cudaGetLastError(), name);
}

// ---- accepted rows moved down ------------------------------------------------------

constexpr int kMoveThreads = 256;

struct MoveParams {
  CacheView cache;
  const int32_t *starts, *path, *accepted;
  int T, columns;  // columns: 16-byte columns of a sequence, layers x 2 x n_kv x D / 8
  uint16_t* pool[2 * kMaxOpLayers];  // k of layer 0, v of layer 0, k of layer 1, ...
};

// A block takes one sequence and kMoveThreads of its columns: the list of moves
// (row numbers at kv-head 0) once in shared memory, then each thread moves its
// 16-byte column of every row. Sources ascend and no source lies below its
// destination, so loading eight rows before storing them never meets a row
// that an earlier store has overwritten. Bound by latency, the rows are few: one to
// six accepted rows of 8 sequences in 16 layers of the 1B shape, 24 of them to move,
// 1.6 MB, take 3.8 us.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const __grid_constant__ MoveParams p) {
  __shared__ uint32_t from[MK_MAX_TREE], to[MK_MAX_TREE];
  __shared__ int s_n;
  const int b = blockIdx.y, tid = threadIdx.x;
  if (tid < 32) {
    const int n = clamped(p.accepted, b, p.T);
    const int start = clamped(p.starts, b, p.cache.capacity);
    int last = -1, m = 0;  // the largest source so far, moves so far
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + tid;
      const int src = i < n ? __ldg(p.path + (size_t)b * p.T + i) : -1;
      const bool fits = i < n && src >= i && src < p.T;
      // ascending: above every fitting entry before it
      int above = fits ? src : -1;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, above, d);
        if (tid >= d) above = max(above, v);
      }
      int before = __shfl_up_sync(0xffffffffu, above, 1);
      before = tid ? max(last, before) : last;
      last = max(last, __shfl_sync(0xffffffffu, above, 31));
      bool moves = fits && src > before && src != i && start + src < p.cache.capacity;
      uint32_t f = kNoRow, t = kNoRow;
      if (moves) {
        f = cache_row(p.cache, b, start + src);
        t = cache_row(p.cache, b, start + i);
        moves = f != kNoRow && t != kNoRow;
      }
      const unsigned who = __ballot_sync(0xffffffffu, moves);
      if (moves) {
        const int at = m + __popc(who & ((1u << tid) - 1));
        from[at] = f;
        to[at] = t;
      }
      m += __popc(who);
    }
    if (tid == 0) s_n = m;
  }
  __syncthreads();
  const int n = s_n, col = blockIdx.x * kMoveThreads + tid;
  if (n == 0 || col >= p.columns) return;
  constexpr int CPR = D / 8;
  const int piece = col / CPR, g = piece % p.cache.n_kv;
  uint16_t* pool = p.pool[piece / p.cache.n_kv] +
                   ((size_t)g * p.cache.block_size * CPR + col % CPR) * 8;
  for (int i = 0; i < n; i += 8) {
    uint4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) x[j] = *reinterpret_cast<const uint4*>(pool + (size_t)from[i + j] * D);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) *reinterpret_cast<uint4*>(pool + (size_t)to[i + j] * D) = x[j];
  }
}

// ---- pages copied ---------------------------------------------------------------------

constexpr int kCopyThreads = 256, kCopyUnroll = 8;
constexpr int kCopyVecs = kCopyThreads * kCopyUnroll;  // 16-byte vectors of a block: 32 KB

constexpr int kCopyList = 1024;                        // copies of a launch

struct CopyParams {
  int n_kv, row_vecs, block_size, parts;
  uint16_t* pool[2 * kMaxOpLayers];
  mk_block_copy copies[kCopyList];
};

// A block copies up to 32 KB of one page of one pool: eight 16-byte loads per
// thread in flight, then the stores. The list travels in the kernel parameters
// (13 KB; a short list in a shorter block of parameters was no faster), so a call needs no device memory and can be captured.
// Bound by the bytes: 500 pages of 16 rows in 32 layers of the 8B shape, 2.1 GB, take
// 301 us, 7.0 TB/s.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
  const mk_block_copy c = p.copies[blockIdx.x / p.parts];
  const int part = blockIdx.x % p.parts;
  const int head = c.rows * p.row_vecs;            // vectors copied of each kv-head
  const int stride = p.block_size * p.row_vecs;    // vectors between kv-heads
  const int total = head * p.n_kv;
  uint4* pool = reinterpret_cast<uint4*>(p.pool[blockIdx.y]);
  const uint4* src = pool + (size_t)c.src * p.n_kv * stride;
  uint4* dst = pool + (size_t)c.dst * p.n_kv * stride;
  const int first = part * kCopyVecs + threadIdx.x;
  uint4 x[kCopyUnroll];
  int at[kCopyUnroll];
#pragma unroll
  for (int j = 0; j < kCopyUnroll; ++j) {
    const int v = first + j * kCopyThreads;
    at[j] = -1;
    if (v < total) {
      at[j] = head == stride ? v : v / head * stride + v % head;
      x[j] = src[at[j]];
    }
  }
#pragma unroll
  for (int j = 0; j < kCopyUnroll; ++j)
    if (at[j] >= 0) dst[at[j]] = x[j];
}

int launch_copies(const mk_cache* c, const mk_block_copy* copies, int n, cudaStream_t st) {
  CopyParams p;
  p.n_kv = c->n_kv_heads;
  p.row_vecs = c->head_dim / 8;
  p.block_size = c->block_size;
  for (int l = 0; l < c->n_layers; ++l) {
    p.pool[2 * l] = (uint16_t*)c->k[l];
    p.pool[2 * l + 1] = (uint16_t*)c->v[l];
  }
  int most = 0;
  for (int i = 0; i < n; ++i) {
    p.copies[i] = copies[i];
    most = copies[i].rows > most ? copies[i].rows : most;
  }
  if (most == 0) return MK_OK;
  p.parts = (int)(((int64_t)most * p.row_vecs * p.n_kv + kCopyVecs - 1) / kCopyVecs);
  copy_kernel<<<dim3((unsigned)n * p.parts, 2 * c->n_layers), kCopyThreads, 0, st>>>(p);
  return op_cuda(cudaGetLastError(), "mk_cache_copy_blocks");
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

int mk_rope_init(const mk_rope_config* c, mk_rope* out) {
  if (!c || !out) return op_fail(MK_ERR_INVALID, "config / out is NULL");
  if (c->head_dim != 64 && c->head_dim != 128)
    return op_fail(MK_ERR_INVALID, "rope: head_dim must be 64 or 128");
  const int n = c->rotary_dim;
  if (n < 2 || n > c->head_dim || n % 2)
    return op_fail(MK_ERR_INVALID, "rope: rotary_dim must be even, 2 to head_dim");
  if (!(c->theta >= 1) || !(c->factor >= 1) || std::isinf(c->theta) || std::isinf(c->factor))
    return op_fail(MK_ERR_INVALID, "rope: theta and factor must be at least 1 and finite");
  if (c->scaling < MK_ROPE_NONE || c->scaling > MK_ROPE_YARN ||
      (c->interleaved != 0 && c->interleaved != 1))
    return op_fail(MK_ERR_INVALID, "rope: unknown scaling or layout");
  const bool by_length = c->scaling == MK_ROPE_BANDS || c->scaling == MK_ROPE_YARN;
  if (by_length && (c->original_length < 1 || !(c->low > 0) || !(c->high > c->low) ||
                    std::isinf(c->high)))
    return op_fail(MK_ERR_INVALID, "rope: original_length >= 1 and 0 < low < high are needed");
  if (c->scaling == MK_ROPE_YARN && !(c->theta > 1))
    return op_fail(MK_ERR_INVALID, "rope: MK_ROPE_YARN needs theta above 1");
  if (!(c->magnitude >= 0.f) || std::isinf(c->magnitude))
    return op_fail(MK_ERR_INVALID, "rope: magnitude must be finite and not negative");
  const double two_pi = 6.283185307179586476925, length = c->original_length;
  double first = 0, last = 0;  // MK_ROPE_YARN: the ramp over the pairs
  if (c->scaling == MK_ROPE_YARN) {
    const double per = n / (2 * std::log(c->theta));
    first = std::floor(per * std::log(length / (c->high * two_pi)));
    last = std::ceil(per * std::log(length / (c->low * two_pi)));
    if (first < 0) first = 0;
    if (last > n - 1) last = n - 1;
  }
  out->head_dim = c->head_dim;
  out->rotary_dim = n;
  out->interleaved = c->interleaved;
  out->magnitude = c->magnitude > 0.f ? c->magnitude
                   : c->scaling == MK_ROPE_YARN ? (float)(0.1 * std::log(c->factor) + 1)
                                                : 1.f;
  for (int i = 0; i < 64; ++i) out->turns[i] = 0;
  for (int i = 0; i < n / 2; ++i) {
    double f = std::pow(c->theta, -2.0 * i / n);
    const double far = f / c->factor;
    if (c->scaling == MK_ROPE_LINEAR) {
      f = far;
    } else if (c->scaling == MK_ROPE_BANDS) {
      const double mix = (length * f / two_pi - c->low) / (c->high - c->low);
      f = mix <= 0 ? far : mix >= 1 ? f : (1 - mix) * far + mix * f;
    } else if (c->scaling == MK_ROPE_YARN) {
      const double ramp = last > first ? (i - first) / (last - first) : i > first ? 1.0 : 0.0;
      f = ramp <= 0 ? f : ramp >= 1 ? far : far * ramp + f * (1 - ramp);
    }
    out->turns[i] = (uint64_t)(f / two_pi * 18446744073709551616.0);  // f <= 1: below 2^62
  }
  return MK_OK;
}

int mk_rope_append(const mk_rope* rope, const mk_cache* cache, int layer, int batch,
                   int n_tokens, int n_heads, int type, const void* q, int64_t q_stride,
                   const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                   int64_t q_out_stride, const int32_t* starts, const int32_t* parents,
                   const int32_t* counts, void* stream) {
  RopeParams p;
  p.q_norm = p.k_norm = nullptr;
  p.eps = 0.f;
  return rope_append<false>(p, "mk_rope_append", rope, cache, layer, batch, n_tokens, n_heads, type, q,
                            q_stride, k, k_stride, v, v_stride, q_out, q_out_stride, starts, parents,
                            counts, stream);
}

int mk_norm_rope_append(const mk_rope* rope, const void* q_norm, const void* k_norm, float eps,
                        const mk_cache* cache, int layer, int batch, int n_tokens, int n_heads,
                        int type, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, void* q_out, int64_t q_out_stride,
                        const int32_t* starts, const int32_t* parents, const int32_t* counts,
                        void* stream) {
  if (!aligned(q_norm, 16) || !aligned(k_norm, 16))
    return op_fail(MK_ERR_INVALID, "q_norm, k_norm: not 16-byte aligned");
  if (!(eps >= 1e-30f) || !(eps <= 1.f))
    return op_fail(MK_ERR_INVALID, "eps must be 1e-30 to 1");
  RopeParams p;
  p.q_norm = (const uint16_t*)q_norm;
  p.k_norm = (const uint16_t*)k_norm;
  p.eps = eps;
  return rope_append<true>(p, "mk_norm_rope_append", rope, cache, layer, batch, n_tokens, n_heads, type, q,
                            q_stride, k, k_stride, v, v_stride, q_out, q_out_stride, starts, parents,
                            counts, stream);
}

int mk_cache_compact(const mk_cache* cache, int batch, int n_tokens, const int32_t* starts,
                     const int32_t* path, const int32_t* accepted, void* stream) {
  MoveParams p;
  if (int rc = check_cache(cache, batch, true, &p.cache)) return rc;
  if (!starts || !path || !accepted)
    return op_fail(MK_ERR_INVALID, "mk_cache_compact: a NULL argument");
  if (n_tokens < 1 || n_tokens > MK_MAX_TREE)
    return op_fail(MK_ERR_INVALID, "n_tokens must be 1 to MK_MAX_TREE");
  const int64_t columns = (int64_t)cache->n_layers * 2 * cache->n_kv_heads * (cache->head_dim / 8);
  if (columns > (1 << 30)) return op_fail(MK_ERR_INVALID, "cache: too many kv-heads");
  p.starts = starts, p.path = path, p.accepted = accepted;
  p.T = n_tokens;
  p.columns = (int)columns;
  for (int l = 0; l < cache->n_layers; ++l) {
    p.pool[2 * l] = (uint16_t*)cache->k[l];
    p.pool[2 * l + 1] = (uint16_t*)cache->v[l];
  }
  const dim3 grid((p.columns + kMoveThreads - 1) / kMoveThreads, batch);
  cudaStream_t st = (cudaStream_t)stream;
  if (cache->head_dim == 64) compact_kernel<64><<<grid, kMoveThreads, 0, st>>>(p);
  else compact_kernel<128><<<grid, kMoveThreads, 0, st>>>(p);
  return op_cuda(cudaGetLastError(), "mk_cache_compact");
}

int mk_cache_copy_blocks(const mk_cache* cache, const mk_block_copy* copies, int n_copies,
                         void* stream) {
  if (int rc = check_cache(cache, 1, false, nullptr)) return rc;
  if (n_copies < 0 || (n_copies > 0 && !copies))
    return op_fail(MK_ERR_INVALID, "copies is NULL or n_copies negative");
  if ((int64_t)cache->n_kv_heads * cache->block_size * (cache->head_dim / 8) > (1 << 30))
    return op_fail(MK_ERR_INVALID, "cache: a page above 16 GB");
  std::vector<uint64_t> is_dst;  // one bit per page
  try {
    is_dst.assign((size_t)cache->n_blocks / 64 + 1, 0);
  } catch (const std::exception&) {
    return op_fail(MK_ERR_OOM, "no host memory");
  }
  for (int i = 0; i < n_copies; ++i) {
    const mk_block_copy& c = copies[i];
    if (c.src < 0 || c.src >= cache->n_blocks || c.dst < 0 || c.dst >= cache->n_blocks ||
        c.rows < 0 || c.rows > cache->block_size)
      return op_fail(MK_ERR_INVALID, "a copy's page or rows are out of range");
    uint64_t& word = is_dst[c.dst / 64];
    if (word >> (c.dst % 64) & 1)
      return op_fail(MK_ERR_INVALID, "a page is the destination of two copies");
    word |= 1ull << (c.dst % 64);
  }
  for (int i = 0; i < n_copies; ++i)
    if (is_dst[copies[i].src / 64] >> (copies[i].src % 64) & 1)
      return op_fail(MK_ERR_INVALID, "a page is a source and a destination");
  for (int64_t i = 0; i < n_copies; i += kCopyList) {
    const int n = (int)std::min<int64_t>(n_copies - i, kCopyList);
    if (int rc = launch_copies(cache, copies + i, n, (cudaStream_t)stream)) return rc;
  }
  return MK_OK;
}

}  // extern "C"
