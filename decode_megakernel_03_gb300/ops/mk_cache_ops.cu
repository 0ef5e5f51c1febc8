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

constexpr int kRopeThreads = 256;
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
};

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
// 125 us as neighbours, 6.4 TB/s; U heads of a lane are in flight: 133 us with 2,
// 136 with 8. 200 rows take 4 to 5 us, a launch's latency.
template <typename T, int D, int PIECE>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, WARPS = kRopeThreads / 32, U = 4;
  __shared__ float2 cs[kRopeTokens][D / 2];
  __shared__ int s_pos[kRopeTokens];
  __shared__ uint32_t s_row[kRopeTokens];
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
      s_pos[warp] = pos;
      s_row[warp] = crow;
    }
  }
  __syncthreads();
  for (int i = tid; i < p.tokens * (D / 2); i += kRopeThreads) {
    const int tok = i / (D / 2), pair = i % (D / 2);
    float2 v = make_float2(1.f, 0.f);  // behind rotary_dim: passes through
    if (2 * pair < p.rope.rotary_dim) {
      const int64_t turn = (int64_t)(p.rope.turns[pair] * (uint64_t)max(s_pos[tok], 0));
      sincospif(2.f * ((float)turn * 0x1p-64f), &v.y, &v.x);
      v.x *= p.rope.magnitude;
      v.y *= p.rope.magnitude;
    }
    cs[tok][pair] = v;
  }
  __syncthreads();

  const int tok = warp % p.tokens;  // tokens divides WARPS
  if (s_pos[tok] < 0) return;
  const int n_kv = p.cache.n_kv, heads = p.nh + 2 * n_kv, step = WARPS / p.tokens * HPW;
  const int c = lane % LPH, half = p.rope.rotary_dim / 2;
  const int64_t row = row0 + tok;
  const uint32_t crow = s_row[tok];
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
    w[j] = cs[tok][4 * c + j];
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

template <typename T, int D>
void launch_rope(const RopeParams& p, cudaStream_t st) {
  const dim3 grid((p.rows + p.tokens - 1) / p.tokens);
  const int half = p.rope.rotary_dim / 2;
  if (p.rope.interleaved) rope_append_kernel<T, D, 8><<<grid, kRopeThreads, 0, st>>>(p);
  else if (half % 4 == 0) rope_append_kernel<T, D, 4><<<grid, kRopeThreads, 0, st>>>(p);
  else if (half % 2 == 0) rope_append_kernel<T, D, 2><<<grid, kRopeThreads, 0, st>>>(p);
  else rope_append_kernel<T, D, 1><<<grid, kRopeThreads, 0, st>>>(p);
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
  if (int rc = check_cache(cache, batch, true, &p.cache)) return rc;
  if (!rope || !q || !k || !v || !q_out || !starts)
    return op_fail(MK_ERR_INVALID, "mk_rope_append: a NULL argument");
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
  // Rows of a block: one where the blocks are few (8B shape, bf16, 512 rows: 6.2 us
  // against 7.2 with four), four where there are enough, since a block's rows
  // then find their angles together (1024 rows 7.2 us against 8.2 with one, 2048
  // 11.0 against 14.1, 32768 126 against 168).
  p.tokens = p.rows >= 1024 ? kRopeTokens : 1;
  cudaStream_t st = (cudaStream_t)stream;
  if (type == MK_TYPE_FP32) {
    if (cache->head_dim == 64) launch_rope<float, 64>(p, st);
    else launch_rope<float, 128>(p, st);
  } else {
    if (cache->head_dim == 64) launch_rope<uint16_t, 64>(p, st);
    else launch_rope<uint16_t, 128>(p, st);
  }
  return op_cuda(cudaGetLastError(), "mk_rope_append");
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
