// Attention of a tree of drafted tokens (include/mk.h, mk_tree_attention): the
// kernel for many rows of bf16 activations, on the tensor-memory matrix unit.
//
// One block per SM, twelve warps:
//   warps 0-3, 4-7  softmax of stream 0 and 1: one thread per row
//   warp 8          one thread issues every product
//   warps 9-11      load the key and value tiles (128 keys each)
// With two row blocks (TWO) stream s is the rows of block s, over every tile;
// with one, both streams take the same rows, stream s the tiles of parity s,
// and stream 0 joins the two at the end. Either way one stream's softmax runs
// while the matrix unit works for the other.
//
// Per stream and tile: S = Q K^T (128 x 128, fp32, tensor memory); the row's
// thread reads it, masks it, and writes the weights p = 2^(s - m) back as bf16
// over S; O += P V (128 x D, fp32, tensor memory). The reference m of a row
// follows its maximum only when that exceeds it by 2^8 (or at the first key), so
// O is almost never rescaled; the sum of the weights is kept in fp32 from the
// unrounded weights. The weights' rounding to bf16 (relative 2^-8) is the
// size of the output's own.
//
// K and V tiles go through a ring of 16 or 32 KB buffers in the order the
// products use them, with 16-byte asynchronous copies, so that any page size,
// rows that are not there (zeroed) and odd starts need nothing special; they
// lie in the 128-byte-swizzled form in which the matrix unit reads K by rows and
// V by columns.
//
// Every wait ends: after kWaitNs a thread stops waiting for good and goes on, and
// the rows of the block come out as NaN.
#include "mk_tree_attention.cuh"

namespace mk {
namespace {

constexpr int kKeys = 128;          // keys of a tile
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9, kLoadWarps = 3;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr int kLoadThreads = 32 * kLoadWarps;
constexpr int kMasks = 8;           // tiles whose masks are kept
constexpr int kTabs = 4;            // tiles whose row numbers are kept
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kSlack = 8.f;       // log2 of how far a weight may exceed 1

// ---- tensor memory and the matrix unit -------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t smem_addr, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// arrives on the barrier when every product issued by this thread is done
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// 32 columns of the lane's row
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory operand of 128-byte swizzled rows (64 bf16 each, groups of eight
// rows 1024 bytes apart). Read by rows (K-major) `lead` is unused; read by
// columns (MN-major) it is the distance of the next 64 columns.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         1ull << 46 | 2ull << 61;
}
// bf16 operands, fp32 accumulator, M = 128
__host__ __device__ constexpr uint32_t instruction(int n, bool b_by_columns) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_by_columns ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 |
         (128u / 16) << 24;
}
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t what,
                                         uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(what), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t what,
                                         uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(what), "r"(add)
      : "memory");
}

// arrives when this thread's earlier asynchronous copies have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int D, bool TWO>
struct Layout {
  static constexpr int kBuf = kKeys * D * 2;            // a K or V tile
  static constexpr int kBufs = D == 64 ? 8 : TWO ? 4 : 5;
  static constexpr int kQ = (TWO ? 2 : 1) * 128 * D * 2;
  static constexpr int kBytes = kQ + kBufs * kBuf + 1024;  // 1024: alignment of the base
};

struct Shared {
  uint64_t full[8], empty[8];
  uint64_t s_full[2], p_full[2];   // a stream's scores / weights are in tensor memory
  uint64_t q_full, o_full;         // a share's queries are loaded / its products done
  uint64_t done[2];                // a share (by parity) is written
  uint32_t tmem;
  int failed;                      // a wait ran out
  alignas(16) uint32_t mask[kMasks][4];  // keys of a tile that are there
  uint32_t tab[kTabs][kKeys];      // row numbers of a tile's keys
  // non-finite values of the nodes' v rows (share parity): +inf in [0], -inf in
  // [1], NaN in both; odd: whether there are any
  uint32_t odd[2];
  uint32_t odd_at[2][MK_MAX_TREE][2][4];
  float ml[128][2];                // stream 1's (m, l), one row block
};

// Waits with an end: a thread whose wait ran out does not wait again (its
// control flow goes on unchanged, so that barriers keep their counts).
struct Waiter {
  Shared& sm;
  bool ok = true;
  __device__ __forceinline__ explicit Waiter(Shared& s) : sm(s) {}
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!ok || mbar_try_wait(bar, parity & 1)) return;
    const uint64_t since = globaltimer();
    while (!mbar_try_wait(bar, parity & 1)) {
      if (globaltimer() - since > kWaitNs) {
        ok = false;
        *reinterpret_cast<volatile int*>(&sm.failed) = 1;
        return;
      }
    }
  }
};

// ---- the loading warps -------------------------------------------------------------

template <int D, bool TWO>
__device__ __forceinline__ void load_role(const AttnParams& p, Shared& sm, const int* prefix,
                                          uint32_t ring, uint8_t* ring_ptr, int u_begin,
                                          int u_end, int rt) {
  using Lay = Layout<D, TWO>;
  constexpr int LEAD = TWO ? 1 : 2;      // K tiles ahead of V
  constexpr int CPR = D / 8, RPW = 32 / CPR;
  const int lt = threadIdx.x - 32 * kLoadWarp, lw = lt / 32, lane = lt % 32;
  Waiter wait(sm);
  uint32_t buf = 0, round = 0;           // next buffer of the ring, its round
  uint32_t tile_no = 0;                  // K tiles loaded so far
  int u = u_begin;
  Share sh;
  for (uint32_t share = 0; next_share(p, prefix, u_begin, u_end, u, sh);) {
    if (rt * p.row_tile >= sh.rows) continue;
    auto row_of = [&](int t, int r) -> uint32_t {
      const int slot = (sh.k0 + t) * kKeys + r;
      if (t >= sh.n || r >= kKeys || slot >= sh.len) return kNoRow;
      const uint32_t row = cache_row(p.cache, sh.b, slot);
      return row == kNoRow ? row : row + (uint32_t)sh.g * p.cache.block_size;
    };
    uint32_t r0 = row_of(0, lt), r1 = row_of(0, lt + kLoadThreads);
    const uint32_t first = tile_no;      // number of the share's tile 0

    auto copy = [&](const uint16_t* pool, const uint32_t* tab) {
      const uint32_t base = ring + buf * Lay::kBuf;
      const int c = lane % CPR;
#pragma unroll 4
      for (int r = lw * RPW + lane / CPR; r < kKeys; r += kLoadWarps * RPW) {
        const uint32_t row = tab[r];
        const bool there = row != kNoRow;
        cp_async16(base + (c / 8) * (kKeys * 128) + r * 128 + (((c % 8) ^ (r & 7)) * 16),
                   pool + (there ? (size_t)row * D + 8 * c : 0), there ? 16 : 0);
      }
    };
    auto advance = [&] {
      if (++buf == Lay::kBufs) buf = 0, ++round;
    };

    for (int j = -LEAD; j < sh.n; ++j) {
      if (j >= 0) {
        wait(&sm.empty[buf], round + 1);
        copy(p.v, sm.tab[(first + j) % kTabs]);
        const int slot0 = (sh.k0 + j) * kKeys;
        if (slot0 + kKeys > sh.start) {
          // nodes in the tile: a value that some rows must not see is not
          // cancelled by a zero weight if it is not finite, so it is taken out
          // here and added at the end to the rows that see it
          asm volatile("cp.async.wait_all;" ::: "memory");
          if (share >= 2) wait(&sm.done[share & 1], share / 2 - 1);  // its list is free again
          named_bar(2, kLoadThreads);
          const uint32_t* tab = sm.tab[(first + j) % kTabs];
          uint8_t* base = ring_ptr + buf * Lay::kBuf;
          for (int i = lt; i < kKeys * CPR; i += kLoadThreads) {
            const int r = i / CPR, c = i % CPR, node = slot0 + r - sh.start;
            if (node < 0 || node >= sh.count || tab[r] == kNoRow) continue;
            uint16_t* x = reinterpret_cast<uint16_t*>(base + (c / 8) * (kKeys * 128) + r * 128 +
                                                      (((c % 8) ^ (r & 7)) * 16));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint16_t v = x[e];
              if ((v & 0x7f80) == 0x7f80) {
                const int d = c * 8 + e;
                const bool nan = v & 0x7f;
                uint32_t(*at)[4] = sm.odd_at[share & 1][node];
                if (nan || !(v & 0x8000)) atomicOr(&at[0][d / 32], 1u << (d % 32));
                if (nan || (v & 0x8000)) atomicOr(&at[1][d / 32], 1u << (d % 32));
                atomicOr(&sm.odd[share & 1], 1u);
                x[e] = 0;
              }
            }
          }
          fence_async_smem();
          mbar_arrive(&sm.full[buf]);
        } else {
          cp_async_arrive(&sm.full[buf]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[buf]);
        advance();
      }
      if (const int t = j + LEAD; t < sh.n) {
        uint32_t* tab = sm.tab[tile_no % kTabs];
        uint32_t* mask = sm.mask[tile_no % kMasks];
        tab[lt] = r0;
        const uint32_t m0 = __ballot_sync(0xffffffffu, r0 != kNoRow);
        const uint32_t m1 = __ballot_sync(0xffffffffu, r1 != kNoRow);
        if (lt + kLoadThreads < kKeys) tab[lt + kLoadThreads] = r1;
        named_bar(2, kLoadThreads);
        wait(&sm.empty[buf], round + 1);
        if (lane == 0) {
          mask[lw] = m0;
          if (lw == 0) mask[3] = m1;
        }
        copy(p.k, tab);
        cp_async_arrive(&sm.full[buf]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[buf]);
        advance();
        ++tile_no;
        r0 = row_of(t + 1, lt);
        r1 = row_of(t + 1, lt + kLoadThreads);
      }
    }
    ++share;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- the issuing thread ----------------------------------------------------------------

template <int D, bool TWO>
__device__ __forceinline__ void mma_role(const AttnParams& p, Shared& sm, const int* prefix,
                                         uint32_t q_smem, uint32_t ring, uint32_t tmem,
                                         int u_begin, int u_end, int rt) {
  using Lay = Layout<D, TWO>;
  constexpr uint32_t kScores = instruction(kKeys, false), kValues = instruction(D, true);
  Waiter wait(sm);
  uint32_t buf = 0, round = 0;
  uint32_t p_uses[2] = {0, 0};
  int u = u_begin;
  Share sh;
  auto advance = [&] {
    tc_commit(&sm.empty[buf]);
    if (++buf == Lay::kBufs) buf = 0, ++round;
  };
  auto arrived = [&] {  // the next buffer of the ring is there
    wait(&sm.full[buf], round);
    fence_async_smem();
  };
  // S of stream s from the K tile in the next buffer
  auto scores = [&](int s) {
    const uint32_t k = ring + buf * Lay::kBuf, q = q_smem + (TWO ? s * 128 * D * 2 : 0);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t at = (i / 4) * (kKeys * 128) + (i % 4) * 32;
      mma_smem(tmem + s * kKeys, operand(q + at, 16), operand(k + at, 16), kScores, i > 0);
    }
    tc_commit(&sm.s_full[s]);
    mbar_arrive(&sm.s_full[s]);  // hands on the tile's mask
  };
  auto values = [&](int s, bool add) {
    const uint32_t v = ring + buf * Lay::kBuf;
    wait(&sm.p_full[s], p_uses[s]++);
    tc_fence_after();
#pragma unroll
    for (int i = 0; i < kKeys / 16; ++i)
      mma_tmem(tmem + 2 * kKeys + s * D, tmem + s * kKeys + i * 8, operand(v + i * 2048, kKeys * 128),
               kValues, add || i > 0);
  };
  for (uint32_t share = 0; next_share(p, prefix, u_begin, u_end, u, sh);) {
    if (rt * p.row_tile >= sh.rows) continue;
    wait(&sm.q_full, share);
    fence_async_smem();
    tc_fence_after();
    if constexpr (TWO) {
      arrived();
      scores(0);
      scores(1);
      advance();
      for (int j = 0; j < sh.n; ++j) {
        arrived();  // V of tile j; the K behind it is waited for below
        const uint32_t v_buf = buf, v_round = round;
        uint32_t k_buf = buf + 1, k_round = round;
        if (k_buf == Lay::kBufs) k_buf = 0, ++k_round;
        for (int s = 0; s < 2; ++s) {
          buf = v_buf, round = v_round;
          values(s, j > 0);
          if (s == 1) tc_commit(&sm.empty[v_buf]);
          buf = k_buf, round = k_round;
          if (j + 1 < sh.n) {
            if (s == 0) arrived();
            scores(s);
          }
        }
        if (j + 1 < sh.n) advance();
      }
    } else {
      for (int s = 0; s < 2 && s < sh.n; ++s) {
        arrived();
        scores(s);
        advance();
      }
      for (int j = 0; j < sh.n; ++j) {
        const int s = j & 1;
        arrived();
        values(s, j >= 2);
        advance();
        if (j + 2 < sh.n) {
          arrived();
          scores(s);
          advance();
        }
      }
    }
    tc_commit(&sm.o_full);
    mbar_arrive(&sm.o_full);
    ++share;
  }
}

// ---- the softmax warps -------------------------------------------------------------------

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int from) {
  return __shfl_sync(0xffffffffu, v, from);
}

// The nodes that node `t` sees (t < 64, -1: none), by doubling inside the warp:
// lane l holds nodes l and l + 32, `up` the next ancestor behind `seen`.
__device__ __forceinline__ uint64_t nodes_seen(const AttnParams& p, int b, int count, int t) {
  const int lane = threadIdx.x % 32;
  uint64_t seen[2];
  int up[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = lane + 32 * h;
    int x = -1;
    if (n < count) {
      x = p.parents ? __ldg(p.parents + (size_t)b * p.T + n) : n - 1;
      if (x < 0 || x >= n) x = -1;
    }
    up[h] = x;
    seen[h] = 1ull << n;
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    uint64_t s2[2];
    int u2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int from = up[h] & 31;
      const uint64_t a = shfl64(seen[0], from), c = shfl64(seen[1], from);
      const int ua = __shfl_sync(0xffffffffu, up[0], from), uc = __shfl_sync(0xffffffffu, up[1], from);
      s2[h] = seen[h] | (up[h] < 0 ? 0 : up[h] < 32 ? a : c);
      u2[h] = up[h] < 0 ? -1 : up[h] < 32 ? ua : uc;
    }
    seen[0] = s2[0], seen[1] = s2[1];
    up[0] = u2[0], up[1] = u2[1];
  }
  const uint64_t a = shfl64(seen[0], t & 31), c = shfl64(seen[1], t & 31);
  return t < 0 ? 0 : t < 32 ? a : c;
}

template <int D, bool TWO>
__device__ __forceinline__ void softmax_role(const AttnParams& p, Shared& sm, const int* prefix,
                                             uint8_t* q_ptr, uint32_t tmem, int u_begin,
                                             int u_end, int rt, int group) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int stream = warp / 4, r = (warp % 4) * 32 + lane;  // row of the stream's block
  const uint32_t lanes = (uint32_t)(warp % 4) * 32 << 16;
  const uint32_t t_s = tmem + lanes + stream * kKeys, t_o = tmem + lanes + 2 * kKeys + stream * D;
  const int block_rows = TWO ? p.row_tile / 2 : 128;       // rows of a stream's block
  const int local = TWO ? stream * block_rows + r : r;     // row of the row tile
  Waiter wait(sm);
  uint32_t s_uses = 0, tile_no = 0;
  int u = u_begin;
  Share sh;
  for (uint32_t share = 0; next_share(p, prefix, u_begin, u_end, u, sh);) {
    if (rt * p.row_tile >= sh.rows) continue;
    const int row = rt * p.row_tile + local;
    const bool live = r < block_rows && row < sh.rows;
    const bool warp_live = __any_sync(0xffffffffu, live);

    // ---- the row's queries, swizzled; rows that are not there are zero
    if (TWO || stream == 0) {
      uint8_t* dst = q_ptr + (TWO ? stream * 128 * D * 2 : 0) + r * 128;
      const uint4* src = reinterpret_cast<const uint4*>(
          (const uint16_t*)p.q + (live ? row_offset(p, sh.b, sh.g, row, D, p.qs) : 0));
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<uint4*>(dst + (c / 8) * (128 * 128) + (((c % 8) ^ (r & 7)) * 16)) =
            live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      fence_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
    const uint64_t seen = nodes_seen(p, sh.b, sh.count, live ? row / p.G : -1);

    float m = -INFINITY, l = 0.f;  // m: the reference, scaled by log2(e)
    for (int j = TWO ? 0 : stream; j < sh.n; j += TWO ? 1 : 2) {
      wait(&sm.s_full[stream], s_uses++);
      tc_fence_after();
      if (warp_live) {
        uint32_t x[kKeys];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load32(t_s + 32 * c, x + 32 * c);
        const uint4 there = *reinterpret_cast<const uint4*>(sm.mask[(tile_no + j) % kMasks]);
        const int off = sh.start - (sh.k0 + j) * kKeys;  // first node's place in the tile
        tmem_wait_ld();
        if ((there.x & there.y & there.z & there.w) != 0xffffffffu || off < kKeys) {
          // context keys below `off`, then the nodes that the row sees
          uint64_t lo, hi;
          if (off >= 128) lo = hi = ~0ull;
          else if (off >= 64) {
            lo = ~0ull;
            hi = off == 64 ? seen : ((1ull << (off - 64)) - 1) | seen << (off - 64);
          } else if (off > 0) {
            lo = ((1ull << off) - 1) | seen << off;
            hi = seen >> (64 - off);
          } else {
            lo = off > -64 ? seen >> -off : 0;
            hi = 0;
          }
          const uint32_t see[4] = {(uint32_t)lo & there.x, (uint32_t)(lo >> 32) & there.y,
                                   (uint32_t)hi & there.z, (uint32_t)(hi >> 32) & there.w};
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (!(see[c / 32] >> (c % 32) & 1)) x[c] = 0xff800000u;  // -inf
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) top = fmaxf(top, __uint_as_float(x[c]));
        top *= p.scale_log2;
        float keep = 1.f;
        if (top > m + kSlack || m == -INFINITY) {
          keep = fast_exp2(m - top);  // 0 at the first key
          if (m == -INFINITY) keep = 0.f;
          m = top;
          l *= keep;
        }
        const int before = TWO ? j : j / 2;  // tiles already in O
        if (before > 0 && __any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_load32(t_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
            tmem_store32(t_o + c, o);
          }
        }
        const float from = m == -INFINITY ? 0.f : -m;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float a = fast_exp2(fmaf(__uint_as_float(x[64 * h + 2 * c]), p.scale_log2, from));
            const float b = fast_exp2(fmaf(__uint_as_float(x[64 * h + 2 * c + 1]), p.scale_log2, from));
            l += a + b;
            w[c] = bf16x2_rn(a, b);
          }
          tmem_store32(t_s + 32 * h, w);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[stream]);
    }
    tile_no += sh.n;

    // ---- the share's rows
    if (!TWO && stream == 1) {
      sm.ml[r][0] = m;
      sm.ml[r][1] = l;
    }
    wait(&sm.o_full, share);
    tc_fence_after();
    if (!TWO) named_bar(1, 32 * kSoftWarps);
    const bool writes = TWO || stream == 0;
    if (writes && warp_live) {
      float f0 = 1.f, f1 = 0.f;  // factors of the streams' shares (one row block)
      float l1 = 0.f;
      if (!TWO) {
        const float m1 = sm.ml[r][0];
        l1 = sm.ml[r][1];
        const float both = fmaxf(m, m1);
        f0 = l == 0.f ? 0.f : fast_exp2(m - both);
        f1 = l1 == 0.f ? 0.f : fast_exp2(m1 - both);
        l = (l == 0.f ? 0.f : l * f0) + (l1 == 0.f ? 0.f : l1 * f1);
        m = both;
      }
      if (*reinterpret_cast<volatile int*>(&sm.failed)) l = NAN;
      const bool any0 = TWO ? l != 0.f : true, any1 = !TWO && sh.n > 1;
      const bool whole = sh.n == sh.nt;
      const float scale = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const uint32_t odd = sm.odd[share & 1];
      const size_t slot = part_slot(p, group, sh.begins, rt) * p.row_tile + local;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32], o1[32];
        tmem_load32(t_o + c, o);
        if (!TWO && any1) tmem_load32(t_o + D + c, o1);
        tmem_wait_ld();
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          y[e] = any0 && f0 != 0.f ? __uint_as_float(o[e]) * f0 : 0.f;
          if (!TWO && any1 && f1 != 0.f) y[e] += __uint_as_float(o1[e]) * f1;
        }
        if (odd) {
          for (uint64_t left = seen; left; left &= left - 1) {
            const int node = __ffsll((long long)left) - 1;
            const uint32_t up = sm.odd_at[share & 1][node][0][c / 32];
            const uint32_t down = sm.odd_at[share & 1][node][1][c / 32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (up >> e & 1) y[e] += INFINITY;
              if (down >> e & 1) y[e] -= INFINITY;
            }
          }
        }
        if (live && whole) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            w[e] = bf16x2_rn(y[2 * e] * scale, y[2 * e + 1] * scale);
            if (l == 0.f) w[e] = 0;  // no key seen
          }
          uint4* dst = reinterpret_cast<uint4*>((uint16_t*)p.out +
                                                row_offset(p, sh.b, sh.g, row, D, p.os) + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + slot * D + c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        }
        __syncwarp();
      }
      if (live && !whole) {
        p.part_ml[slot * 2] = m;
        p.part_ml[slot * 2 + 1] = l;
      }
    }
    // The list of odd values is cleared for the share after next, O may be
    // overwritten. (All of a stream's readers of the list are behind this
    // barrier.)
    named_bar(1, 32 * kSoftWarps);
    if (sm.odd[share & 1]) {
      for (int i = threadIdx.x; i < MK_MAX_TREE * 8; i += 32 * kSoftWarps)
        (&sm.odd_at[share & 1][0][0][0])[i] = 0;
      named_bar(1, 32 * kSoftWarps);
      if (threadIdx.x == 0) sm.odd[share & 1] = 0;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.done[share & 1]);
    ++share;
  }
}

template <int D, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_tc_kernel(const __grid_constant__ AttnParams p) {
  using Lay = Layout<D, TWO>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sm;
  __shared__ int prefix[kMaxSeqs + 1];
  const int warp = threadIdx.x / 32;
  const int rt = blockIdx.x % p.row_tiles, group = blockIdx.x / p.row_tiles;
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* ring_ptr = base + Lay::kQ;

  griddep_launch();
  if (warp == 0) work_line(p, prefix);
  if (warp == 1 && threadIdx.x % 32 == 0) {
    for (int i = 0; i < Lay::kBufs; ++i) {
      mbar_init(&sm.full[i], kLoadThreads + kLoadWarps);
      mbar_init(&sm.empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 2);
      mbar_init(&sm.p_full[s], 4);
      mbar_init(&sm.done[s], kSoftWarps);
      sm.odd[s] = 0;
    }
    mbar_init(&sm.q_full, kSoftWarps);
    mbar_init(&sm.o_full, 2);
    sm.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&sm.tmem), 512);
  for (int i = threadIdx.x; i < 2 * MK_MAX_TREE * 8; i += kThreads) (&sm.odd_at[0][0][0][0])[i] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const Cut cut(prefix[p.B], p.groups);
  const int u_begin = cut.begin(group), u_end = cut.begin(group + 1);

  // 12 warps launched with 168 registers each: 8 x 208 + 4 x 88 is the same sum
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp >= kLoadWarp)
      load_role<D, TWO>(p, sm, prefix, smem_u32(ring_ptr), ring_ptr, u_begin, u_end, rt);
    else if (threadIdx.x % 32 == 0)
      mma_role<D, TWO>(p, sm, prefix, smem_u32(base), smem_u32(ring_ptr), tmem, u_begin, u_end, rt);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax_role<D, TWO>(p, sm, prefix, base, tmem, u_begin, u_end, rt, group);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

template <int D, bool TWO>
int launch(const AttnParams& p, cudaStream_t st) {
  using Lay = Layout<D, TWO>;
  auto* fn = tree_attention_tc_kernel<D, TWO>;
  static std::atomic<uint64_t> ready{0};
  if (int rc = allow_shared(ready, (const void*)fn, Lay::kBytes)) return rc;
  fn<<<p.groups * p.row_tiles, kThreads, Lay::kBytes, st>>>(p);
  return op_cuda(cudaGetLastError(), "mk_tree_attention");
}

}  // namespace

int launch_tree_attention_tc(const AttnParams& p, int head_dim, cudaStream_t st) {
  const bool two = p.row_tile > 128;
  if (head_dim == 64) return two ? launch<64, true>(p, st) : launch<64, false>(p, st);
  return two ? launch<128, true>(p, st) : launch<128, false>(p, st);
}

}  // namespace mk
