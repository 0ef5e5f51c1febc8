// Attention of a tree of drafted tokens (include/mk.h, mk_tree_attention): the
// kernel for many rows, on the tensor-memory matrix unit.
//
// One block per SM, sixteen warps in warpgroups of four:
//   warps 0-3, 4-7  softmax of stream 0 and 1, one thread per row; fp32: of
//                   the halves of the rows
//   warps 8-11      load the key and value tiles (128 keys each, 32 per warp)
//   warp 12         one thread issues every product (13-15 idle)
// bf16 activations. With two row blocks stream s is the rows of block s, over
// every tile; with one, both streams take the same rows, stream s the tiles of
// parity s, and stream 0 joins the two at the end. Either way one stream's
// softmax runs while the matrix unit works for the other. Per stream and tile:
// S = Q K^T (128 x 128, fp32, tensor memory); the row's thread reads it, masks
// it, and writes the weights p = 2^(s - m) back over S as two bf16 parts, which are
// p to 2^-16 (as the decode step holds its own; with one part, 2^-9, the output
// was 1.2 to 1.4 times as far from 64 bits as its rounding); O += P V (128 x D, fp32,
// tensor memory), once per part. The reference m of a row follows its maximum
// only when that exceeds it by 2^8 (or at the first key), so O is almost never
// rescaled; the sum of the weights is kept in fp32 from the unrounded weights.
//
// fp32 activations. Queries and weights go in as three bf16 parts (2^-24 of the
// value), each product runs once per part; up to 32 rows stand three times in the
// block, each time with another part of the weights, so that the weights' products
// run once. The matrix unit truncates as it
// accumulates, which over a long context costs more than fp32's own rounding, so
// it sums one tile only (two score buffers, one product) and the rows' threads
// add the tiles up in registers. (Accumulated in tensor memory the error against
// 64 bits was 2.5e-6 on 10 thousand keys, twice that of a plain fp32
// computation.)
//
// K and V tiles go through a ring of 16 or 32 KB buffers in the order the
// products use them, with 16-byte asynchronous copies, so that any page size,
// rows that are not there (zeroed) and odd starts need nothing special; they
// lie in the 128-byte-swizzled form in which the matrix unit reads K by rows and
// V by columns.
//
// Measured, 8 sequences over 16384 keys each, 8B shape (537 MB): bf16 with 64 rows 98
// us, 5.5 TB/s, bound by the bytes; with 256 rows 168 us, 3.2 TB/s and 1.23 PFLOP/s of
// both parts' products. Its tiles are bound by the products, with which stores and
// softmax overlap in part: 4660 cycles or 2.44 us a tile of both streams, 1.57 PFLOP/s
// at the power limit (a plain library product sustains 1.71); 3950 cycles without
// the second parts' products, 4100 without their stores. fp32 with 32 rows 111 us, with
// 256 rows 265 us (in bf16 parts 1.6 PFLOP/s).
//
// Every wait ends: after kWaitNs and a last try of kLastTryNs a thread stops waiting
// for good and goes on, the rows of the block come out as NaN, and the block ends
// when its copies and products in flight have.
//
// P is the call: AttnParams or PrefixParams (mk_prefix_attention.cu), which bring their
// line of work (P::Line, work_line, all_places, next_share, put_plans) and say where a share's keys and rows
// are: first_slot, first_row, row_there, row_node, row_offset, is_final, share_slot.
#pragma once

#include <type_traits>

#include "mk_tree_attention.cuh"

namespace mk {
namespace {

constexpr int kSoftWarps = 8, kLoadWarp = 8, kLoadWarps = 4, kMmaWarp = 12;
constexpr int kThreads = 512;

constexpr int kMasks = 8;           // tiles whose masks are kept
constexpr uint64_t kWaitNs = 2000000000ull;
// The clock goes on while a block is off its SM (another process's turn), and what
// the block waits for went no further either: time for that behind the limit.
constexpr uint32_t kLastTryNs = 20000000;
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
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// Waits for the loads; r (n of what they load) is not to be used before.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory operand of 128-byte swizzled rows (64 bf16 each, groups of eight
// rows 1024 bytes apart). Read by rows (K-major) `lead` is unused; read by
// columns (MN-major) it is the distance of the next 64 columns. The address
// field counts 16-byte units: a place inside the tile is an addition to it.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return (uint64_t)(addr >> 4 | (lead >> 4) << 16) | (uint64_t)(1024 >> 4 | 1u << 14 | 2u << 29) << 32;
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

// one thread of a converged warp (the products' operands live in uniform
// registers: code that a whole warp runs up to this choice computes them there)
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
// the largest of three (a NaN loses against a number)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// a += b, lane by lane
__device__ __forceinline__ void add2(unsigned long long& a, unsigned long long b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
}

// arrives when this thread's earlier asynchronous copies have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Kinds of call: bf16 with one or two row blocks, fp32 with up to 128 or 32 rows.
enum { kOne, kTwo, kExact, kFew };

constexpr int kKeys = 128;  // keys of a tile

// Columns of tensor memory (512): kOne, kTwo: scores (the two parts of the weights
// over them) of stream s at 128 s, its output at 256 + D s. kExact: scores of tile
// parity s, the three parts of the weights over them, at 192 s, a tile's product at
// 384. kFew: scores (weights over them) of tile parity s at 128 s, the tile's
// product at 256 + D s.
template <int D, int KIND>
struct Layout {
  static constexpr bool TWO = KIND == kTwo;
  static constexpr bool EXACT = KIND == kExact || KIND == kFew;
  static constexpr int PARTS = EXACT ? 3 : 1;             // of the queries
  static constexpr int WEIGHT_PARTS = KIND == kExact ? 3 : KIND == kFew ? 1 : 2;  // one after another
  static constexpr int PRODUCTS = KIND == kExact ? 1 : 2;      // outputs or products
  static constexpr int kScoreStep = KIND == kExact ? 192 : 128;
  static constexpr int kOut = 2 * kScoreStep;
  static constexpr int kBuf = kKeys * D * 2;  // a K or V tile
  static constexpr int kBufs = D == 64 ? 8 : TWO ? 4 : KIND == kOne ? 5 : 3;
  static constexpr int kQ = (TWO ? 2 : PARTS) * 128 * D * 2;
  static constexpr int kBytes = kQ + kBufs * kBuf + 1024;  // 1024: alignment of the base
};

// Whether a share's rows are two blocks, a stream each. A call may mix shares of both kinds (P::kMixed):
// kTwo's shares of up to 128 rows are then taken as kOne's are.
template <int KIND, class P>
__device__ __forceinline__ bool two_blocks(const typename P::Share& sh) {
  if constexpr (KIND != kTwo) return false;
  else if constexpr (P::kMixed) return sh.rows - first_row(sh) > 128;
  else return true;
}

struct Shared {
  uint64_t full[8], empty[8];
  uint64_t s_full[2];              // a stream's scores are in tensor memory
  uint64_t p_full[2][2];           // the weights of a stream's first, last 64 keys are
  uint64_t q_full, o_full;         // a share's queries are loaded / its products done
  uint64_t drained;                // every product of the block is done
  uint64_t done[2];                // a share (by parity) is written
  uint32_t tmem;
  int failed;                      // a wait ran out
  alignas(16) uint32_t mask[kMasks][4];  // keys of a tile that are there
  // non-finite values of the nodes' v rows (share parity): +inf in [0], -inf in
  // [1], NaN in both; odd: whether there are any
  uint32_t odd[2];
  uint32_t odd_at[2][MK_MAX_TREE][2][4];
  float ml[128][2];                // kOne: stream 1's (m, l)
  float run_m[2][128];             // RUNS: the reference of a stream's earlier runs
  // fp32: a tile's product is in tensor memory / has been read; the halves'
  // maxima (by tile parity) and sums
  uint64_t t_full[2], t_free[2];
  float top[2][2][128], sum[2][128];
};

// mbar_try_wait that may suspend the thread for up to about `ns`
__device__ __forceinline__ bool mbar_try_wait_for(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
      : "memory");
  return done != 0;
}

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
      if (globaltimer() - since > kWaitNs && !mbar_try_wait_for(bar, parity & 1, kLastTryNs)) {
        ok = false;
        *reinterpret_cast<volatile int*>(&sm.failed) = 1;
        return;
      }
    }
  }
};

// ---- the loading warps -------------------------------------------------------------

// Warp w of the four takes a quarter of every tile's keys: lane i finds the row of
// the quarter's key i, the copies take it by a shuffle.
template <int D, int KIND, class P>
__device__ __forceinline__ void load_role(const P& p, Shared& sm, const typename P::Line& line,
                                          uint32_t ring, uint8_t* ring_ptr, int u_begin, int u_end,
                                          int rt) {
  using Lay = Layout<D, KIND>;
  constexpr int CPR = D / 8, RPW = 32 / CPR;
  constexpr int kLoadRows = kKeys / kLoadWarps;  // keys of a tile that a warp takes
  const int lw = threadIdx.x / 32 - kLoadWarp, lane = threadIdx.x % 32;
  const int c = lane % CPR, r_first = lw * kLoadRows + lane / CPR;
  Waiter wait(sm);
  uint32_t buf = 0, round = 0;           // next buffer of the ring, its round
  uint32_t tile_no = 0;                  // K tiles loaded so far
  int u = u_begin;
  typename P::Share sh;
  for (uint32_t share = 0; next_share(p, line, u_begin, u_end, u, sh);) {
    if (rt * p.row_tile >= sh.rows) continue;
    auto row_of = [&](int t) -> uint32_t {
      const int slot = first_slot(sh) + (sh.k0 + t) * kKeys + lw * kLoadRows + lane;
      if (t >= sh.n || slot >= sh.len) return kNoRow;
      const uint32_t row = cache_row(p.cache, sh.b, slot);
      return row == kNoRow ? row : row + (uint32_t)sh.g * p.cache.block_size;
    };
    const bool two = two_blocks<KIND, P>(sh);
    const int lead = two ? 1 : 2;          // K tiles ahead of V
    // rows of the tile whose K is next, of the `lead` tiles before it (V is to come)
    uint32_t next = row_of(0), held[2] = {};

    auto copy = [&](const uint16_t* pool, uint32_t rows) {
      const uint32_t base = ring + buf * Lay::kBuf + (c / 8) * (kKeys * 128);
      const uint16_t* from = pool + 8 * c;
      if (__all_sync(0xffffffffu, rows != kNoRow)) {
#pragma unroll
        for (int i = 0; i < kLoadRows / RPW; ++i) {
          const uint32_t row = __shfl_sync(0xffffffffu, rows, i * RPW + lane / CPR);
          const int r = r_first + i * RPW;
          cp_async16(base + r * 128 + (((c % 8) ^ (r & 7)) * 16), from + (size_t)row * D);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kLoadRows / RPW; ++i) {
          const uint32_t row = __shfl_sync(0xffffffffu, rows, i * RPW + lane / CPR);
          const bool there = row != kNoRow;
          const int r = r_first + i * RPW;
          cp_async16(base + r * 128 + (((c % 8) ^ (r & 7)) * 16),
                     from + (there ? (size_t)row * D : 0), there ? 16 : 0);
        }
      }
    };
    auto advance = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.full[buf]);
      if (++buf == Lay::kBufs) buf = 0, ++round;
    };

    for (int j = -lead; j < sh.n; ++j) {
      if (j >= 0) {
        // the share's list of odd values is free again (the share before last is
        // written). For every share, whether it has odd values or not: a parity tells
        // only neighbouring phases apart, so none may be passed over.
        if (j == 0 && share >= 2) wait(&sm.done[share & 1], share / 2 - 1);
        wait(&sm.empty[buf], round + 1);
        const uint32_t rows = held[0];
        copy(p.v, rows);
        const int slot0 = first_slot(sh) + (sh.k0 + j) * kKeys;
        if (slot0 + kKeys > sh.start) {
          // nodes in the tile: a value that some rows must not see is not
          // cancelled by a zero weight if it is not finite, so it is taken out
          // here and added at the end to the rows that see it
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
          uint8_t* base = ring_ptr + buf * Lay::kBuf + (c / 8) * (kKeys * 128);
          for (int i = 0; i < kLoadRows / RPW; ++i) {
            const uint32_t row = __shfl_sync(0xffffffffu, rows, i * RPW + lane / CPR);
            const int r = r_first + i * RPW, node = slot0 + r - sh.start;
            if (node < 0 || node >= sh.count || row == kNoRow) continue;
            uint16_t* x = reinterpret_cast<uint16_t*>(base + r * 128 + (((c % 8) ^ (r & 7)) * 16));
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
        advance();
      }
      if (!two) held[0] = held[1];
      if (const int t = j + lead; t < sh.n) {
        const uint32_t there = __ballot_sync(0xffffffffu, next != kNoRow);
        wait(&sm.empty[buf], round + 1);
        if (lane == 0) sm.mask[tile_no % kMasks][lw] = there;
        copy(p.k, next);
        cp_async_arrive(&sm.full[buf]);
        advance();
        ++tile_no;
        if (two) held[0] = next;
        else held[1] = next;
        next = row_of(t + 1);
      }
    }
    ++share;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- the issuing warp ------------------------------------------------------------------
// The whole warp runs the loops and waits; one elected thread issues. (Issued from
// a branch on the thread's number a product took about 100 cycles, its operands
// being moved to uniform registers one by one; so it takes the 64 of the unit.)
// Products run in the order of their issue, so the scores of a stream's next tile
// may be issued over the weights that its last products read.

template <int D, int KIND, bool RUNS, class P>
__device__ __forceinline__ void mma_role(const P& p, Shared& sm, const typename P::Line& line,
                                         uint32_t q_smem, uint32_t ring, uint32_t tmem, int u_begin,
                                         int u_end, int rt) {
  using Lay = Layout<D, KIND>;
  constexpr uint32_t kScores = instruction(kKeys, false), kValues = instruction(D, true);
  Waiter wait(sm);
  uint32_t buf = 0, round = 0;
  uint32_t p_uses[2] = {0, 0};
  uint32_t t_uses[2] = {0, 0};
  int u = u_begin;
  typename P::Share sh;
  // S of stream s from the K tile in buffer `at`; free: it is not needed again
  bool two = false;  // of the share
  // whether tile `i` of a stream adds to what is in tensor memory
  auto goes_on = [](int i) { return RUNS ? i % kRun != 0 : i > 0; };
  auto scores = [&](int s, uint32_t at, bool free) {
    if (elect_one()) {
      const uint64_t k = operand(ring + at * Lay::kBuf, 16);
      const uint64_t q = operand(q_smem + (two ? s * 128 * D * 2 : 0), 16);
#pragma unroll
      for (int part = Lay::PARTS - 1; part >= 0; --part)  // the smallest part first
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_smem(tmem + s * Lay::kScoreStep,
                   q + (part * 128 * D * 2 + (i / 4) * (128 * 128) + (i % 4) * 32) / 16,
                   k + ((i / 4) * (kKeys * 128) + (i % 4) * 32) / 16, kScores,
                   part < Lay::PARTS - 1 || i > 0);
      tc_commit(&sm.s_full[s]);
      mbar_arrive(&sm.s_full[s]);  // hands on the tile's mask
      if (free) tc_commit(&sm.empty[at]);
    }
    __syncwarp();
  };
  // Weights of stream (fp32: tile parity) s times the V tile in buffer `at`: into
  // the stream's output (add: to what is there), fp32: into the tile's product
  auto values = [&](int s, uint32_t at, bool add, bool free) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      wait(&sm.p_full[s][h], p_uses[s]);
      if (Lay::EXACT && h == 0) {
        wait(&sm.t_free[s % Lay::PRODUCTS], t_uses[s % Lay::PRODUCTS] + 1);
        ++t_uses[s % Lay::PRODUCTS];
      }
      tc_fence_after();
      if (elect_one()) {
        const uint64_t v = operand(ring + at * Lay::kBuf, kKeys * 128);
#pragma unroll
        for (int part = Lay::WEIGHT_PARTS - 1; part >= 0; --part)
#pragma unroll
          for (int i = 4 * h; i < 4 * h + 4; ++i)
            mma_tmem(tmem + Lay::kOut + s % Lay::PRODUCTS * D,
                     tmem + s * Lay::kScoreStep + part * 64 + i * 8, v + i * (2048 / 16), kValues,
                     h > 0 || part < Lay::WEIGHT_PARTS - 1 || i > 0 ? 1u : add);
        if (h == 1) {
          if (free) tc_commit(&sm.empty[at]);
          if (Lay::EXACT) {
            tc_commit(&sm.t_full[s % Lay::PRODUCTS]);
            mbar_arrive(&sm.t_full[s % Lay::PRODUCTS]);  // hands on the tile's odd values
          }
        }
      }
      __syncwarp();
    }
    ++p_uses[s];
  };
  // Waits for the next buffer of the ring and moves behind it. The copies wrote it
  // through the generic proxy, the products read it through the asynchronous one.
  auto take = [&]() -> uint32_t {
    wait(&sm.full[buf], round);
    fence_async_smem();
    const uint32_t at = buf;
    if (++buf == Lay::kBufs) buf = 0, ++round;
    return at;
  };
  for (uint32_t share = 0; next_share(p, line, u_begin, u_end, u, sh);) {
    if (rt * p.row_tile >= sh.rows) continue;
    wait(&sm.q_full, share);
    fence_async_smem();
    tc_fence_after();
    two = two_blocks<KIND, P>(sh);
    if (two) {
      uint32_t k_at = take(), v_at = 0;
#pragma unroll 1
      for (int i = -2; i < 2 * sh.n; ++i) {  // stream i & 1: products of tile i / 2, then the next scores
        const int s = i & 1;
        if (i >= 0) {
          if (s == 0) v_at = take();
          values(s, v_at, goes_on(i / 2), s == 1);
          if (s == 0 && i + 2 < 2 * sh.n) k_at = take();
        }
        if (i + 2 < 2 * sh.n) scores(s, k_at, s == 1);
      }
    } else {
      for (int s = 0; s < 2 && s < sh.n; ++s) scores(s, take(), true);
      for (int j = 0; j < sh.n; ++j) {
        const int s = j & 1;
        values(s, take(), !Lay::EXACT && goes_on(j / 2), true);
        if (j + 2 < sh.n) scores(s, take(), true);
      }
    }
    if (!Lay::EXACT && elect_one()) {
      tc_commit(&sm.o_full);
      mbar_arrive(&sm.o_full);
    }
    __syncwarp();
    ++share;
  }
  // Products may be in flight yet where a wait ran out (else the rows' threads have
  // waited for them): the tensor memory is given back behind them. The wait runs
  // beside the writing of the last rows.
  if (elect_one()) tc_commit(&sm.drained);
  __syncwarp();
  Waiter last(sm);
  last(&sm.drained, 0);
}

// ---- the softmax warps -------------------------------------------------------------------

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int from) {
  return __shfl_sync(0xffffffffu, v, from);
}

// The nodes that node `t` sees (t < 64, -1: none), by doubling inside the warp:
// lane l holds nodes l and l + 32, `up` the next ancestor behind `seen`.
__device__ __forceinline__ uint64_t nodes_seen(const AttnParams& p, int b, int count, int t) {
  if (count <= 1) return t == 0 ? 1 : 0;  // no tree: nothing to read
  if (!p.parents) return t < 0 ? 0 : (2ull << t) - 1;
  const int lane = threadIdx.x % 32;
  uint64_t seen[2];
  int up[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = lane + 32 * h;
    int x = -1;
    if (n < count) {
      x = __ldg(p.parents + (size_t)b * p.T + n);
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

// The queries of rows `row` to `row` + n - 1 into rows 0 to n - 1 of a block of shared memory
// (COPIES of them, 32 rows apart), swizzled, in PARTS bf16 parts, by THREADS threads
// of which this is number `tid`: lanes that follow one another take 16 bytes that do (a row
// for each thread took 3200 cycles, of a few rows as of 128). Rows that are not there keep
// what the block held: what comes of them goes nowhere.
template <int D, int PARTS, int COPIES, int THREADS, class P>
__device__ __forceinline__ void load_queries(const P& p, const typename P::Line& line,
                                             const typename P::Share& sh, int row, int n, int tid,
                                             uint8_t* block) {
  constexpr int CPR = D / 8;
  auto place = [](int r, int c) { return r * 128 + (c / 8) * (128 * 128) + (((c % 8) ^ (r & 7)) * 16); };
  if constexpr (PARTS == 1) {
    const uint32_t to = smem_u32(block);
    for (int i = tid; i < n * CPR; i += THREADS) {
      const int r = i / CPR, c = i % CPR;
      if (row_there(p, line, sh, row + r))
        cp_async16(to + place(r, c), (const uint16_t*)p.q + row_offset(p, sh, row + r, D, p.qs) + 8 * c);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    constexpr int U = COPIES == 1 ? 2 : 1;  // pieces in flight
    for (int i0 = tid; i0 < n * CPR; i0 += U * THREADS) {
      uint4 w[U][2];
      bool there[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * THREADS, r = i / CPR;
        there[u] = i < n * CPR && row_there(p, line, sh, row + r);
        if (!there[u]) continue;
        const float* src = (const float*)p.q + row_offset(p, sh, row + r, D, p.qs) + 8 * (i % CPR);
        w[u][0] = __ldg(reinterpret_cast<const uint4*>(src));
        w[u][1] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!there[u]) continue;
        const int i = i0 + u * THREADS;
        uint32_t part[4][PARTS];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          split(__uint_as_float(w[u][h].x), __uint_as_float(w[u][h].y), part[2 * h]);
          split(__uint_as_float(w[u][h].z), __uint_as_float(w[u][h].w), part[2 * h + 1]);
        }
#pragma unroll
        for (int k = 0; k < COPIES; ++k)
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            *reinterpret_cast<uint4*>(block + place(i / CPR + 32 * k, i % CPR) + q * 128 * D * 2) =
                make_uint4(part[0][q], part[1][q], part[2][q], part[3][q]);
      }
    }
  }
  fence_async_smem();
}

// What a row sees of a tile: the context keys below `off` (the first node's place
// in the tile), the nodes of `seen`, of the keys that are there.
struct Sight {
  bool some;  // not simply all
  uint32_t bits[4];
};
__device__ __forceinline__ Sight sight_of(const uint32_t (&mask)[4], int off, uint64_t seen) {
  const uint4 there = *reinterpret_cast<const uint4*>(mask);
  Sight v;
  v.some = (there.x & there.y & there.z & there.w) != 0xffffffffu || off < kKeys;
  v.bits[0] = v.bits[1] = v.bits[2] = v.bits[3] = ~0u;
  if (v.some) {
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
    v.bits[0] = (uint32_t)lo & there.x, v.bits[1] = (uint32_t)(lo >> 32) & there.y;
    v.bits[2] = (uint32_t)hi & there.z, v.bits[3] = (uint32_t)(hi >> 32) & there.w;
  }
  return v;
}

// Reads N scores of the lane's row, those it does not see (bits) as -inf, and
// returns their maximum.
template <int N>
__device__ __forceinline__ float read_scores(uint32_t at, bool some, const uint32_t* bits,
                                             uint32_t (&x)[N]) {
#pragma unroll
  for (int h = 0; h < N / 32; ++h) tmem_load32(at + 32 * h, x + 32 * h);
  tmem_wait_ld<N>(x);
  if (some) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!(bits[e / 32] >> (e % 32) & 1)) x[e] = 0xff800000u;  // -inf
  }
  float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < N; e += 8)
#pragma unroll
    for (int h = 0; h < 4; ++h)
      tops[h] = max3(tops[h], __uint_as_float(x[e + 2 * h]), __uint_as_float(x[e + 2 * h + 1]));
  return fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
}

// Moves the reference m where the tile's maximum asks for it and returns the
// factor of what was summed under the old one.
__device__ __forceinline__ float move_reference(float top, float& m, float& l) {
  if (!(top > m + kSlack) && m != -INFINITY) return 1.f;
  const float keep = m == -INFINITY ? 0.f : fast_exp2(m - top);  // 0 at the first key
  m = top;
  l *= keep;
  return keep;
}

// The weights of two neighbouring keys, added to the sum
__device__ __forceinline__ float2 weights2(uint32_t a, uint32_t b, unsigned long long scale2,
                                           unsigned long long from2, unsigned long long& sum) {
  unsigned long long z = from2;
  ffma2(z, pack2(__uint_as_float(a), __uint_as_float(b)), scale2);
  float2 w = unpack2(z);
  w.x = fast_exp2(w.x);
  w.y = fast_exp2(w.y);
  add2(sum, pack2(w.x, w.y));
  return w;
}

// Part q of two weights (not negative; a NaN stays one), as bf16: the upper 8 bits of the
// significand, the next 8, the last 8, so that the three parts' sum is the weight.
template <int q>
__device__ __forceinline__ uint32_t weight_part(float2 w) {
  constexpr uint32_t kUpTo = q == 0 ? ~0u : q == 1 ? 0xffffff00u : ~0u, kFrom = q == 1 ? 0xffff0000u : 0xffffff00u;
  uint32_t x = __float_as_uint(w.x), y = __float_as_uint(w.y);
  if (q > 0) {
    unsigned long long part = pack2(__uint_as_float(x & kUpTo), __uint_as_float(y & kUpTo));
    add2(part, pack2(-__uint_as_float(x & kFrom), -__uint_as_float(y & kFrom)));
    const float2 z = unpack2(part);
    x = __float_as_uint(z.x), y = __float_as_uint(z.y);
  }
  return __byte_perm(x, y, 0x7632);  // the upper halves
}
// What part 0 leaves of two weights, rounded to bf16: with part 0 the weight to
// 2^-16 of it.
__device__ __forceinline__ uint32_t weight_rest(float2 w) {
  const uint32_t x = __float_as_uint(w.x), y = __float_as_uint(w.y);
  unsigned long long rest = pack2(w.x, w.y);
  add2(rest, pack2(-__uint_as_float(x & 0xffff0000u), -__uint_as_float(y & 0xffff0000u)));
  const float2 z = unpack2(rest);
  return bf16x2_rn(z.x, z.y);
}

// 32 columns of a finished row: the odd values it sees added, then written out
// (whole: divided by the sum, in the type of the call) or to the workspace.
template <int D, int PARTS, class P>
__device__ __forceinline__ void put_columns(const P& p, const typename P::Share& sh, const Shared& sm,
                                            uint32_t share, uint64_t seen, int row, int c, bool live,
                                            float l, size_t slot, float (&y)[32]) {
  if (sm.odd[share & 1]) {
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
  if (live && is_final(sh)) {
    const int64_t off = row_offset(p, sh, row, D, p.os) + c;
    const float scale = 1.f / l;
#pragma unroll
    for (int e = 0; e < 32; ++e) y[e] = l == 0.f ? 0.f : y[e] * scale;  // 0: no key seen
    if constexpr (PARTS > 1) {
      float4* dst = reinterpret_cast<float4*>((float*)p.out + off);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    } else {
      uint4* dst = reinterpret_cast<uint4*>((uint16_t*)p.out + off);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        dst[e] = make_uint4(bf16x2_rn(y[8 * e], y[8 * e + 1]), bf16x2_rn(y[8 * e + 2], y[8 * e + 3]),
                            bf16x2_rn(y[8 * e + 4], y[8 * e + 5]), bf16x2_rn(y[8 * e + 6], y[8 * e + 7]));
    }
  } else if (live) {
    int step;
    float4* dst = part_place(p, slot, D, c, step);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      dst[e / 2 * step + e % 2] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
  }
  __syncwarp();
}

// The end of a share, for the eight warps of the rows: the list of odd values is
// cleared for the share after next, and what the share used is free again.
__device__ __forceinline__ void end_share(Shared& sm, uint32_t share) {
  named_bar(1, 32 * kSoftWarps);
  if (sm.odd[share & 1]) {
    for (int i = threadIdx.x; i < MK_MAX_TREE * 8; i += 32 * kSoftWarps)
      (&sm.odd_at[share & 1][0][0][0])[i] = 0;
    named_bar(1, 32 * kSoftWarps);
    if (threadIdx.x == 0) sm.odd[share & 1] = 0;
  }
  tc_fence_before();
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(&sm.done[share & 1]);
}

__device__ __forceinline__ bool wait_failed(Shared& sm) {
  return *reinterpret_cast<volatile int*>(&sm.failed) != 0;
}

// kOne, kTwo: softmax of a stream.
template <int D, int KIND, bool RUNS, class P>
__device__ __forceinline__ void softmax_role(const P& p, Shared& sm, const typename P::Line& line,
                                             uint8_t* q_ptr, uint32_t tmem, int u_begin,
                                             int u_end, int rt, int group) {
  using Lay = Layout<D, KIND>;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int stream = warp / 4, r = (warp % 4) * 32 + lane;  // row of the stream's block
  const uint32_t lanes = (uint32_t)(warp % 4) * 32 << 16;
  const uint32_t t_s = tmem + lanes + stream * Lay::kScoreStep;
  const uint32_t t_o = tmem + lanes + Lay::kOut + stream * D;
  const unsigned long long scale2 = pack2(p.scale_log2, p.scale_log2);
  // What is in tensor memory and the sums of the runs before it (some), added up relative to
  // m: to where those are (keep) or to tensor memory.
  auto end_run = [&](float m, bool some, bool keep) {
    const float from = some ? sm.run_m[stream][r] : m, back = from == m ? 1.f : fast_exp2(from - m);
    if (keep) sm.run_m[stream][r] = m;
    float4* runs = p.runs + ((size_t)blockIdx.x * 2 + stream) * (D / 4) * 128 + r;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      tmem_load32(t_o + c, o);
      tmem_wait_ld<32>(o);
#pragma unroll
      for (int e = 0; e < 32; e += 4, runs += 128) {
        float4 y = {};
        if (some) y = *runs;
        y.x = fmaf(y.x, back, __uint_as_float(o[e]));
        y.y = fmaf(y.y, back, __uint_as_float(o[e + 1]));
        y.z = fmaf(y.z, back, __uint_as_float(o[e + 2]));
        y.w = fmaf(y.w, back, __uint_as_float(o[e + 3]));
        if (keep) {
          *runs = y;
        } else {
          o[e] = __float_as_uint(y.x), o[e + 1] = __float_as_uint(y.y);
          o[e + 2] = __float_as_uint(y.z), o[e + 3] = __float_as_uint(y.w);
        }
      }
      if (!keep) tmem_store32(t_o + c, o);
    }
    if (!keep) tmem_wait_st();
    __syncwarp();
  };
  Waiter wait(sm);
  uint32_t s_uses = 0, tile_no = 0;
  int u = u_begin;
  typename P::Share sh;
  for (uint32_t share = 0; next_share(p, line, u_begin, u_end, u, sh);) {
    if (rt * p.row_tile >= sh.rows) continue;
    const bool two = two_blocks<KIND, P>(sh);
    const int block_rows = two ? p.row_tile / 2 : 128;       // rows of a stream's block
    const int local = two ? stream * block_rows + r : r;     // row of the row tile
    const int row = first_row(sh) + rt * p.row_tile + local;
    const bool live = r < block_rows && row_there(p, line, sh, row);
    const bool warp_live = __any_sync(0xffffffffu, live);
    if (two)
      load_queries<D, 1, 1, 128>(p, line, sh, row - r, block_rows, r, q_ptr + stream * 128 * D * 2);
    else
      load_queries<D, 1, 1, 256>(p, line, sh, row - r, min(128, sh.rows - (row - r)), threadIdx.x, q_ptr);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
    const uint64_t seen = nodes_seen(p, sh.b, sh.count, live ? row_node(p, sh, row) : -1);

    float m = -INFINITY, l = 0.f;  // m: the reference, scaled by log2(e)
    for (int j = two ? 0 : stream; j < sh.n; j += two ? 1 : 2) {
      wait(&sm.s_full[stream], s_uses++);
      tc_fence_after();
      bool run_ends = false;  // before this tile
      if constexpr (RUNS) {
        const int i = two ? j : j / 2;  // the stream's tiles before this one
        run_ends = i > 0 && i % kRun == 0;
        if (run_ends && warp_live) end_run(m, i > kRun, true);
      }
      if (warp_live) {
        uint32_t x[kKeys];
        const Sight v = sight_of(sm.mask[(tile_no + j) % kMasks], sh.start - first_slot(sh) - (sh.k0 + j) * kKeys, seen);
        const float top = read_scores(t_s, v.some, v.bits, x);
        const float keep = move_reference(top * p.scale_log2, m, l);
        const int before = two ? j : j / 2;  // tiles already in O
        if (before > 0 && !run_ends && __any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_load32(t_o + c, o);
            tmem_wait_ld<32>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
            tmem_store32(t_o + c, o);
          }
        }
        const float from = m == -INFINITY ? 0.f : -m;
        const unsigned long long from2 = pack2(from, from);
        unsigned long long sums[2] = {0, 0};
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          uint32_t w[2][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 a = weights2(x[16 * h + 2 * e], x[16 * h + 2 * e + 1], scale2, from2, sums[e % 2]);
            w[0][e] = weight_part<0>(a);
            w[1][e] = weight_rest(a);
          }
          tmem_store8(t_s + 8 * h, w[0]);
          tmem_store8(t_s + 64 + 8 * h, w[1]);
          if (h == 3) {  // its products need not wait for the second half
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[stream][0]);
          }
        }
        add2(sums[0], sums[1]);
        const float2 sum = unpack2(sums[0]);
        l += sum.x + sum.y;
        tmem_wait_st();
      } else if (lane == 0) {
        mbar_arrive(&sm.p_full[stream][0]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[stream][1]);
    }
    tile_no += sh.n;

    // ---- the share's rows
    if (!two && stream == 1) {
      sm.ml[r][0] = m;
      sm.ml[r][1] = l;
    }
    wait(&sm.o_full, share);
    tc_fence_after();
    if (RUNS && (two ? sh.n : (sh.n + 1 - stream) / 2) > kRun && warp_live) {
      end_run(m, true, false);
      tc_fence_before();
    }
    if (!two) named_bar(1, 32 * kSoftWarps);
    if (RUNS && !two) tc_fence_after();
    if ((two || stream == 0) && warp_live) {
      float f0 = 1.f, f1 = 0.f;  // factors of the streams' shares (one row block)
      if (!two) {
        const float m1 = sm.ml[r][0], l1 = sm.ml[r][1];
        const float both = fmaxf(m, m1);
        f0 = l == 0.f ? 0.f : fast_exp2(m - both);
        f1 = l1 == 0.f ? 0.f : fast_exp2(m1 - both);
        l = (l == 0.f ? 0.f : l * f0) + (l1 == 0.f ? 0.f : l1 * f1);
        m = both;
      } else if (l == 0.f) {
        f0 = 0.f;
      }
      if (wait_failed(sm)) l = NAN;
      const bool second = !two && sh.n > 1;  // stream 1 had a tile
      const size_t slot = share_slot(p, group, sh, rt, local, row);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        float y[32];
        tmem_load32(t_o + c, o);
        tmem_wait_ld<32>(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = f0 != 0.f ? __uint_as_float(o[e]) * f0 : 0.f;
        if (second) {
          tmem_load32(t_o + D + c, o);
          tmem_wait_ld<32>(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] += f1 != 0.f ? __uint_as_float(o[e]) * f1 : 0.f;
        }
        put_columns<D, 1>(p, sh, sm, share, seen, row, c, live, l, slot, y);
      }
      if (live && !is_final(sh)) {
        p.part_ml[slot * 2] = m;
        p.part_ml[slot * 2 + 1] = l;
      }
    }
    end_share(sm, share);
    ++share;
  }
}

// fp32: a row has two threads, half 0 in warps 0-3 and half 1 in warps 4-7. Each
// makes the weights of half of every tile's keys (their maxima meet in shared
// memory) and keeps half of the row's output columns in registers, to which it
// adds a tile's product while the next one is made.
// kFew: the rows stand three times in the block, rows 32 i to 32 i + 31 with part i of
// the weights, so that one product takes all three parts; the three sums are
// added at the end of the share.
template <int D, int KIND, class P>
__device__ __forceinline__ void exact_role(const P& p, Shared& sm, const typename P::Line& line,
                                           uint8_t* q_ptr, uint32_t tmem, int u_begin, int u_end,
                                           int rt, int group) {
  using Lay = Layout<D, KIND>;
  constexpr bool FEW = KIND == kFew;
  const int half = threadIdx.x / 128, r = threadIdx.x % 128, lane = threadIdx.x % 32;
  const int copy = FEW ? r / 32 : 0;
  const uint32_t lanes = (uint32_t)(r / 32) * 32 << 16;
  const uint32_t t_o = tmem + lanes + Lay::kOut + half * (D / 2);
  const unsigned long long scale2 = pack2(p.scale_log2, p.scale_log2);
  Waiter wait(sm);
  uint32_t s_uses[2] = {0, 0}, t_uses[2] = {0, 0}, tile_no = 0;
  int u = u_begin;
  typename P::Share sh;
  for (uint32_t share = 0; next_share(p, line, u_begin, u_end, u, sh);) {
    if (rt * p.row_tile >= sh.rows) continue;
    const int row = first_row(sh) + rt * p.row_tile + (FEW ? lane : r);
    const bool live = copy < 3 && row_there(p, line, sh, row), warp_live = __any_sync(0xffffffffu, live);
    const int row0 = row - (FEW ? lane : r);
    load_queries<D, 3, FEW ? 3 : 1, 256>(p, line, sh, row0, min(FEW ? 32 : 128, sh.rows - row0),
                                         threadIdx.x, q_ptr);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
    const uint64_t seen = nodes_seen(p, sh.b, sh.count, live ? row_node(p, sh, row) : -1);
    float m = -INFINITY, l = 0.f, keep = 1.f, acc[D / 2];
#pragma unroll
    for (int e = 0; e < D / 2; ++e) acc[e] = 0.f;
    for (int j = 0; j <= sh.n; ++j) {
      const float last_keep = keep;  // the factor of the tile before
      if (j < sh.n) {
        const int s = j & 1;
        const uint32_t t_s = tmem + lanes + s * Lay::kScoreStep;
        wait(&sm.s_full[s], s ? s_uses[1]++ : s_uses[0]++);
        tc_fence_after();
        uint32_t x[64];
        float top = -INFINITY;
        if (warp_live) {
          const Sight v = sight_of(sm.mask[(tile_no + j) % kMasks], sh.start - first_slot(sh) - (sh.k0 + j) * kKeys, seen);
          const uint32_t bits[2] = {half ? v.bits[2] : v.bits[0], half ? v.bits[3] : v.bits[1]};
          top = read_scores(t_s + 64 * half, v.some, bits, x);
          sm.top[s][half][r] = top;
        }
        // both halves' scores have been read (the weights go over them), both
        // maxima are there
        tc_fence_before();
        named_bar(1, 32 * kSoftWarps);
        tc_fence_after();
        if (warp_live) {
          keep = move_reference(fmaxf(top, sm.top[s][half ^ 1][r]) * p.scale_log2, m, l);
          const float from = m == -INFINITY ? 0.f : -m;
          const unsigned long long from2 = pack2(from, from);
          unsigned long long sums[2] = {0, 0};
          __syncwarp();
          // the weights, and their parts FIRST to LAST put down
          auto put_weights = [&](auto first_part, auto last_part) {
            constexpr int FIRST = decltype(first_part)::value, LAST = decltype(last_part)::value;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t w[3][8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 a = weights2(x[16 * h + 2 * e], x[16 * h + 2 * e + 1], scale2, from2, sums[e % 2]);
                w[0][e] = weight_part<0>(a);
                w[1][e] = weight_part<1>(a);
                w[2][e] = weight_part<2>(a);
              }
#pragma unroll
              for (int q = FIRST; q <= LAST; ++q)
                tmem_store8(t_s + (q - FIRST) * 64 + 32 * half + 8 * h, w[q]);
            }
          };
          using Part0 = std::integral_constant<int, 0>;
          using Part1 = std::integral_constant<int, 1>;
          using Part2 = std::integral_constant<int, 2>;
          if (!FEW) put_weights(Part0{}, Part2{});
          else if (copy == 0) put_weights(Part0{}, Part0{});
          else if (copy == 1) put_weights(Part1{}, Part1{});
          else put_weights(Part2{}, Part2{});
          add2(sums[0], sums[1]);
          const float2 sum = unpack2(sums[0]);
          l += sum.x + sum.y;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[s][half]);
      }
      if (j > 0) {
        const int t = FEW ? (j - 1) & 1 : 0;
        wait(&sm.t_full[t], t ? t_uses[1]++ : t_uses[0]++);
        tc_fence_after();
        if (warp_live) {
#pragma unroll
          for (int c = 0; c < D / 2; c += 32) {
            uint32_t y[32];
            tmem_load32(t_o + t * D + c, y);
            tmem_wait_ld<32>(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[c + e] = fmaf(acc[c + e], last_keep, __uint_as_float(y[e]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.t_free[t]);
      }
    }
    tile_no += sh.n;
    sm.sum[half][r] = l;
    // The share's products are done, so the queries' place is free for the sums
    // of the second and third parts.
    float* other = reinterpret_cast<float*>(q_ptr) + half * (D / 2) * 32 + lane;
    if (FEW && warp_live && copy > 0) {
#pragma unroll
      for (int e = 0; e < D / 2; ++e) other[((copy - 1) * D + e) * 32] = acc[e];
    }
    named_bar(1, 32 * kSoftWarps);
    if (warp_live && copy == 0) {
      if (FEW) {
#pragma unroll
        for (int e = 0; e < D / 2; ++e) acc[e] += other[(D + e) * 32] + other[e * 32];
      }
      l = sm.sum[0][r] + sm.sum[1][r];
      if (wait_failed(sm)) l = NAN;
      const size_t slot = share_slot(p, group, sh, rt, FEW ? lane : r, row);
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = l == 0.f ? 0.f : acc[c + e];
        put_columns<D, 3>(p, sh, sm, share, seen, row, half * (D / 2) + c, live, l, slot, y);
      }
      if (live && !is_final(sh) && half == 0) {
        p.part_ml[slot * 2] = m;
        p.part_ml[slot * 2 + 1] = l;
      }
    }
    end_share(sm, share);
    ++share;
  }
}

template <int D, int KIND, bool RUNS, class P>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_tc_kernel(const __grid_constant__ P p) {
  using Lay = Layout<D, KIND>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sm;
  __shared__ typename P::Line line;
  const int warp = threadIdx.x / 32;
  const int rt = blockIdx.x % p.row_tiles, group = blockIdx.x / p.row_tiles;
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* ring_ptr = base + Lay::kQ;

  griddep_launch();
  if (warp == 0) work_line(p, line);
  if (warp == 1 && threadIdx.x % 32 == 0) {
    for (int i = 0; i < Lay::kBufs; ++i) {
      mbar_init(&sm.full[i], 32 * kLoadWarps + kLoadWarps);
      mbar_init(&sm.empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 2);
      mbar_init(&sm.p_full[s][0], 4);
      mbar_init(&sm.p_full[s][1], 4);
      mbar_init(&sm.t_full[s], 2);
      mbar_init(&sm.t_free[s], kSoftWarps);
      mbar_init(&sm.done[s], kSoftWarps);
      sm.odd[s] = 0;
    }
    mbar_init(&sm.q_full, kSoftWarps);
    mbar_init(&sm.o_full, 2);
    mbar_init(&sm.drained, 1);
    sm.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&sm.tmem), 512);
  for (int i = threadIdx.x; i < 2 * MK_MAX_TREE * 8; i += kThreads) (&sm.odd_at[0][0][0][0])[i] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const Cut cut(all_places(p, line), p);
  const int u_begin = cut.begin(group), u_end = cut.begin(group + 1);

  // Registers: 16 warps launched with 128 each, 8 x 184 + 8 x 72 is the
  // same sum. A row's thread holds a tile's 128 scores; the loading warps need
  // room for the addresses of the copies in flight (56 registers: 105 cycles a
  // copy, because each waited for the last one's operands to be read).
  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    if constexpr (Lay::EXACT) {
      exact_role<D, KIND, P>(p, sm, line, base, tmem, u_begin, u_end, rt, group);
    } else {
      softmax_role<D, KIND, RUNS, P>(p, sm, line, base, tmem, u_begin, u_end, rt, group);
    }
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    load_role<D, KIND, P>(p, sm, line, smem_u32(ring_ptr), ring_ptr, u_begin, u_end, rt);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kMmaWarp + 1) put_plans(p, line);
    if (warp == kMmaWarp)
      mma_role<D, KIND, RUNS, P>(p, sm, line, smem_u32(base), smem_u32(ring_ptr), tmem, u_begin, u_end, rt);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

template <int D, int KIND, bool RUNS, class P>
int launch_kernel(const P& p, int blocks, const char* name, cudaStream_t st) {
  using Lay = Layout<D, KIND>;
  auto* fn = tree_attention_tc_kernel<D, KIND, RUNS, P>;
  static std::atomic<uint64_t> ready{0};
  if (int rc = allow_shared(ready, (const void*)fn, Lay::kBytes, name)) return rc;
  fn<<<blocks, kThreads, Lay::kBytes, st>>>(p);
  return op_cuda(cudaGetLastError(), name);
}

template <int D, int KIND, class P>
int launch_kind(const P& p, int blocks, const char* name, cudaStream_t st) {
  if constexpr (!Layout<D, KIND>::EXACT)
    if (p.runs) return launch_kernel<D, KIND, true>(p, blocks, name, st);
  return launch_kernel<D, KIND, false>(p, blocks, name, st);
}

// The kind by the row tile: fp32 32 or 128 rows, bf16 up to 128 or 256.
template <class P>
int launch_tc(const P& p, int blocks, int head_dim, int type, const char* name, cudaStream_t st) {
  const bool two = p.row_tile > 128, few = p.row_tile == 32;
  if (head_dim == 64)
    return type == MK_TYPE_FP32 ? (few ? launch_kind<64, kFew>(p, blocks, name, st)
                                       : launch_kind<64, kExact>(p, blocks, name, st))
           : two                ? launch_kind<64, kTwo>(p, blocks, name, st)
                                : launch_kind<64, kOne>(p, blocks, name, st);
  return type == MK_TYPE_FP32 ? (few ? launch_kind<128, kFew>(p, blocks, name, st)
                                     : launch_kind<128, kExact>(p, blocks, name, st))
         : two                ? launch_kind<128, kTwo>(p, blocks, name, st)
                              : launch_kind<128, kOne>(p, blocks, name, st);
}

}  // namespace
}  // namespace mk
