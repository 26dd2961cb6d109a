// What the dense kernels over the paged cache share: bounded waits that sleep,
// the elected lane, paired fp32 arithmetic, and the TMA gather of 128-token
// tiles of one KV head from the pages.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "tc_util.cuh"

namespace qsa {

constexpr int PT_ROWS = 128;                   // tokens (MMA rows) of a tile
constexpr int PT_MAX_LEN = 1 << 30;            // tokens of a sequence (token arithmetic is 32-bit)
constexpr uint32_t PT_HALF = PT_ROWS * 128;    // bytes of its 64-value half (128-byte swizzle)
constexpr uint32_t PT_TILE = 2 * PT_HALF;      // a tile: 128 rows of 128 bf16 values

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two fp32 values in one register pair, and their paired operations.
__device__ __forceinline__ unsigned long long f2_pack(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(unsigned long long x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ unsigned long long f2_fma(unsigned long long a, unsigned long long b,
                                                      unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long f2_add(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                          int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Bounded wait, as mbar_wait, but a round may sleep up to PT_WAIT_NS until the
// phase completes, and rounds are 20 ns apart: the other warps' polling takes
// issue slots from the softmax (ragged chunks 248 us without the pause, 228 with
// it and no less with a longer one).
// A round that nothing ends takes 4 us: PT_WAIT_ROUNDS are 0.27 s. A wait for a
// whole item of the attention weights (KV heads x up to 4,096 query blocks, 1.4 us
// each) takes PT_LONG_ROUNDS, 34 s; when another role gives up, it ends within a
// round.
constexpr uint32_t PT_WAIT_NS = 20000, PT_WAIT_ROUNDS = 1u << 16, PT_LONG_ROUNDS = 1u << 23;
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                         unsigned *err, uint32_t rounds = PT_WAIT_ROUNDS) {
  for (uint32_t i = 0; i < rounds; ++i) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.b32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(PT_WAIT_NS)
        : "memory");
    if (done) return true;
    __nanosleep(20);
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  raise_err(err, ERR_TIMEOUT);
  return false;
}

// The same by every lane of a warp.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                            unsigned *err) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, err));
}

// Both of two barriers, whose checks overlap.
__device__ __forceinline__ bool wait_all2(uint32_t bar, uint32_t parity, uint32_t bar2,
                                             uint32_t parity2, volatile int *abort_flag,
                                             unsigned *err) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p, q;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n and.pred p, p, q;\n"
      " selp.b32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(bar2), "r"(parity2)
      : "memory");
  if (__all_sync(0xffffffffu, done)) return true;
  return wait_all(bar, parity, abort_flag, err) && wait_all(bar2, parity2, abort_flag, err);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Whole-warp bounded wait: lane 0 polls. What it has seen complete is ordered
// before the other lanes' accesses by __syncwarp; a shuffle alone orders none.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                             unsigned *err) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, abort_flag, err);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok;
}

// Where the pages are, and how a tile's 128 tokens fall on them.
struct PagedTiles {
  const int32_t *table;  // block table
  int max_pages, num_pages, P;
  int box;               // tokens of a piece: the largest power of two in P, at most 128
  int pages, slots;      // 128 tokens in whole pages and slots
  unsigned *err;
};

// The pieces of the steps' 128 tokens, one lane each, in step order: where
// they lie in their pages, and the page ids, read two steps ahead. (A piece of
// `box` tokens never crosses a page. No division per step: the loaders' few
// instructions are on the path from a free stage to its next tile.)
struct PagePieces {
  static constexpr int NONE = -0x7fffffff - 1;
  const int32_t *row;  // the sequence's block-table row, at the page read next
  int tok, rslot, L;   // the piece read next: its first token, its slot
  int slot;            // the slot of the step being issued
  int id[2];
  __device__ __forceinline__ void start(const PagedTiles &p, int seq, int seq_len, int first, int lane) {
    const bool has = lane * p.box < PT_ROWS;
    tok = first * PT_ROWS + (has ? lane * p.box : 0);
    L = has ? seq_len : 0;
    const int col = tok / p.P;
    slot = rslot = tok - col * p.P;
    row = p.table + (size_t)seq * p.max_pages + col;
    id[0] = read(p);
    id[1] = read(p);
  }
  __device__ __forceinline__ int read(const PagedTiles &p) {
    if (tok >= L) return NONE;
    const int v = __ldg(row);
    tok += PT_ROWS;
    rslot += p.slots;
    row += p.pages;
    if (rslot >= p.P) {
      rslot -= p.P;
      ++row;
    }
    return v;
  }
  // The page of this step's piece (-1: past L, or a bad page).
  __device__ __forceinline__ int take(const PagedTiles &p) {
    int v = id[0];
    id[0] = id[1];
    id[1] = read(p);
    if (v < 0 || v >= p.num_pages) {
      if (v != NONE) raise_err(p.err, ERR_PAGE);
      v = -1;
    }
    return v;
  }
  __device__ __forceinline__ void step(const PagedTiles &p) {
    slot += p.slots;
    if (slot >= p.P) slot -= p.P;
  }
};

// Copies a tile: every piece's two halves of 64 values, by the elected lane.
// `page` and `slot` are this lane's piece's; `bar` expects the bytes already.
__device__ __forceinline__ void issue_tile(const PagedTiles &p, const CUtensorMap *map, uint32_t dst,
                                           uint32_t bar, int page, int slot, int h, bool lead) {
  for (int i = 0, off = 0; off < PT_ROWS; ++i, off += p.box) {
    const int pg = __shfl_sync(0xffffffffu, page, i), sl = __shfl_sync(0xffffffffu, slot, i);
    if (pg >= 0 && lead) {
      tma_load_4d(dst + off * 128, map, bar, 0, h, sl, pg);
      tma_load_4d(dst + PT_HALF + off * 128, map, bar, 64, h, sl, pg);
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void load_tile(const PagedTiles &p, const CUtensorMap *map, uint32_t dst,
                                          uint32_t bar, int page, int slot, int h, bool lead) {
  const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
  if (lead) mbar_arrive_expect(bar, (uint32_t)(__popc(live) * p.box * 256));
  __syncwarp();
  issue_tile(p, map, dst, bar, page, slot, h, lead);
}

// Failure injection for the two kernels that stream the cache through these tiles,
// read at each launch from the environment variable QSA_DEBUG_STALL_DENSE: a CTA
// issues that many K tiles (pairs of them, for the attention weights) and then no
// more, as if a copy had been lost, and every role's waits run out (after 0.27 s).
// -1 where it is unset: no limit.
int debug_stall_dense();

inline PagedTiles paged_tiles(const qsa_dims &d, const qsa_cache &c, unsigned *err) {
  PagedTiles t;
  t.table = c.block_table;
  t.max_pages = c.max_pages_per_seq;
  t.num_pages = c.num_pages;
  t.P = d.P;
  t.box = (d.P & -d.P) < PT_ROWS ? (d.P & -d.P) : PT_ROWS;
  t.pages = PT_ROWS / d.P;
  t.slots = PT_ROWS % d.P;
  t.err = err;
  return t;
}

// Tensor map of a K or V pool [num_pages, P, Hkv, 128] for the gather above.
inline bool pool_map(EncodeTiledFn enc, CUtensorMap *map, void *pool, const qsa_dims &d,
                     const qsa_cache &c, int box) {
  const cuuint64_t row = (cuuint64_t)d.Hkv * 256;
  const cuuint64_t dims[4] = {128, (cuuint64_t)d.Hkv, (cuuint64_t)d.P, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {256, row, row * d.P};
  const cuuint32_t boxes[4] = {64u, 1u, (cuuint32_t)box, 1u}, ones[4] = {1u, 1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of query rows [Nq, Hq, 128]: boxes of `tokens` tokens x G heads, one
// 64-value half each. Rows past Nq read as zeros.
inline bool query_map(EncodeTiledFn enc, CUtensorMap *map, const void *q, const qsa_dims &d, int Nq,
                      int tokens) {
  const cuuint64_t dims[3] = {128, (cuuint64_t)d.Hq, (cuuint64_t)Nq};
  const cuuint64_t strides[2] = {256, (cuuint64_t)d.Hq * 256};
  const cuuint32_t boxes[3] = {64u, (cuuint32_t)(d.Hq / d.Hkv), (cuuint32_t)tokens};
  const cuuint32_t ones[3] = {1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, boxes,
             ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qsa
