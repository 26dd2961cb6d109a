// qsa_evict: the micro-blocks of each sequence that received least attention
// leave the cache; the others are copied, in order, to the pages of a
// destination table.
//
// Two kernels. select: one CTA per sequence finds the kept blocks (exactly,
// ties by the lowest index): a radix select over the weights' ordered bits,
// 11 + 11 + 10 bits, then one ordered emission. copy: one warp per kept block
// moves its 4 tokens' K, V and indexer keys (contiguous in a page, since
// pages hold whole blocks) and its side-cache key. The copy is memory: every
// kept byte is read and written once. 24 ragged sequences of up to 65,536 tokens
// down to 8,192 (4 KV heads): select 22 us, copy 124 us (6.2 TB/s).
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace qsa {
namespace {

constexpr int EV_THREADS = 1024;
constexpr int EV_WARPS = EV_THREADS / 32;
constexpr int EV_BINS = 2048;
constexpr int EV_CACHED = 50 * 1024;  // weights: 200 KB, 204,800 tokens

struct EvictArgs {
  const int32_t *seq_lens, *table, *dst;
  const float *mass;
  float *mass_out;
  int32_t *kept, *new_lens;
  uint4 *k_pool, *v_pool, *x_pool, *side_pool;
  int ld, keep, sink, recent;
  int cached;  // weights that fit the select kernel's shared memory
  int P, max_pages, num_pages;
  int kv_vec, x_vec;  // 16-byte vectors per token row of K (= of V), per indexer key
  unsigned *err;
};

// Ordered bits of a weight: a larger weight has the larger key, -0 equals +0,
// NaN is the smallest.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (!(m == m)) return 0u;
  const uint32_t b = __float_as_uint(m + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

constexpr int EV_BATCH = 8;  // weights that a thread requests together

// Sum of the values of the warps before this one (v: this warp's, the same in
// every lane). wsum: one value per warp; barriers included.
__device__ __forceinline__ int before_warp(int v, int *wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) wsum[warp] = v;
  __syncthreads();
  int x = lane < warp ? wsum[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  return x;
}

__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(EvictArgs a) {
  extern __shared__ float cache[];
  __shared__ int hist[EV_BINS];
  __shared__ int wsum[EV_WARPS];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  const int L = a.seq_lens[b];
  const float *row = a.mass + (size_t)b * a.ld;
  float *mass_out = a.mass_out + (size_t)b * a.ld;
  int32_t *kept = a.kept + (size_t)b * a.keep;
  const bool bad = L < 0 || (long long)L > 4LL * a.ld;
  if (bad && tid == 0) raise_err(a.err, ERR_LEN);
  const int nb = bad ? 0 : (L + 3) >> 2;
  const int n = min(a.keep, nb);
  if (tid == 0) a.new_lens[b] = n == 0 ? 0 : 4 * (n - 1) + (L - 4 * (nb - 1));
  for (int i = n + tid; i < a.keep; i += EV_THREADS) kept[i] = -1;
  for (int i = n + tid; i < a.ld; i += EV_THREADS) mass_out[i] = 0.f;
  if (n == nb) {
    for (int i = tid; i < n; i += EV_THREADS) {
      kept[i] = i;
      mass_out[i] = row[i];
    }
    return;
  }
  // the weights are read five times: from shared memory where they fit
  const float *mass = row;
  if (nb <= a.cached) {
    for (int j0 = tid; j0 < nb; j0 += EV_THREADS * EV_BATCH) {
      float m[EV_BATCH];
#pragma unroll
      for (int u = 0; u < EV_BATCH; ++u)
        if (j0 + u * EV_THREADS < nb) m[u] = row[j0 + u * EV_THREADS];
#pragma unroll
      for (int u = 0; u < EV_BATCH; ++u)
        if (j0 + u * EV_THREADS < nb) cache[j0 + u * EV_THREADS] = m[u];
    }
    __syncthreads();
    mass = cache;
  }
  // candidates: [sink, nb - recent); `need` of them stay
  const int c0 = a.sink, c1 = nb - a.recent;
  int need = a.keep - a.sink - a.recent;
  uint32_t prefix = 0, mask = 0;
  const int shifts[3] = {21, 10, 0};
  const int widths[3] = {11, 11, 10};
  for (int r = 0; r < 3 && need > 0; ++r) {
    const int sh = shifts[r], bins = 1 << widths[r];
    for (int i = tid; i < bins; i += EV_THREADS) hist[i] = 0;
    __syncthreads();
    for (int j0 = c0; j0 < c1; j0 += EV_THREADS * EV_BATCH) {
      float m[EV_BATCH];
#pragma unroll
      for (int u = 0; u < EV_BATCH; ++u) {
        const int j = j0 + u * EV_THREADS + tid;
        m[u] = j < c1 ? mass[j] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < EV_BATCH; ++u) {
        if (j0 + u * EV_THREADS >= c1) break;
        int bin = -1;
        const uint32_t key = mass_key(m[u]);
        if (j0 + u * EV_THREADS + tid < c1 && (key & mask) == prefix)
          bin = (int)((key >> sh) & (uint32_t)(bins - 1));
        // (32 equal weights are one add; otherwise few lanes meet in a bin)
        if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
          if (bin >= 0 && lane == 0) atomicAdd(&hist[bin], 32);
        } else if (bin >= 0) {
          atomicAdd(&hist[bin], 1);
        }
      }
    }
    __syncthreads();
    // from the top bin down: the bin in which the need-th largest lies
    constexpr int PER = EV_BINS / EV_THREADS;
    int mine[PER], tot = 0;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int bin = bins - 1 - (tid * PER + u);
      mine[u] = bin >= 0 ? hist[bin] : 0;
      tot += mine[u];
    }
    int x = tot;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    int before = x - tot + before_warp(__shfl_sync(0xffffffffu, x, 31), wsum);
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      if (before < need && before + mine[u] >= need) {
        s_prefix = prefix | ((uint32_t)(bins - 1 - (tid * PER + u)) << sh);
        s_need = need - before;
      }
      before += mine[u];
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    mask |= (uint32_t)(bins - 1) << sh;
    __syncthreads();
  }
  // prefix is now the weight of the last kept candidate; of the blocks that
  // equal it, the first `need` stay (none where need is 0)
  const uint32_t cut = need > 0 ? prefix : 0xffffffffu;
  const int per = ((nb + EV_WARPS - 1) / EV_WARPS + 31) / 32 * 32;
  const int j0 = warp * per, j1 = min(nb, j0 + per);
  int gt = 0, eq = 0;
  for (int jb = j0; jb < j1; jb += 32 * EV_BATCH) {
    float m[EV_BATCH];
#pragma unroll
    for (int u = 0; u < EV_BATCH; ++u) {
      const int j = jb + 32 * u + lane;
      m[u] = j < j1 ? mass[j] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < EV_BATCH; ++u) {
      const int j = jb + 32 * u + lane;
      const bool in = j < j1, always = in && (j < c0 || j >= c1);
      const uint32_t key = mass_key(m[u]);
      gt += always || (in && key > cut);
      eq += in && !always && key == cut;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  int gb = before_warp(gt, wsum), eb = before_warp(eq, wsum);
  const unsigned below = (1u << lane) - 1u;
  for (int jb = j0; jb < j1; jb += 32 * EV_BATCH) {
    float m[EV_BATCH];
#pragma unroll
    for (int u = 0; u < EV_BATCH; ++u) {
      const int j = jb + 32 * u + lane;
      m[u] = j < j1 ? mass[j] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < EV_BATCH; ++u) {
      const int j = jb + 32 * u + lane;
      if (jb + 32 * u >= j1) break;
      const bool in = j < j1, always = in && (j < c0 || j >= c1);
      const uint32_t key = mass_key(m[u]);
      const bool g = always || (in && key > cut), e = in && !always && key == cut;
      const unsigned bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
      const int er = eb + __popc(be & below);  // equal ones before this block
      if (g || (e && er < need)) {
        const int at = gb + __popc(bg & below) + min(er, need);
        kept[at] = j;
        mass_out[at] = m[u];
      }
      gb += __popc(bg);
      eb += __popc(be);
    }
  }
}

// Physical page of block `blk` of a table row, or -1 after flagging an error.
__device__ __forceinline__ int block_page(const EvictArgs &a, const int32_t *row, int blk,
                                          int lane) {
  const int col = (int)((4LL * blk) / a.P);
  if (col >= a.max_pages) {
    if (lane == 0) raise_err(a.err, ERR_BT);
    return -1;
  }
  const int page = row[col];
  if (page < 0 || page >= a.num_pages) {
    if (lane == 0) raise_err(a.err, ERR_PAGE);
    return -1;
  }
  return page;
}

// n vectors from each of two rows of sources, all of a round requested before
// the first is written.
__device__ __forceinline__ void copy_vecs(uint4 *d0, const uint4 *s0, uint4 *d1, const uint4 *s1,
                                          int n, int lane) {
  constexpr int U = 8;
  for (int i0 = lane; i0 < n; i0 += 32 * U) {
    uint4 v[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 32 * u < n) {
        v[u] = s0[i0 + 32 * u];
        w[u] = s1[i0 + 32 * u];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 32 * u < n) {
        d0[i0 + 32 * u] = v[u];
        d1[i0 + 32 * u] = w[u];
      }
  }
}

__global__ void __launch_bounds__(256) evict_copy_kernel(EvictArgs a) {
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  const int nl = a.new_lens[b];
  if (4LL * i >= nl) return;
  const int blk = a.kept[(size_t)b * a.keep + i];
  const int toks = min(4, nl - 4 * i);
  const int sp = block_page(a, a.table + (size_t)b * a.max_pages, blk, lane);
  const int dp = block_page(a, a.dst + (size_t)b * a.max_pages, i, lane);
  if (sp < 0 || dp < 0) return;
  const int rpp = a.P / 4;
  const size_t s = (size_t)sp * rpp + blk % rpp, d = (size_t)dp * rpp + i % rpp;
  // (the small rows first: their loads overlap with the large ones')
  uint4 x[2], y;
  const int xn = toks * a.x_vec;  // at most 64
  const uint4 *xs = a.x_pool + s * 4 * a.x_vec;
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (lane + 32 * u < xn) x[u] = xs[lane + 32 * u];
  if (toks == 4 && lane < a.x_vec) y = a.side_pool[s * a.x_vec + lane];
  copy_vecs(a.k_pool + d * 4 * a.kv_vec, a.k_pool + s * 4 * a.kv_vec,
            a.v_pool + d * 4 * a.kv_vec, a.v_pool + s * 4 * a.kv_vec, toks * a.kv_vec, lane);
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (lane + 32 * u < xn) a.x_pool[d * 4 * a.x_vec + lane + 32 * u] = x[u];
  if (toks == 4 && lane < a.x_vec) a.side_pool[d * a.x_vec + lane] = y;
}

}  // namespace

cudaError_t launch_evict(const qsa_dims &d, const qsa_cache &c, int B, const int32_t *seq_lens,
                         const float *mass, int ld, int keep, int sink, int recent,
                         const int32_t *dst_table, int32_t *kept, int32_t *new_lens,
                         float *mass_out, unsigned *err, cudaStream_t st) {
  EvictArgs a;
  a.seq_lens = seq_lens;
  a.table = c.block_table;
  a.dst = dst_table;
  a.mass = mass;
  a.mass_out = mass_out;
  a.kept = kept;
  a.new_lens = new_lens;
  a.k_pool = static_cast<uint4 *>(c.k_pool);
  a.v_pool = static_cast<uint4 *>(c.v_pool);
  a.x_pool = static_cast<uint4 *>(c.kidx_pool);
  a.side_pool = static_cast<uint4 *>(c.side_pool);
  a.ld = ld;
  a.keep = keep;
  a.sink = sink;
  a.recent = recent;
  a.P = d.P;
  a.max_pages = c.max_pages_per_seq;
  a.num_pages = c.num_pages;
  a.kv_vec = d.Hkv * d.D / 8;
  a.x_vec = d.di / 8;
  a.err = err;
  a.cached = std::min(ld, EV_CACHED);
  const size_t smem = (size_t)a.cached * sizeof(float);
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(evict_select_kernel), smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(evict_select_kernel, B, EV_THREADS, smem, st, a);
  if (e != cudaSuccess) return e;
  const int most = std::min(keep, ld);
  return launch_pdl(evict_copy_kernel, dim3((most + 7) / 8, B), 256, 0, st, a);
}

}  // namespace qsa
