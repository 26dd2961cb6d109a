// qsa_attention_mass: the attention weight that the rows of appended chunks
// gave to each micro-block, summed over rows and heads.
//
//   mass[s, j] = mass_in[s, j] + sum_{t in block j} sum_{rows i of s that see t}
//                sum_h e^(scale q_ih.K_t - LSE_ih)
//
// The rows' LSEs are known, so a weight needs no running maximum, and the sum
// runs over rows and heads for a fixed token. So the scores are computed
// transposed, S^T = K Q^T (tcgen05, M = 128 tokens, N = up to 128 rows x
// heads of one KV head): a thread holds one token and adds its weights up in
// registers, without any exchange.
//
// Three kernels, chained by programmatic dependent launch:
//   plan    one CTA: the prefix of the sequences' work; the others copy
//           mass_in to mass. An item is 256 tokens of a sequence, its steps
//           the KV heads x the blocks of TT = 128 / G chunk tokens that see
//           any of them;
//   weigh   one CTA per SM over an equal range of the flattened steps. An item
//           that several CTAs share leaves its partial sums in the workspace;
//   join    adds those in CTA order.
// Every block's sum is formed in a fixed order: the same call, the same bits.
//
// weigh: two K tiles of 128 tokens stay in shared memory for a head while the
// query blocks stream past them (each query block from L2 serves 256 tokens,
// 16 bytes a clock per SM), so prompts are bound by the exponentials: 16 a
// clock per SM, 2,048 clocks a step of 256 x 128. A quarter of them goes to the
// fp32 units instead: 8,192 rows of a prompt (32 query heads) 403 us without,
// 389 with an eighth, 378 with a quarter, 387 with three eighths. One decode token
// per sequence is bound by reading K once: 182 us for 32 x 32,768 tokens, 5.9 TB/s.
//   warps 0-7, 8-15 the weights of the even and the odd steps (S^T is double
//                   buffered), 4 warps for each of the two K tiles
//   warp 16         issues the MMAs
//   warp 17, 18     TMA of K tiles; of query blocks, and their LSEs
//   warp 19         announces the items to the other warps, a few ahead
// A step's sum is added to the token's sum with its rounding error carried
// along (a token of a long prompt receives up to a million weights).
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "paged_tiles.cuh"
#include "tc_util.cuh"
#include "umma_desc.h"

namespace qsa {
namespace {

constexpr int AM_THREADS = 640;
constexpr int AM_KBUF = 2;     // pairs of K tiles
constexpr int AM_QST = 3;      // query blocks
constexpr int AM_ITEMS = 3;    // items announced ahead
constexpr int AM_READERS = 19;
constexpr int AM_TOK = 2 * PT_ROWS;  // tokens of an item
constexpr uint32_t AM_CTL = 3 * 1024;
constexpr size_t AM_SMEM = AM_CTL + (size_t)(2 * AM_KBUF + AM_QST) * PT_TILE;
constexpr int AM_PLAN_THREADS = 1024;
constexpr int AM_POLY = 2;  // of 8 pairs of exponentials, those on the fp32 units
constexpr int AM_FEW = 4;  // chunk tokens that are loaded one by one

struct AmArgs {
  PagedTiles pages;
  const int32_t *seq_lens, *row_start;
  const float *lse, *mass_in;
  float *mass;
  int *hdr;         // [0] CTAs with work
  long long *base;  // [S + 1] prefix of the sequences' steps
  float *rec;       // [CTAs][2][64] partial sums of shared items
  int S, Nq, Hq, Hkv, G, TT, ld;
  int k_tiles;      // failure injection: pairs of K tiles that a CTA issues
  float c2;         // scale * log2(e)
  unsigned *err;
};

// Chunk of sequence s (T rows from r0, length L), or false if it is skipped.
__device__ __forceinline__ bool am_chunk(const AmArgs &a, int s, int &r0, int &T, int &L) {
  r0 = a.row_start[s];
  const int r1 = a.row_start[s + 1];
  L = a.seq_lens[s];
  T = r1 - r0;
  return !(r0 < 0 || r1 < r0 || r1 > a.Nq || T > L || L > PT_MAX_LEN ||
           (long long)L > (long long)a.pages.max_pages * a.pages.P || (long long)L > 4LL * a.ld);
}
// First query block of a chunk that sees any token of item u.
__device__ __forceinline__ int am_first(const AmArgs &a, int u, int T, int L) {
  const int x = u * AM_TOK - (L - T);
  return x < 0 ? 0 : x / a.TT;
}
// Items whose every query block counts.
__device__ __forceinline__ int am_full_items(const AmArgs &a, int T, int L) {
  return min((L + AM_TOK - 1) / AM_TOK, (L - T + a.TT + AM_TOK - 1) / AM_TOK);
}

__global__ void __launch_bounds__(AM_PLAN_THREADS) am_plan_kernel(AmArgs a, int ctas) {
  __shared__ long long wsum[AM_PLAN_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  if (blockIdx.x > 0) {
    const long long n = (long long)a.S * a.ld, step = (long long)(gridDim.x - 1) * blockDim.x;
    for (long long i = (long long)(blockIdx.x - 1) * blockDim.x + tid; i < n; i += step)
      a.mass[i] = a.mass_in != nullptr ? a.mass_in[i] : 0.f;
    return;
  }
  long long tbase = 0;
  for (int b0 = 0; b0 < a.S; b0 += AM_PLAN_THREADS) {
    const int s = b0 + tid;
    long long n = 0;
    if (s < a.S) {
      int r0, T, L;
      if (!am_chunk(a, s, r0, T, L)) {
        raise_err(a.err, ERR_LEN);
      } else if (T > 0) {
        const int nq = (T + a.TT - 1) / a.TT, U = (L + AM_TOK - 1) / AM_TOK;
        const int full = am_full_items(a, T, L);
        n = (long long)full * nq;
        for (int u = full; u < U; ++u) n += nq - am_first(a, u, T, L);
        n *= a.Hkv;
      }
    }
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    long long off = tbase, tot = 0;
    for (int i = 0; i < AM_PLAN_THREADS / 32; ++i) {
      if (i < warp) off += wsum[i];
      tot += wsum[i];
    }
    __syncthreads();
    if (s < a.S) a.base[s] = off + x - n;
    tbase += tot;
  }
  if (tid == 0) {
    a.base[a.S] = tbase;
    a.hdr[0] = (int)min((long long)ctas, max(1LL, tbase));
  }
}

__device__ __forceinline__ long long am_bound(long long total, int c, int n) { return total * c / n; }
// The CTA whose range holds a step.
__device__ __forceinline__ int am_owner(long long total, long long step, int n) {
  int c = (int)(step * n / total);
  while (c + 1 < n && am_bound(total, c + 1, n) <= step) ++c;
  while (c > 0 && am_bound(total, c, n) > step) --c;
  return c;
}

// An item and this CTA's steps [a, b) of it, none at the end of the range.
// Step k is KV head k / nq and query block q0 + k % nq.
struct __align__(16) AmItem {
  int a, b, nq, q0;
  int seq, u, whole, steps;
  int r0, T, L, pad;
};

// The item that holds step `at` of all; fills everything but [a, b). Returns
// the item's first step.
__device__ long long am_find(const AmArgs &p, long long at, AmItem &it) {
  int x = 0, y = p.S - 1;  // last sequence that starts at or before it (with steps)
  while (x < y) {
    const int m = (x + y + 1) >> 1;
    if (p.base[m] <= at) x = m; else y = m - 1;
  }
  it.seq = x;
  am_chunk(p, x, it.r0, it.T, it.L);
  const int nq = (it.T + p.TT - 1) / p.TT, full = am_full_items(p, it.T, it.L);
  const long long rel = at - p.base[x], per = (long long)p.Hkv * nq;
  long long first;
  if (rel < full * per) {
    it.u = (int)(rel / per);
    first = it.u * per;
  } else {
    it.u = full;
    first = full * per;
    for (;;) {
      const long long n = (long long)p.Hkv * (nq - am_first(p, it.u, it.T, it.L));
      if (rel < first + n) break;
      first += n;
      ++it.u;
    }
  }
  it.q0 = am_first(p, it.u, it.T, it.L);
  it.nq = nq - it.q0;
  it.steps = p.Hkv * it.nq;
  return p.base[x] + first;
}

// ------------------------------------------------------------------ weigh

// sum + 2^x of a pair on the fp32 units: x = n + f with n the nearest whole
// number (left in the low bits of x + 1.5 * 2^23) and |f| <= 1/2, 2^f by the
// polynomial 1 + f (c1 + ... c5 f^4) of least relative error there (a linear
// program on a grid; 1.7e-7 with its fp32 roundings), and 2^n, whose bits are n
// in the exponent's place, in the multiplication that adds to the sum. x is held
// in [-127, 128], where 2^n is exactly 0 and infinity; a NaN stays one.
__device__ __forceinline__ float nan_clamp(float x) {
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;\n min.NaN.f32 %0, %0, 0f43000000;" : "+f"(x));
  return x;
}
__device__ __forceinline__ unsigned long long add_exp2_poly(unsigned long long sum, float x0,
                                                            float x1) {
  const unsigned long long m = f2_pack(nan_clamp(x0), nan_clamp(x1));
  const unsigned long long r = f2_add(m, f2_pack(12582912.f, 12582912.f));
  const unsigned long long f =
      f2_fma(f2_add(r, f2_pack(-12582912.f, -12582912.f)), f2_pack(-1.f, -1.f), m);
  unsigned long long y = f2_fma(f, f2_pack(0x1.5bba0cp-10f, 0x1.5bba0cp-10f),
                                f2_pack(0x1.3cea88p-7f, 0x1.3cea88p-7f));
  y = f2_fma(f, y, f2_pack(0x1.c6b754p-5f, 0x1.c6b754p-5f));
  y = f2_fma(f, y, f2_pack(0x1.ebf9bcp-3f, 0x1.ebf9bcp-3f));
  y = f2_fma(f, y, f2_pack(0x1.62e42ap-1f, 0x1.62e42ap-1f));
  y = f2_fma(f, y, f2_pack(1.f, 1.f));
  float r0, r1;
  f2_unpack(r, r0, r1);
  return f2_fma(y, f2_pack(__uint_as_float((__float_as_uint(r0) << 23) + 0x3f800000u),
                           __uint_as_float((__float_as_uint(r1) << 23) + 0x3f800000u)),
                sum);
}

struct AmCtrl {
  uint64_t kfull[AM_KBUF], kempty[AM_KBUF];
  uint64_t qfull[AM_QST], qempty[AM_QST], nfull[AM_QST], nempty[AM_QST];
  uint64_t sfull[2], sempty[2], ffull, fempty, drain;
  uint64_t ifull[AM_ITEMS], iempty[AM_ITEMS];
  AmItem item[AM_ITEMS];
  uint32_t tmem;
  int abort_flag, kissued, qissued;
  float nl[AM_QST][PT_ROWS];  // -LSE log2(e) of a query block's rows
  float fin[AM_TOK];          // an item's sums over its odd steps
};

struct AmItems {
  int slot = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ bool next(AmCtrl &c, AmItem &it, unsigned *err) {
    if (!wait_all(smem_u32(&c.ifull[slot]), ph, &c.abort_flag, err)) return false;
    const int4 *v = reinterpret_cast<const int4 *>(&c.item[slot]);
    reinterpret_cast<int4 *>(&it)[0] = v[0];
    reinterpret_cast<int4 *>(&it)[1] = v[1];
    reinterpret_cast<int4 *>(&it)[2] = v[2];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&c.iempty[slot]));
    if (++slot == AM_ITEMS) {
      slot = 0;
      ph ^= 1u;
    }
    return it.b > it.a;
  }
};

// Columns (row x head) of a step: those of the chunk's tokens in the block.
__device__ __forceinline__ int am_cols(const AmArgs &p, int T, int qb) {
  return min(p.TT, T - qb * p.TT) * p.G;
}

__global__ void __launch_bounds__(AM_THREADS, 1)
    am_weigh_kernel(const __grid_constant__ CUtensorMap q_map,
                    const __grid_constant__ CUtensorMap q1_map,
                    const __grid_constant__ CUtensorMap k_map, const AmArgs p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  static_assert(sizeof(AmCtrl) <= AM_CTL, "control block");
  AmCtrl &ctl = *reinterpret_cast<AmCtrl *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t k_s = smem_u32(smem_raw) + AM_CTL;
  if (k_s & 1023u) {  // the swizzled tiles need it; the same for every CTA
    if (threadIdx.x == 0) raise_err(p.err, ERR_TIMEOUT);
    pdl_wait();
    return;
  }
  const uint32_t q_s = k_s + 2 * AM_KBUF * PT_TILE;
  const uint32_t kfull = smem_u32(&ctl.kfull[0]), kempty = smem_u32(&ctl.kempty[0]);
  const uint32_t qfull = smem_u32(&ctl.qfull[0]), qempty = smem_u32(&ctl.qempty[0]);
  const uint32_t nfull = smem_u32(&ctl.nfull[0]), nempty = smem_u32(&ctl.nempty[0]);
  const uint32_t sfull = smem_u32(&ctl.sfull[0]), sempty = smem_u32(&ctl.sempty[0]);
  const uint32_t ffull = smem_u32(&ctl.ffull), fempty = smem_u32(&ctl.fempty);
  const uint32_t drain = smem_u32(&ctl.drain);

  if (threadIdx.x == 0) {
    for (int i = 0; i < AM_KBUF; ++i) {
      mbar_init(kfull + 8 * i, 1);
      mbar_init(kempty + 8 * i, 1);
    }
    for (int i = 0; i < AM_QST; ++i) {
      mbar_init(qfull + 8 * i, 1);
      mbar_init(qempty + 8 * i, 1);
      mbar_init(nfull + 8 * i, 1);
      mbar_init(nempty + 8 * i, 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + 8 * i, 1);
      mbar_init(sempty + 8 * i, 8);
    }
    mbar_init(drain, 1);
    mbar_init(ffull, 8);
    mbar_init(fempty, 8);
    for (int i = 0; i < AM_ITEMS; ++i) {
      mbar_init(smem_u32(&ctl.ifull[i]), 1);
      mbar_init(smem_u32(&ctl.iempty[i]), AM_READERS);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ctl.abort_flag = 0;
    ctl.kissued = ctl.qissued = 0;
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctl.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's: they start at 0
  volatile int *abort_flag = &ctl.abort_flag;
  pdl_wait();

  AmItem it;
  AmItems items;
  bool ok = true;
  if (warp < 16) {
    // ---------------------------------------------------------------- weights
    // (this warp's steps: those of its buffer)
    const int buf = warp >> 3, s = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
    const uint32_t ts =
        tmem + (uint32_t)(s * 256 + buf * 128) + ((uint32_t)((warp & 3) * 32) << 16);
    const unsigned long long cc = f2_pack(p.c2, p.c2);
    int turn = 0, st = 0;
    uint32_t sph = 0, nph = 0, fph = 0;
    while (ok && items.next(ctl, it, p.err)) {
      const int t = it.u * AM_TOK + s * PT_ROWS + r;  // this thread's token
      const int before = it.L - it.T;                 // tokens before the chunk
      float sum = 0.f, lost = 0.f;
      int qb = it.q0 + it.a % it.nq;
      for (int k = it.a; k < it.b; ++k) {
        const int cols = am_cols(p, it.T, qb);
        const bool mine = turn == buf;
        if (mine) {
          ok = wait_all2(sfull + 8 * buf, sph, nfull + 8 * st, nph, abort_flag, p.err);
          if (!ok) break;
          sph ^= 1u;
          tc_fence_after();
          // the first column that sees the token: row i sees its first before + i + 1
          // (a token can lie 2^30 before the rows, which times G passes 32 bits;
          // from 32 before them on, every lane's first column is below 0 either way)
          const int c0 = max(t - before - qb * p.TT, -32) * p.G;
          // (lanes are consecutive tokens: the warp's least and largest)
          const int cmin = __shfl_sync(0xffffffffu, c0, 0), cmax = cmin + 31 * p.G;
          unsigned long long la = f2_pack(0.f, 0.f), lb = la;
          const float *nl = ctl.nl[st];
          const int chunks = (cols + 31) >> 5;
#pragma unroll 1
          for (int c = max(0, cmin) >> 5; c < chunks; ++c) {
            uint32_t u[32];
            const float *v = reinterpret_cast<const float *>(u);
            tc_ld32_nowait(ts + 32 * c, u);
            tc_wait_ld();
            float e[32];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 n = *reinterpret_cast<const float4 *>(nl + 32 * c + i);
              f2_unpack(f2_fma(f2_pack(v[i], v[i + 1]), cc, f2_pack(n.x, n.y)), e[i], e[i + 1]);
              f2_unpack(f2_fma(f2_pack(v[i + 2], v[i + 3]), cc, f2_pack(n.z, n.w)), e[i + 2],
                        e[i + 3]);
            }
            if (32 * c < cmax || 32 * c + 32 > cols) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i < c0 || 32 * c + i >= cols) e[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              la = (i / 2) % 8 < AM_POLY
                       ? add_exp2_poly(la, e[i], e[i + 1])
                       : f2_add(la, f2_pack(ex2_approx(e[i]), ex2_approx(e[i + 1])));
              lb = (i / 2 + 1) % 8 < AM_POLY
                       ? add_exp2_poly(lb, e[i + 2], e[i + 3])
                       : f2_add(lb, f2_pack(ex2_approx(e[i + 2]), ex2_approx(e[i + 3])));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(sempty + 8 * buf);
            mbar_arrive(nempty + 8 * st);
          }
          float a0, a1, b0, b1;
          f2_unpack(la, a0, a1);
          f2_unpack(lb, b0, b1);
          // the sum with what its last rounding lost (bounded below: NaN once the
          // sum is infinite, which then stays so; a selection in the bound's place
          // is 2% slower)
          const float y = __fsub_rn((a0 + b0) + (a1 + b1), lost), z = __fadd_rn(sum, y);
          lost = fmaxf(__fsub_rn(__fsub_rn(z, sum), y), -3.4028235e38f);
          sum = z;
        }
        turn ^= 1;
        if (++st == AM_QST) {
          st = 0;
          nph ^= 1u;
        }
        if (++qb == it.q0 + it.nq) qb = it.q0;
      }
      if (!ok) break;
      // the sums over both buffers' steps; fin is read before it is written again
      if (buf == 1) {
        ok = wait_all(fempty, fph ^ 1u, abort_flag, p.err);
        fph ^= 1u;
        if (!ok) break;
        ctl.fin[s * PT_ROWS + r] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(ffull);
        continue;
      }
      ok = wait_all(ffull, fph, abort_flag, p.err);
      fph ^= 1u;
      if (!ok) break;
      sum += ctl.fin[s * PT_ROWS + r];
      __syncwarp();
      if (lane == 0) mbar_arrive(fempty);
      float v = t < it.L ? sum : 0.f;  // (slots past L hold anything)
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      if ((lane & 3) == 0 && t < it.L) {
        if (it.whole)
          p.mass[(size_t)it.seq * p.ld + (t >> 2)] += v;
        else
          p.rec[((size_t)blockIdx.x * 2 + (it.a == 0 ? 1 : 0)) * 64 + s * 32 + (r >> 2)] = v;
      }
    }
  } else if (warp == 16) {
    // -------------------------------------------------------------- MMA issuer
    const bool lead = elect_one();
    const uint64_t k_desc = sw128_desc(k_s), q_desc = sw128_desc(q_s);
    int kb = 0, st = 0, buf = 0;
    uint32_t kph = 0, qph = 0, eph = 1;
    while (ok && items.next(ctl, it, p.err)) {
      int qb = it.q0 + it.a % it.nq;
      bool fresh = true;  // a new pair of K tiles begins
      for (int k = it.a; k < it.b; ++k) {
        if (fresh) ok = wait_all(kfull + 8 * kb, kph, abort_flag, p.err);
        ok = ok && wait_all2(qfull + 8 * st, qph, sempty + 8 * buf, eph, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after();
        const int cols = am_cols(p, it.T, qb);
        const uint32_t idesc = f16_idesc(128, 16) + ((uint32_t)((cols + 15) / 16 - 1) << 18);
        const bool last = qb + 1 == it.q0 + it.nq || k + 1 == it.b;  // of this head's here
        if (lead) {
#pragma unroll 1
          for (int s = 0; s < 2; ++s) {
            const uint64_t da = k_desc + (uint64_t)((2 * kb + s) * (PT_TILE >> 4));
            const uint64_t db = q_desc + (uint64_t)(st * (PT_TILE >> 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint64_t o = (uint64_t)(((i >> 2) * PT_HALF + (i & 3) * 32) >> 4);
              tc_mma(s * 256 + buf * 128, da + o, db + o, idesc, i > 0 ? 1u : 0u);
            }
          }
          tc_commit(sfull + 8 * buf);
          tc_commit(qempty + 8 * st);
          if (last) tc_commit(kempty + 8 * kb);
        }
        __syncwarp();
        fresh = last;
        if (last && ++kb == AM_KBUF) {
          kb = 0;
          kph ^= 1u;
        }
        if (++st == AM_QST) {
          st = 0;
          qph ^= 1u;
        }
        buf ^= 1;
        if (buf == 0) eph ^= 1u;
        if (++qb == it.q0 + it.nq) qb = it.q0;
      }
    }
    if (ctl.abort_flag && lead) {  // gave up: wait for what was issued
      tc_commit(drain);
      mbar_wait(drain, 0, abort_flag, p.err, TC_DRAIN_LIMIT, false);
    }
    __syncwarp();
  } else if (warp == 17) {
    // ---------------------------------------------------------------- K tiles
    const bool lead = elect_one();
    int kb = 0, cnt = 0;
    uint32_t kph = 1;
    while (ok && items.next(ctl, it, p.err)) {
      // both tiles' pieces; the same pages for every head
      PagePieces t0;
      t0.start(p.pages, it.seq, it.L, 2 * it.u, lane);
      const int sl0 = t0.slot, p0 = t0.take(p.pages);
      t0.step(p.pages);
      const int sl1 = t0.slot, p1 = t0.take(p.pages);
      for (int h = it.a / it.nq; h <= (it.b - 1) / it.nq; ++h) {
        ok = wait_all(kempty + 8 * kb, kph, abort_flag, p.err) && cnt != p.k_tiles;
        if (!ok) break;
        const unsigned l0 = __ballot_sync(0xffffffffu, p0 >= 0);
        const unsigned l1 = __ballot_sync(0xffffffffu, p1 >= 0);
        const uint32_t bar = kfull + 8 * kb, dst = k_s + 2 * kb * PT_TILE;
        if (lead)
          mbar_arrive_expect(bar, (uint32_t)((__popc(l0) + __popc(l1)) * p.pages.box * 256));
        __syncwarp();
        issue_tile(p.pages, &k_map, dst, bar, p0, sl0, h, lead);
        issue_tile(p.pages, &k_map, dst + PT_TILE, bar, p1, sl1, h, lead);
        ++cnt;
        if (++kb == AM_KBUF) {
          kb = 0;
          kph ^= 1u;
        }
      }
    }
    if (lane == 0) ctl.kissued = cnt;
  } else if (warp == 18) {
    // ------------------------------------------------- query blocks, their LSEs
    const bool lead = elect_one();
    int st = 0, cnt = 0;
    uint32_t ph = 1;
    // this lane's columns lane + 32 i: where their LSEs lie from the block's
    // first row on, and the values of the next step, read one step ahead
    int off[4];
    float n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      off[i] = (lane + 32 * i) / p.G * p.Hq + (lane + 32 * i) % p.G;
    auto read = [&](int h, int qb) {
      const int cols = am_cols(p, it.T, qb);
      const float *l = p.lse + (size_t)(it.r0 + qb * p.TT) * p.Hq + h * p.G;
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = lane + 32 * i < cols ? __ldg(l + off[i]) : INFINITY;
    };
    while (ok && items.next(ctl, it, p.err)) {
      int h = it.a / it.nq, qb = it.q0 + it.a % it.nq;
      read(h, qb);
      for (int k = it.a; k < it.b; ++k) {
        const int cols = am_cols(p, it.T, qb), row = it.r0 + qb * p.TT, hk = h;
        float nl[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) nl[i] = n[i];
        if (++qb == it.q0 + it.nq) {
          qb = it.q0;
          ++h;
        }
        if (k + 1 < it.b) read(h, qb);
        ok = wait_all2(qempty + 8 * st, ph, nempty + 8 * st, ph, abort_flag, p.err);
        if (!ok) break;
        if (lead) {
          const uint32_t bar = qfull + 8 * st, dst = q_s + st * PT_TILE;
          const int toks = cols / p.G;
          if (toks <= AM_FEW) {
            mbar_arrive_expect(bar, (uint32_t)(cols * 256));
            for (int i = 0; i < toks; ++i)
              for (int x = 0; x < 2; ++x)
                tma_load_3d(dst + x * PT_HALF + i * p.G * 128, &q1_map, bar, x * 64, hk * p.G,
                            row + i);
          } else {
            mbar_arrive_expect(bar, (uint32_t)(p.TT * p.G * 256));
            for (int x = 0; x < 2; ++x)
              tma_load_3d(dst + x * PT_HALF, &q_map, bar, x * 64, hk * p.G, row);
          }
        }
        __syncwarp();
        // no weight where the LSE is -inf, nor in columns without a row
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ctl.nl[st][lane + 32 * i] =
              nl[i] == -INFINITY ? -INFINITY : -nl[i] * 1.4426950408889634f;
        __syncwarp();
        if (lane == 0) mbar_arrive(nfull + 8 * st);
        ++cnt;
        if (++st == AM_QST) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (lane == 0) ctl.qissued = cnt;
  } else {
    // --------------------------------------------------------- the items, ahead
    if (lane == 0) {
      const int n = p.hdr[0];
      const long long total = p.base[p.S];
      long long at = 0, hi = 0;
      if (total > 0 && (int)blockIdx.x < n) {
        at = am_bound(total, blockIdx.x, n);
        hi = am_bound(total, blockIdx.x + 1, n);
      }
      for (int i = 0;; ++i) {
        const int slot = i % AM_ITEMS;
        AmItem x = {};
        if (at < hi) {
          const long long first = am_find(p, at, x);
          x.a = (int)(at - first);
          x.b = (int)min((long long)x.steps, hi - first);
          x.whole = x.a == 0 && x.b == x.steps;
          at = first + x.b;
        }
        // (for as long as an item takes: Hkv x up to 4,096 query blocks)
        if (!wait_bar(smem_u32(&ctl.iempty[slot]), (uint32_t)((i / AM_ITEMS) & 1) ^ 1u, abort_flag,
                      p.err, PT_LONG_ROUNDS))
          break;
        ctl.item[slot] = x;
        mbar_arrive(smem_u32(&ctl.ifull[slot]));
        if (x.a == x.b) break;
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (ctl.abort_flag && threadIdx.x == 0) {  // copies that were issued
    for (int i = 0; i < AM_KBUF; ++i) {
      const int k = ctl.kissued - 1 - i;
      if (k >= 0)
        mbar_wait(kfull + 8 * (k % AM_KBUF), (uint32_t)((k / AM_KBUF) & 1), abort_flag, p.err,
                  TC_DRAIN_LIMIT, false);
    }
    for (int i = 0; i < AM_QST; ++i) {
      const int q = ctl.qissued - 1 - i;
      if (q >= 0)
        mbar_wait(qfull + 8 * (q % AM_QST), (uint32_t)((q / AM_QST) & 1), abort_flag, p.err,
                  TC_DRAIN_LIMIT, false);
    }
  }
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// One block of 64 threads per CTA of the weigh kernel: the item that started
// there and went on in the next ones; its pieces are added in order.
__global__ void __launch_bounds__(64) am_join_kernel(const AmArgs p) {
  pdl_wait();
  const int c0 = blockIdx.x, i = threadIdx.x, n = p.hdr[0];
  const long long total = p.base[p.S];
  if (total == 0 || c0 + 1 >= n) return;
  const long long end = am_bound(total, c0 + 1, n);
  AmItem it;
  const long long first = am_find(p, end - 1, it);
  if (first < am_bound(total, c0, n)) return;  // began in an earlier CTA
  const int c1 = am_owner(total, first + it.steps - 1, n);
  const int t = it.u * AM_TOK + 4 * i;
  if (c1 == c0 || t >= it.L) return;
  double sum = 0.0;  // (up to one piece per SM)
  for (int c = c0; c <= c1; ++c) sum += __ldcg(p.rec + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * 64 + i);
  p.mass[(size_t)it.seq * p.ld + (t >> 2)] += (float)sum;
}

struct AmLayout {
  size_t base, rec, bytes;
  int ctas;
};
AmLayout am_layout(int S) {
  AmLayout l;
  l.ctas = device_sm_count();
  l.base = 256;
  l.rec = l.base + (8 * ((size_t)S + 1) + 255) / 256 * 256;
  l.bytes = l.rec + (size_t)l.ctas * 2 * 64 * 4;
  return l;
}

}  // namespace

size_t attention_mass_ws_bytes(const qsa_dims &d, int S, int Nq) {
  (void)d;
  (void)Nq;
  return am_layout(S).bytes;
}

cudaError_t launch_attention_mass(const qsa_dims &d, const qsa_cache &c, int S,
                                  const int32_t *seq_lens, const int32_t *row_start, int Nq,
                                  const void *q, const float *lse, const float *mass_in,
                                  float *mass, int ld, void *ws, unsigned *err, cudaStream_t st) {
  cudaError_t e;
  EncodeTiledFn enc = encode_tiled_fn(&e);
  if (e != cudaSuccess) return e;
  if (enc == nullptr) return cudaErrorNotSupported;
  const AmLayout l = am_layout(S);
  char *w = static_cast<char *>(ws);
  AmArgs a;
  a.pages = paged_tiles(d, c, err);
  a.seq_lens = seq_lens;
  a.row_start = row_start;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass = mass;
  a.hdr = reinterpret_cast<int *>(w);
  a.base = reinterpret_cast<long long *>(w + l.base);
  a.rec = reinterpret_cast<float *>(w + l.rec);
  a.S = S;
  a.Nq = Nq;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.G = d.Hq / d.Hkv;
  a.TT = 128 / a.G;
  a.ld = ld;
  a.k_tiles = debug_stall_dense();
  a.c2 = d.scale * 1.4426950408889634f;
  a.err = err;
  // the copy of mass_in (none where it is mass itself), 16 KB a block
  int copies = 0;
  if (mass_in != mass)
    copies = (int)std::min<long long>(2LL * l.ctas, ((long long)S * ld + 4095) / 4096);
  e = launch_pdl(am_plan_kernel, 1 + copies, AM_PLAN_THREADS, 0, st, a, l.ctas);
  if (e != cudaSuccess || Nq == 0) return e;
  CUtensorMap q_map, q1_map, k_map;
  if (!query_map(enc, &q_map, q, d, Nq, a.TT) || !query_map(enc, &q1_map, q, d, Nq, 1) ||
      !pool_map(enc, &k_map, c.k_pool, d, c, a.pages.box))
    return cudaErrorInvalidValue;
  e = ensure_dynamic_smem(reinterpret_cast<const void *>(am_weigh_kernel), AM_SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(am_weigh_kernel, l.ctas, AM_THREADS, AM_SMEM, st, q_map, q1_map, k_map, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(am_join_kernel, l.ctas, 64, 0, st, a);
}

}  // namespace qsa
