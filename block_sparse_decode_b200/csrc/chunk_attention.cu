// qsa_chunk_attention: dense causal attention of the rows of appended chunks
// over the paged cache.
//
//   z_t = scale q.K_t for the row's len = L - T + i + 1 first tokens,
//   LSE = ln sum e^(z_t), out = sum e^(z_t - LSE) V_t
//
// Three kernels, chained by programmatic dependent launch:
//   plan    one CTA: the list of groups (up to 2 * TT tokens of one chunk,
//           TT = 128 / G) and the prefix of their work; an item is a group and
//           a KV head, its steps the 128-token tiles of the cache that its
//           last row sees;
//   attend  one CTA per SM over an equal range of the flattened steps, so that
//           one long sequence and many short ones fill the machine alike. An
//           item that several CTAs share leaves partial results in the
//           workspace. A long range of steps is done in parts of 1,024, which
//           are added up there;
//   join    merges those by their LSEs.
//
// attend: the G query heads of a KV head share its K and V, so a tile of 128
// MMA rows holds TT tokens x G heads. An item has two such tiles, one per
// slot, that use the same K and V (a group of at most TT tokens has one: its
// slots then take the odd and even steps, and are merged at the end). Per
// step and slot S = Q K^T (M = N = K = 128), the softmax of S as bf16 P in
// tensor memory over S itself, and O += P V, both tcgen05. While one slot's
// warps work on its softmax, the tensor cores work for the other.
//   warps 0-7, 8-15 softmax of slot 0, 1: a thread holds half a row of S (two
//                   warps hold a row's halves, and exchange its maximum)
//                   At an item's end each writes half of the rows' results
//   warps 16-19     rescale O where a maximum grew
//   warp 20         issues the MMAs
//   warp 21, 22     TMA of K tiles; of V tiles, whose rows past L_s are set to
//                   zero (0 * NaN in a stale slot would reach the sum)
//   warp 23         announces the items to the other warps, one or two ahead,
//                   and loads their query tiles
// The maximum is held in the exponent's unit (log2) and rounded up to a whole
// number, so every rescaling is by a power of two and exact, and it is only
// raised when it grew by more than 8 since O was last rescaled (P stays below
// 256, the sums in fp32): few tiles rescale at all.
// P is rounded to bf16 (2^-8 of a weight, as V's own precision), the row sum
// adds the fp32 values.
// Every mbarrier wait is bounded; after a timeout the roles stop, wait for
// their copies and MMAs, and free the tensor memory.
//
// Measured (B200, 32 query and 4 KV heads): 4,096 rows at 65,536 tokens in
// 4.6-4.8 ms (0.89-0.93 PFLOP/s; 4.06 ms in the first passes, until the 1 kW
// cap lowers the clock to 1.5 GHz). A step of both slots takes about 4,200
// clocks: 2,560 for a slot's softmax, 1,660 for its products and the next
// scores, which the other slot's softmax covers in part. The tensor memory has
// no room for a third S. One token over 32 x 32,768 tokens: 340 us before the
// cap acts, 359-392 after; its bytes take 328 at the copy rate. Tried, and
// slower: S in halves of 64 tokens, double buffered (4.7 -> 5.5 ms); the masks
// of a chunk's last tiles inside the softmax loop (4.58 -> 4.91 ms); some of
// the exponentials as a polynomial on the fp32 units.
#include <cuda.h>

#include <algorithm>
#include <cstdlib>

#include "common.cuh"
#include "launch.h"
#include "paged_tiles.cuh"
#include "tc_util.cuh"
#include "umma_desc.h"

namespace qsa {
namespace {

constexpr int CA_D = 128;
constexpr int CA_KT = 128;  // cache tokens per step
constexpr int CA_THREADS = 768;
constexpr int CA_STAGES = 5;
constexpr int CA_ITEMS = 4;     // items announced ahead
constexpr int CA_READERS = 23;  // warps that read them
// control block, padded to the tiles' alignment, and the tiles: 227 KB exactly
constexpr uint32_t CA_CTL = 3 * 1024;
constexpr size_t CA_SMEM = CA_CTL + 2 * PT_TILE + CA_STAGES * PT_TILE;
constexpr int CA_PLAN_THREADS = 1024;
// An item's start (queries, first tiles, its result) counts as this many steps
// where a CTA has at least CA_MANY units: ragged chunks 327 us without, 280, 247,
// 254 and 253 with 2, 3, 4 and 6. (With fewer, every CTA gets a step or two: a
// single sequence's time is latency.)
constexpr int CA_START = 3, CA_MANY = 16;
constexpr int CA_MAX_UNITS = 1 << 30;  // units of a CTA (about 20 minutes of work)
// Chunk tokens that are loaded one by one into a tile that begins as zeros: MMA
// rows of zeros draw less power than other tokens' (the part throttles at 1 kW)
constexpr int CA_FEW = 4;
// Steps after which O leaves the tensor memory: the tensor cores' additions to it
// truncate, a bias of up to 2^-23 of the sum each, 8 a step. Parts of 1,024 steps
// (131,072 tokens) keep that below 2^-10 of sum w |V|. Measured with equal scores
// and positive V in one item of 2^26 tokens: 19% off without parts, 0.01% with them
// (2^28: 51%, 0.012%), at 2% of the time. What the parts add up to is fp32,
// rounded to nearest.
constexpr int CA_PART = 1024;
constexpr float CA_LAZY = 8.f;  // growth of the maximum that is left in the sums

struct CaArgs {
  const int32_t *seq_lens, *row_start;
  int4 *first;       // [CTAs] {group, head, unit, end}: where a CTA's range begins (CaWalk); w < 0: empty
  int4 *shared;      // [CTAs] {group, head, last CTA, -}: the item that goes on past it, or group -1
  int *hdr;          // [0] steps that an item's start counts as
  long long *gpre;   // [Gmax + 1] prefix of the groups' units
  int4 *ginfo;       // [2 Gmax] {seq, first row, tokens, steps}, {tokens its first row sees, L, -, -}
  float *rec_lse;    // [CTAs][2][2][128]
  float *rec_o;      // [CTAs][2][2][128][128]
  float2 *part;      // [CTAs][2][2][128] sum and maximum (log2) of an item's parts so far
  void *out;
  float *lse;
  PagedTiles pages;
  int S, Nq, Gmax, Hq, Hkv, G, TT, out_bf16;
  int k_tiles;  // failure injection: K tiles that a CTA issues (debug_stall_dense())
  float scale;
  unsigned *err;
};

// ------------------------------------------------------------------ plan

__device__ long long ca_scan(long long v, long long *wsum, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  __syncthreads();
  long long off = 0, tot = 0;
  for (int i = 0; i < CA_PLAN_THREADS / 32; ++i) {
    if (i < warp) off += wsum[i];
    tot += wsum[i];
  }
  __syncthreads();
  *total = tot;
  return off + x - v;
}

__device__ __forceinline__ long long ca_bound(long long total, int c, int n) {
  return total * c / n;
}
// The CTA whose range holds a unit.
__device__ __forceinline__ int ca_owner(long long total, long long unit, int n) {
  int c = (int)(unit * n / total);
  while (c + 1 < n && ca_bound(total, c + 1, n) <= unit) ++c;
  while (c > 0 && ca_bound(total, c, n) > unit) --c;
  return c;
}

// Units of one step: a step of two tiles counts twice that of one.
__device__ __forceinline__ int ca_weight(int ntok, int TT) { return ntok > TT ? 2 : 1; }

__global__ void __launch_bounds__(CA_PLAN_THREADS) ca_plan_kernel(CaArgs a, int ctas) {
  __shared__ long long wsum[CA_PLAN_THREADS / 32];
  __shared__ long long pre_s[CA_PLAN_THREADS + 1];  // the prefix, where it is short
  const int tid = threadIdx.x;
  pdl_wait();
  const int GT = 2 * a.TT;  // tokens of a group
  long long gbase = 0;
  for (int base = 0; base < a.S; base += CA_PLAN_THREADS) {
    const int s = base + tid;
    int ng = 0, r0 = 0, T = 0, L = 0;
    if (s < a.S) {
      r0 = a.row_start[s];
      const int r1 = a.row_start[s + 1];
      L = a.seq_lens[s];
      T = r1 - r0;
      if (r0 < 0 || r1 < r0 || r1 > a.Nq || T > L || L > PT_MAX_LEN ||
          (long long)L > (long long)a.pages.max_pages * a.pages.P)
        raise_err(a.err, ERR_LEN);
      else
        ng = (T + GT - 1) / GT;
    }
    long long tot;
    const long long off = gbase + ca_scan(ng, wsum, &tot);
    for (int i = 0; i < ng; ++i) {
      const long long g = off + i;
      if (g >= a.Gmax) {  // only overlapping chunks can need more groups than rows allow
        raise_err(a.err, ERR_LEN);
        break;
      }
      const int ntok = min(GT, T - i * GT);
      const int lim0 = L - T + i * GT + 1;
      const int steps = (lim0 + ntok - 1 + CA_KT - 1) / CA_KT;
      a.ginfo[2 * g] = make_int4(s, r0 + i * GT, ntok, steps);
      a.ginfo[2 * g + 1] = make_int4(lim0, L, 0, 0);
    }
    gbase += tot;
  }
  const int G = (int)min(gbase, (long long)a.Gmax);
  __syncthreads();
  // the groups' steps, to see whether there are enough to count the items'
  // starts too
  long long work = 0;
  for (int base = 0; base < G; base += CA_PLAN_THREADS) {
    const int g = base + tid;
    long long n = 0, tot;
    if (g < G) n = (long long)a.Hkv * a.ginfo[2 * g].w * ca_weight(a.ginfo[2 * g].z, a.TT);
    ca_scan(n, wsum, &tot);
    work += tot;
  }
  const int start = work >= (long long)CA_MANY * ctas ? CA_START : 0;
  long long tbase = 0;
  for (int base = 0; base < G; base += CA_PLAN_THREADS) {
    const int g = base + tid;
    long long n = 0;
    if (g < G) {
      const int4 gi = a.ginfo[2 * g];
      n = (long long)a.Hkv * (gi.w + start) * ca_weight(gi.z, a.TT);
    }
    long long tot;
    const long long off = tbase + ca_scan(n, wsum, &tot);
    if (g < G) {
      if (G <= CA_PLAN_THREADS) pre_s[g] = off;
      else a.gpre[g] = off;
    }
    tbase += tot;
  }
  // a range of the units counts in 32 bits (CaWalk; an item has 2^24 at most)
  if (tbase / ctas >= CA_MAX_UNITS) {
    if (tid == 0) raise_err(a.err, ERR_LEN);
    tbase = 0;
  }
  if (tid == 0) {
    (G <= CA_PLAN_THREADS ? pre_s : a.gpre)[G] = tbase;
    a.hdr[0] = start;
  }
  __syncthreads();
  // where every CTA's range begins, and the items that CTAs share. Every range
  // is at least as long as the units between two steps, so every CTA inside an
  // item's range has a step of it
  const long long *pre = G <= CA_PLAN_THREADS ? pre_s : a.gpre, total = tbase;
  const int n = (int)min((long long)ctas, max(1LL, total / (2 * (start + 1))));
  for (int c = tid; c < ctas; c += CA_PLAN_THREADS) {
    int4 f = make_int4(0, 0, 0, -1), e = make_int4(-1, 0, 0, 0);
    if (total > 0 && c < n) {
      const long long lo = ca_bound(total, c, n), hi = ca_bound(total, c + 1, n);
      auto find = [&](long long unit, int4 &gi, int &h, long long &u0) {
        int x = 0, y = G - 1;  // the last group that starts at or before the unit
        while (x < y) {
          const int m = (x + y + 1) >> 1;
          if (pre[m] <= unit) x = m; else y = m - 1;
        }
        gi = a.ginfo[2 * x];
        const long long per = (long long)ca_weight(gi.z, a.TT) * (gi.w + start);
        h = (int)((unit - pre[x]) / per);
        u0 = pre[x] + h * per;
        return x;
      };
      int4 gi;
      int h;
      long long u0;
      int g = find(lo, gi, h, u0);
      f = make_int4(g, h, (int)(u0 - lo), (int)(hi - lo));
      g = find(hi - 1, gi, h, u0);
      if (u0 >= lo && gi.w > 1) {  // began here
        const int w = ca_weight(gi.z, a.TT);
        const int last = ca_owner(total, u0 + (long long)w * (start + gi.w - 1), n);
        if (last > c) e = make_int4(g, h, last, 0);
      }
    }
    a.first[c] = f;
    a.shared[c] = e;
  }
}

// ------------------------------------------------------------------ items

// The items of one CTA's range, in order. An item of n steps has w (start + n)
// units: with many steps in all, an item's start (queries, first tiles, its
// result) counts as CA_START steps. Units are counted from the range's start,
// which keeps them in 32 bits.
struct CaWalk {
  int u, hi;  // the item's first unit (before 0: it began in an earlier CTA), the range's end
  int g, h, w, start;
  int4 gi;  // {seq, first row, tokens, steps}
  int lim0, L;
  int a = 0, b = 0;  // this CTA's steps of the item
  const CaArgs &p;

  __device__ CaWalk(const CaArgs &args, int c) : p(args) {
    const int4 f = p.first[c];
    start = p.hdr[0];
    g = f.x;
    h = f.y;
    u = f.z;
    hi = f.w;
    w = 1;
    if (hi > 0) load();
  }
  __device__ void load() {
    gi = p.ginfo[2 * g];
    const int4 m = p.ginfo[2 * g + 1];
    lim0 = m.x;
    L = m.y;
    w = ca_weight(gi.z, p.TT);
  }
  // The steps [a, b) of the next item with any here (the range may start
  // inside an item's last step); false when the range is done.
  __device__ bool next(bool first) {
    for (;;) {
      if (!first) {
        u += w * (gi.w + start);
        if (u >= hi) return false;
        if (++h == p.Hkv) {
          h = 0;
          ++g;
          load();
        }
      }
      first = false;
      if (u >= hi) return false;
      // step 0 begins at the item's first unit, step j at unit w (start + j)
      a = u < 0 ? max(1, (-u + w - 1) / w - start) : 0;
      b = min(gi.w, max(1, (hi - u + w - 1) / w - start));
      if (a < b) return true;
    }
  }
};

// An item as the roles see it: this CTA's steps [a, b), or a part of them (of
// CA_PART, the last one of 2 to CA_PART + 1, so that both slots have a step of
// every part but a CTA's first), none at the end of the range. Slot 0's rows of a two-tile item see its steps below n0; a one-tile
// item (n0 = -1) has its steps in turn on slot 0 and slot 1.
struct __align__(16) CaItem {
  int a, b, n0, ntok;
  int h, row0, lim0, whole;  // whole: the result is final, else a record
  int seq, L, part, rec;     // part: 1 adds to the parts before, 2 more follow; rec: which record
  __device__ bool two() const { return n0 >= 0; }
};
__device__ __forceinline__ bool ca_active(int s, int j, int a, int n0) {
  return n0 >= 0 ? (s == 1 || j < n0) : ((j - a) & 1) == s;
}

// ------------------------------------------------------------------ attend

struct CaCtrl {
  uint64_t full[CA_STAGES], empty[CA_STAGES];
  uint64_t qfull, qempty, vraw, drain;
  uint64_t sfull[2], ready[2], ready2[2], corr[2], ofull[2], fin, fread;
  uint64_t ifull[CA_ITEMS], iempty[CA_ITEMS];
  CaItem item[CA_ITEMS];
  uint32_t tmem;
  int abort_flag;
  int qissued;
  int last[CA_STAGES];  // the phase of a stage's last tile (+ 2: there is one)
  __nv_bfloat16 sc[2][128];      // a row's rescaling, a power of two
  // the row maxima of the two column halves; at an item's end a row's sum and
  // its maximum (log2)
  float pm[2][2][128];
};

__device__ __forceinline__ void ca_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void ca_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// D (tensor memory) += A (tensor memory) * B (shared memory)
__device__ __forceinline__ void ca_mma_ts(uint32_t d, uint32_t a, uint64_t db, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(db), "r"(idesc), "r"(accumulate));
}
// 32 columns of a tile with masked ones (or under a scale that is not
// positive, which is then applied here): -inf from column n on.
__device__ __forceinline__ void ca_masked(uint32_t taddr, int n, float sl2, float (&v)[32]) {
  tc_ld32_nowait(taddr, *reinterpret_cast<uint32_t(*)[32]>(v));
  tc_wait_ld();
  const float pre = sl2 > 0.f ? 1.f : sl2;
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = i < n ? v[i] * pre : -INFINITY;
}

// The ring of K and V tiles is filled in the order in which the MMAs use it.
// Two tiles: K_0 V_0 K_1 V_1 ... One tile, whose slots work on two steps at a
// time: K_0 K_1 V_0 K_2 V_1 ... K_{n-1} V_{n-2} V_{n-1}. Distance from tile i of
// an item's n to the next one of its kind (after the last: to the next item),
// and of the first V tile from the item's start.
__device__ __forceinline__ int ca_next_k(bool two, int i, int n) {
  return two ? 2 : i == n - 1 ? (n == 1 ? 2 : 3) : i == 0 ? 1 : 2;
}
__device__ __forceinline__ int ca_next_v(bool two, int i, int n) {
  return i == n - 1 ? 1 : !two && i == n - 2 ? 1 : 2;
}
__device__ __forceinline__ int ca_first_v(bool two, int n) { return two || n == 1 ? 1 : 2; }
// A place in the ring: stage and phase.
struct CaPlace {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void move(int d) {
    st += d;
    if (st >= CA_STAGES) {
      st -= CA_STAGES;
      ph ^= 1u;
    }
  }
};

// The next item of a role's warp (whole warp); false at the end or after an
// abort. Its fields are in registers afterwards and its slot is given back.
struct CaItems {
  int at = 0;
  __device__ __forceinline__ bool next(CaCtrl &c, CaItem &it, unsigned *err) {
    const int i = at % CA_ITEMS;
    if (!wait_warp(smem_u32(&c.ifull[i]), (uint32_t)((at / CA_ITEMS) & 1), &c.abort_flag, err))
      return false;
    ++at;
    const int4 *v = reinterpret_cast<const int4 *>(&c.item[i]);
    reinterpret_cast<int4 *>(&it)[0] = v[0];
    reinterpret_cast<int4 *>(&it)[1] = v[1];
    reinterpret_cast<int4 *>(&it)[2] = v[2];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&c.iempty[i]));
    return it.b > it.a;
  }
};

// The result of an item's row, of this half's columns: the slot's own sum and
// maximum (l, m), and those of slot 1 (l1, m1) where it had a part of a one-tile
// item. A sum of 0: nothing seen, or no weight above 0 here; one that is NaN, from
// a score that is NaN or +inf, goes on to the result and its LSE. With PARTS, what
// the parts before left (not yet divided by its sum) is in this thread's own record.
template <bool PARTS>
__device__ __forceinline__ void ca_finish(const CaArgs &p, const CaItem &it, int s, int half, int r,
                                          int tok, bool valid, bool has1, float l, float m, float l1,
                                          float m1) {
  const int warp = threadIdx.x >> 5;
  const size_t rec = ((size_t)blockIdx.x * 2 + it.rec) * 256 + s * 128 + r;
  const bool adds = PARTS && (it.part & 1) && valid, more = PARTS && (it.part & 2) != 0;
  const size_t mine = ((size_t)blockIdx.x * 4 + s * 2 + half) * 128 + r;
  float2 old = make_float2(0.f, -INFINITY);
  if (adds) old = p.part[mine];
  float M = fmaxf(l != 0.f ? m : -INFINITY, l1 != 0.f ? m1 : -INFINITY);
  if (PARTS) M = fmaxf(M, old.x != 0.f ? old.y : -INFINITY);
  const float e0 = l != 0.f ? ex2_approx(m - M) : 0.f;
  const float e1 = l1 != 0.f ? ex2_approx(m1 - M) : 0.f;
  const float e2 = adds && old.x != 0.f ? ex2_approx(old.y - M) : 0.f;
  float sum = e0 * l + e1 * l1;
  if (PARTS) sum += e2 * old.x;
  // (e0 to e2 are powers of two: one division gives what three would)
  const float inv = more ? 1.f : sum != 0.f ? 1.f / sum : 0.f;
  const float f0 = e0 * inv, f1 = e1 * inv, f2 = e2 * inv;
  const bool whole = it.whole != 0;
  if (more && valid) p.part[mine] = make_float2(sum, M);
  const size_t row = (size_t)(it.row0 + tok) * p.Hq + (size_t)it.h * p.G + r % p.G;
  if (valid && half == 0 && !more) {
    const float lse = sum != 0.f ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    if (!whole) p.rec_lse[rec] = lse;
    else if (p.lse != nullptr) p.lse[row] = lse;
  }
  const uint32_t to =
      (uint32_t)(256 + s * 128 + half * 64) + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    float o[32];
    tc_ld32_nowait(to + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(o));
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = f0 != 0.f ? o[i] * f0 : 0.f;
    if (has1) {
#pragma unroll
      for (int k = 0; k < 32; k += 16) {
        float o1[16];
        tc_ld16(to + 128 + 32 * c + k, o1);
        if (f1 != 0.f) {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[k + i] = fmaf(o1[i], f1, o[k + i]);
        }
      }
    }
    if (!valid) continue;
    const int col = half * 64 + 32 * c;
    if (adds && f2 != 0.f) {
      const float4 *d = reinterpret_cast<const float4 *>(p.rec_o + rec * CA_D + col);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v = d[i];
        o[4 * i] = fmaf(v.x, f2, o[4 * i]);
        o[4 * i + 1] = fmaf(v.y, f2, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(v.z, f2, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(v.w, f2, o[4 * i + 3]);
      }
    }
    if (whole && p.out_bf16) {
      uint4 *d =
          reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + row * CA_D + col);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]),
                          pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                          pack_bf16x2(o[8 * i + 4], o[8 * i + 5]),
                          pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
    } else {
      float4 *d = reinterpret_cast<float4 *>(
          (whole ? static_cast<float *>(p.out) + row * CA_D : p.rec_o + rec * CA_D) + col);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
  }
}
__global__ void __launch_bounds__(CA_THREADS, 1)
    ca_attend_kernel(const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap q1_map,
                     const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const CaArgs p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  static_assert(sizeof(CaCtrl) <= CA_CTL, "control block");
  CaCtrl &ctl = *reinterpret_cast<CaCtrl *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t q_s = smem_u32(smem_raw) + CA_CTL;
  if (q_s & 1023u) {  // the swizzled tiles need it; the same for every CTA
    if (threadIdx.x == 0) raise_err(p.err, ERR_TIMEOUT);
    pdl_wait();
    return;
  }
  const uint32_t ring = q_s + 2 * PT_TILE;
  const uint32_t full0 = smem_u32(&ctl.full[0]), empty0 = smem_u32(&ctl.empty[0]);
  const uint32_t qfull = smem_u32(&ctl.qfull), qempty = smem_u32(&ctl.qempty);
  const uint32_t vraw = smem_u32(&ctl.vraw), drain = smem_u32(&ctl.drain);
  const uint32_t sfull = smem_u32(&ctl.sfull[0]), ready = smem_u32(&ctl.ready[0]);
  const uint32_t ready2 = smem_u32(&ctl.ready2[0]), fread = smem_u32(&ctl.fread);
  const uint32_t fin = smem_u32(&ctl.fin);
  const uint32_t corr = smem_u32(&ctl.corr[0]), ofull = smem_u32(&ctl.ofull[0]);

  if (threadIdx.x == 0) {
    for (int i = 0; i < CA_STAGES; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    mbar_init(vraw, 1);
    mbar_init(drain, 1);
    mbar_init(fin, 4);
    mbar_init(fread, 8);
    for (int i = 0; i < CA_ITEMS; ++i) {
      mbar_init(smem_u32(&ctl.ifull[i]), 1);
      mbar_init(smem_u32(&ctl.iempty[i]), CA_READERS);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(sfull + 8 * s, 1);
      mbar_init(ready + 8 * s, 8);  // 4 softmax and 4 correction warps
      mbar_init(ready2 + 8 * s, 4);
      mbar_init(corr + 8 * s, 4);
      mbar_init(ofull + 8 * s, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ctl.abort_flag = 0;
    ctl.qissued = 0;
    for (int i = 0; i < CA_STAGES; ++i) ctl.last[i] = 0;
  }
  if (warp == 20) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctl.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  for (uint32_t i = threadIdx.x * 16; i < PT_TILE; i += CA_THREADS * 16)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(q_s + i), "r"(0) : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's: they start at 0
  volatile int *abort_flag = &ctl.abort_flag;
  const float sl2 = p.scale * 1.4426950408889634f;
  pdl_wait();

  if (warp < 16) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    const int s = warp >> 3, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
    const uint32_t ts =
        tmem + (uint32_t)(s * 128 + half * 64) + ((uint32_t)((warp & 3) * 32) << 16);
    const float c2 = sl2 > 0.f ? sl2 : 1.f;
    const uint32_t written = (half == 0 ? ready : ready2) + 8 * s;  // this half of P is
    const int pair = 1 + s * 4 + (warp & 3);  // barrier of the two warps of these rows
    uint32_t sph = 0, fph = 0, oph = 0;
    bool ended = false;  // slot 1's part of a one-tile item, which slot 0 has to read first
    // The two warps stop together: every wait that may give up is followed by
    // their barrier, which combines the outcomes.
    auto both = [&](bool ok) {
      uint32_t r;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, 64, p;\n"
          " selp.b32 %0, 1, 0, q;\n}"
          : "=r"(r)
          : "r"((uint32_t)ok), "r"(pair)
          : "memory");
      return r != 0;
    };
    CaItems items;
    CaItem it;
    bool ok = true;
    while (both(ok && items.next(ctl, it, p.err))) {
      const int n0 = it.n0;
      const int tok = (it.two() ? s * p.TT : 0) + r / p.G;
      const bool valid = r < p.TT * p.G && tok < it.ntok;
      const int lim = valid ? it.lim0 + tok : 0x7fffffff;
      const bool live = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.f;
      bool any = false;
      for (int j = it.a; j < it.b; ++j) {
        if (!ca_active(s, j, it.a, n0)) continue;
        if (ended) {
          ok = wait_all(fread, fph, abort_flag, p.err);
          fph ^= 1u;
          ended = false;
        }
        ok = ok && wait_all(sfull + 8 * s, sph, abort_flag, p.err);
        sph ^= 1u;
        tc_fence_after();
        // this row's tokens of this half of the tile
        const int nv = lim - j * CA_KT - half * 64;
        const bool mask = __any_sync(0xffffffffu, nv < 64) || !(sl2 > 0.f);
        float mt = -INFINITY;
        if (!ok || !live) {
        } else if (!mask) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float v[32];
            tc_ld32_nowait(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v));
            tc_wait_ld();
            float t0 = mt, t1 = v[0], t2 = v[1], t3 = v[2];
            t0 = max3(t0, v[3], v[4]);
            t1 = max3(t1, v[5], v[6]);
            t2 = max3(t2, v[7], v[8]);
            t3 = max3(t3, v[9], v[10]);
            t0 = max3(t0, v[11], v[12]);
            t1 = max3(t1, v[13], v[14]);
#pragma unroll
            for (int i = 15; i < 31; i += 8) {
              t0 = max3(t0, v[i], v[i + 1]);
              t1 = max3(t1, v[i + 2], v[i + 3]);
              t2 = max3(t2, v[i + 4], v[i + 5]);
              t3 = max3(t3, v[i + 6], v[i + 7]);
            }
            mt = max3(max3(t0, t1, v[31]), t2, t3);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float v[32];
            ca_masked(ts + 32 * c, nv - 32 * c, sl2, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) mt = fmaxf(mt, v[i]);
          }
        }
        ctl.pm[s][half][r] = mt;
        ok = both(ok);
        if (!ok) break;
        if (live) {
          // the row's new maximum over both halves, its rescaling for the
          // correction warps, and what the exponentials subtract
          mt = fmaxf(mt, ctl.pm[s][half ^ 1][r]);
          const float mt2 = ceilf(mt * c2);
          float f = 1.f;
          if (mt2 > m + CA_LAZY || m == -INFINITY) {
            f = m == -INFINITY ? (any ? 0.f : 1.f) : ex2_approx(m - mt2);
            m = fmaxf(m, mt2);
          }
          if (any) {
            l *= f;
            if (half == 0) {
              ctl.sc[s][r] = __float2bfloat16_rn(valid ? f : 1.f);
              __syncwarp();
              if (lane == 0) mbar_arrive(corr + 8 * s);
            }
          }
          const float off = m == -INFINITY ? 0.f : m;
          const unsigned long long cc = f2_pack(c2, c2), oo = f2_pack(-off, -off);
          unsigned long long la = f2_pack(0.f, 0.f), lb = la;
          // the exponentials in a loop over 32 columns, read again (the whole
          // row unrolled does not stay in the instruction cache); their bf16
          // pairs overwrite columns of this half already read
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float v[32];
            if (mask) {
              ca_masked(ts + 32 * c, nv - 32 * c, sl2, v);
            } else {
              tc_ld32_nowait(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v));
              tc_wait_ld();
            }
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float e0, e1;
              f2_unpack(f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), cc, oo), e0, e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              if (i % 2 == 0) la = f2_add(la, f2_pack(e0, e1));
              else lb = f2_add(lb, f2_pack(e0, e1));
              pk[i] = pack_bf16x2(e0, e1);
            }
            ca_st16(ts + 16 * c, pk);
          }
          float a0, a1, b0, b1;
          f2_unpack(la, a0, a1);
          f2_unpack(lb, b0, b1);
          l += (a0 + b0) + (a1 + b1);
          ca_wait_st();
          tc_fence_before();
          __syncwarp();
        } else if (any && half == 0 && lane == 0) {  // no rows here: P may hold anything
          mbar_arrive(corr + 8 * s);
        }
        if (lane == 0) mbar_arrive(written);
        any = true;
      }
      if (!ok) break;
      const size_t rec = ((size_t)blockIdx.x * 2 + it.rec) * 256 + s * 128 + r;
      if (!any) {  // slot 0's rows see none of this CTA's steps of a two-tile item
        if (it.two() && valid && half == 0) p.rec_lse[rec] = -INFINITY;
        continue;
      }
      // the item's end: the row's sum over both halves, then this half of the
      // result's columns, once the slot's last product is in. (First both warps
      // have to have read the last step's maxima, which the sums overwrite: no
      // further scores follow that would have waited for it.)
      both(true);
      ctl.pm[s][half][r] = l;
      both(true);
      l += ctl.pm[s][half ^ 1][r];
      // (past 2^30 the maximum is rounded by 64 and more, and weights of 2^-127 and
      // below or 2^128 and more would come of it)
      if (m > -INFINITY && fabsf(m) > 0x1p30f) l = NAN;
      ok = wait_all(ofull + 8 * s, oph, abort_flag, p.err);
      oph ^= 1u;
      tc_fence_after();
      const bool two = it.two();
      if (!two && s == 1) {  // one tile: slot 0 writes the result of both
        both(true);  // (the sums have been read)
        if (half == 0) {
          ctl.pm[1][0][r] = l;
          ctl.pm[1][1][r] = m;
          __syncwarp();
          if (lane == 0) mbar_arrive(fin);
        }
        ended = true;
        continue;
      }
      const bool has1 = !two && it.b - it.a > 1;  // slot 1 has a part
      float l1 = 0.f, m1 = -INFINITY;
      if (has1) {
        ok = ok && wait_all(fin, fph, abort_flag, p.err);
        fph ^= 1u;
        tc_fence_after();
        l1 = ctl.pm[1][0][r];
        m1 = ctl.pm[1][1][r];
      }
      if (ok && live) {
        if (it.part == 0) ca_finish<false>(p, it, s, half, r, tok, valid, has1, l, m, l1, m1);
        else ca_finish<true>(p, it, s, half, r, tok, valid, has1, l, m, l1, m1);
      }
      tc_fence_before();
      __syncwarp();
      if (has1 && lane == 0) mbar_arrive(fread);
    }
  } else if (warp < 20) {
    // ------------------------------------------------------------- correction
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int r = (warp & 3) * 32 + lane;
    const uint32_t to = tmem + 256u + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t cph = 0, rph = 0, began = 0;  // a bit per slot
    CaItems items;
    CaItem it;
    bool ok = true;
    while (ok && items.next(ctl, it, p.err)) {
      const int n0 = it.n0;
      // bits per slot: it had a step; the softmax warps of these rows have any
      // of the item's
      uint32_t any = 0, live = 0;
#pragma unroll 1
      for (int s = 0; s < 2; ++s)
        if (__any_sync(0xffffffffu, r < p.TT * p.G &&
                                        (it.two() ? s * p.TT : 0) + r / p.G < it.ntok))
          live |= 1u << s;
      for (int j = it.a; j < it.b && ok; ++j) {
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          if (!ok || !ca_active(s, j, it.a, n0)) continue;
          if ((any >> s) & 1u) {
            ok = wait_all(corr + 8 * s, (cph >> s) & 1u, abort_flag, p.err);
            if (!ok) continue;
            cph ^= 1u << s;
            const float f = (live >> s) & 1u ? __bfloat162float(ctl.sc[s][r]) : 1.f;
            if (__any_sync(0xffffffffu, f != 1.f)) {
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                float o[16];
                tc_ld16(to + s * 128 + 16 * c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= f;
                ca_st16(to + s * 128 + 16 * c, reinterpret_cast<const uint32_t *>(o));
              }
              ca_wait_st();
            }
          } else if ((began >> s) & 1u) {
            // an item's first step has nothing to rescale; but the step before
            // it has to be complete before this one's arrival counts
            ok = wait_all(ready + 8 * s, ((rph >> s) & 1u) ^ 1u, abort_flag, p.err);
            if (!ok) continue;
          }
          any |= 1u << s;
          began |= 1u << s;
          rph ^= 1u << s;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ready + 8 * s);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 20) {
      // -------------------------------------------------------------- MMA issuer
      constexpr uint32_t IDESC_S = f16_idesc(128, 128);
      constexpr uint32_t IDESC_O = f16_idesc(128, 128) | (1u << 16);  // B = V: MN-major
      CaItems items;
      CaItem it;
      uint32_t qph = 0, rph = 0;
      CaPlace kt, vt;  // the next K and V tile
      // V: 64-value halves PT_HALF apart (leading offset), 8-token groups 1024
      // bytes apart
      const uint64_t q_desc = sw128_desc(q_s), k_desc = sw128_desc(ring);
      const uint64_t v_desc = (k_desc & ~(0x3fffull << 16)) | ((uint64_t)(PT_HALF >> 4) << 16);
      bool ok = true;
      // the whole warp runs this loop, so that the operands of the MMAs are
      // warp-uniform; one elected lane issues them
      const bool lead = elect_one();
      while (ok && items.next(ctl, it, p.err)) {
        const bool two = it.two();
        const int a = it.a, b = it.b, n0 = it.n0, n = b - a, stride = two ? 1 : 2;
        // S_s = Q_s K^T with the K tile at the ring's next even position, by
        // the elected lane
        auto scores = [&](int s, bool last_use, bool last) {
          const uint64_t da = q_desc + (uint64_t)(two ? s * (PT_TILE >> 4) : 0);
          const uint64_t db = k_desc + (uint64_t)(kt.st * (PT_TILE >> 4));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint64_t o = (uint64_t)(((k >> 2) * PT_HALF + (k & 3) * 32) >> 4);
            tc_mma(s * 128, da + o, db + o, IDESC_S, k > 0 ? 1u : 0u);
          }
          tc_commit(sfull + 8 * s);
          if (last_use) {
            tc_commit(empty0 + 8 * kt.st);
            if (last) tc_commit(qempty);  // the query tiles' last use
          }
        };
        vt.move(ca_first_v(two, n));
        ok = wait_all(qfull, qph, abort_flag, p.err);
        for (int i = 0; i < (two ? 1 : 2) && ok && a + i < b; ++i) {
          ok = wait_all(full0 + 8 * kt.st, kt.ph, abort_flag, p.err);
          tc_fence_after();
          if (ok && lead) {
            const bool last = a + i == b - 1;
            if (two && a < n0) scores(0, false, false);
            scores(two ? 1 : i, true, last);
          }
          __syncwarp();
          kt.move(ca_next_k(two, i, n));
        }
        // few instructions between the waits, and the tiles' waits ahead of
        // P's, which arrives last: this warp's latency is on every slot's path
        for (int j = a; j < b && ok; ++j) {
          const int jn = j + stride;
          const int s0 = two ? (j < n0 ? 0 : 1) : ((j - a) & 1), s1 = two ? 1 : s0;
          const bool k_now = two && jn < b;  // (one tile: its K tile comes after this V tile)
          ok = wait_all2(full0 + 8 * vt.st, vt.ph, full0 + 8 * (k_now ? kt.st : vt.st),
                         k_now ? kt.ph : vt.ph, abort_flag, p.err);
#pragma unroll 1
          for (int s = s0; s <= s1 && ok; ++s) {
            const uint32_t ph = (rph >> s) & 1u;
            ok = wait_all(ready + 8 * s, ph, abort_flag, p.err);
            if (!ok) break;
            rph ^= 1u << s;
            tc_fence_after();
            const uint64_t db = v_desc + (uint64_t)(vt.st * (PT_TILE >> 4));
            if (lead) {
              const uint32_t began = j > a + (two ? 0 : s) ? 1u : 0u;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                ca_mma_ts(256 + s * 128, s * 128 + 8 * k, db + (uint64_t)((k * 2048) >> 4), IDESC_O,
                          k > 0 ? 1u : began);
            }
            ok = wait_all(ready2 + 8 * s, ph, abort_flag, p.err);
            if (!ok) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
              for (int k = 4; k < 8; ++k)
                ca_mma_ts(256 + s * 128, s * 128 + 32 + 8 * k, db + (uint64_t)((k * 2048) >> 4),
                          IDESC_O, 1u);
              if (s == s1) tc_commit(empty0 + 8 * vt.st);
            }
            if (!two && jn < b) {
              ok = wait_all(full0 + 8 * kt.st, kt.ph, abort_flag, p.err);
              if (!ok) break;
              tc_fence_after();
            }
            if (lead) {
              if (jn < b && (!two || s == 1 || jn < n0)) scores(s, s == s1, jn == b - 1);
              else tc_commit(ofull + 8 * s);  // the slot's last product
            }
            __syncwarp();
          }
          if (jn < b) kt.move(ca_next_k(two, jn - a, n));
          vt.move(ca_next_v(two, j - a, n));
        }
        qph ^= 1u;
      }
      if (ctl.abort_flag && lead) {  // gave up: wait for what was issued
        tc_commit(drain);
        mbar_wait(drain, 0, abort_flag, p.err, TC_DRAIN_LIMIT, false);
      }
      __syncwarp();
    } else if (warp == 21) {
      // ------------------------------------------------------------------ K tiles
      CaItems items;
      CaItem it;
      PagePieces pieces;
      const bool lead = elect_one();
      CaPlace kt;
      int left = p.k_tiles < 0 ? 0x7fffffff : p.k_tiles;
      bool ok = true;
      while (ok && items.next(ctl, it, p.err)) {
        pieces.start(p.pages, it.seq, it.L, it.a, lane);
        for (int j = it.a; j < it.b; ++j) {
          const int page = pieces.take(p.pages);
          ok = wait_all(empty0 + 8 * kt.st, kt.ph ^ 1u, abort_flag, p.err) && --left >= 0;
          if (!ok) break;
          load_tile(p.pages, &k_map, ring + kt.st * PT_TILE, full0 + 8 * kt.st, page, pieces.slot,
                    it.h, lead);
          ctl.last[kt.st] = 2 + (int)kt.ph;
          pieces.step(p.pages);
          kt.move(ca_next_k(it.two(), j - it.a, it.b - it.a));
        }
      }
    } else if (warp == 22) {
      // ------------------------------------------------------------------ V tiles
      CaItems items;
      CaItem it;
      PagePieces pieces;
      const bool lead = elect_one();
      CaPlace vt;
      uint32_t vph = 0;
      bool ok = true;
      while (ok && items.next(ctl, it, p.err)) {
        pieces.start(p.pages, it.seq, it.L, it.a, lane);
        vt.move(ca_first_v(it.two(), it.b - it.a));
        for (int j = it.a; j < it.b; ++j) {
          const int page = pieces.take(p.pages);
          ok = wait_all(empty0 + 8 * vt.st, vt.ph ^ 1u, abort_flag, p.err);
          if (!ok) break;
          const int nrow = it.L - j * CA_KT;  // the tile's rows that hold tokens
          const bool tail = nrow < CA_KT;
          const uint32_t dst = ring + vt.st * PT_TILE;
          load_tile(p.pages, &v_map, dst, tail ? vraw : full0 + 8 * vt.st, page, pieces.slot, it.h, lead);
          pieces.step(p.pages);
          if (tail) {
            // (its own copies: waited for even after another role gave up)
            bool in = true;
            if (lane == 0) in = mbar_wait(vraw, vph, abort_flag, p.err, TC_SPIN_LIMIT, false);
            ok = __shfl_sync(0xffffffffu, in, 0);
            __syncwarp();  // (the copies are in for every lane)
            vph ^= 1u;
            if (!ok) break;
            for (int i = nrow * 8 + lane; i < CA_KT * 8; i += 32)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + h * PT_HALF +
                                                                              i * 16),
                             "r"(0)
                             : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full0 + 8 * vt.st);
          }
          ctl.last[vt.st] = 2 + (int)vt.ph;
          vt.move(ca_next_v(it.two(), j - it.a, it.b - it.a));
        }
      }
    } else {
      // -------------------------------------- the items, ahead, and their Q tiles
      if (lane == 0) {
        CaWalk w(p, blockIdx.x);
        bool more = w.next(true);
        int from = w.a;  // the next part's first step
        for (int at = 0;; ++at) {
          const int i = at % CA_ITEMS;
          if (!wait_bar(smem_u32(&ctl.iempty[i]), (uint32_t)((at / CA_ITEMS) & 1) ^ 1u, abort_flag,
                        p.err))
            break;
          CaItem &it = ctl.item[i];
          it.a = it.b = 0;
          int to = 0;
          if (more) {
            to = w.b - from <= CA_PART + 1 ? w.b : from + CA_PART;
            it.a = from;
            it.b = to;
            it.part = (from > w.a ? 1 : 0) | (to < w.b ? 2 : 0);
            it.rec = w.a == 0 ? 1 : 0;
            it.n0 = w.w == 2 ? (w.lim0 + p.TT - 1 + CA_KT - 1) / CA_KT : -1;
            it.ntok = w.gi.z;
            it.h = w.h;
            it.row0 = w.gi.y;
            it.lim0 = w.lim0;
            it.whole = w.a == 0 && to == w.gi.w;
            it.seq = w.gi.x;
            it.L = w.L;
          }
          mbar_arrive(smem_u32(&ctl.ifull[i]));
          if (!more) break;
          // the item's query tiles, once the one before it has used its own
          // (its K and V tiles are on their way already)
          if (at > 0 && !wait_bar(qempty, (uint32_t)(at - 1) & 1u, abort_flag, p.err)) break;
          const int tiles = w.w == 2 ? 2 : 1;
          if (w.gi.z <= CA_FEW) {  // one by one: the tile's other rows stay zero
            mbar_arrive_expect(qfull, (uint32_t)(w.gi.z * p.G * 256));
            for (int i = 0; i < w.gi.z; ++i)
              for (int h = 0; h < 2; ++h)
                tma_load_3d(q_s + h * PT_HALF + i * p.G * 128, &q1_map, qfull, h * 64, w.h * p.G,
                            w.gi.y + i);
          } else {
            mbar_arrive_expect(qfull, (uint32_t)(tiles * 2 * p.TT * p.G * 128));
            for (int s = 0; s < tiles; ++s)
              for (int h = 0; h < 2; ++h)
                tma_load_3d(q_s + s * PT_TILE + h * PT_HALF, &q_map, qfull, h * 64, w.h * p.G,
                            w.gi.y + s * p.TT);
          }
          ctl.qissued = at + 1;
          from = to;
          if (to == w.b) {
            more = w.next(false);
            from = w.a;
          }
        }
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (ctl.abort_flag && threadIdx.x == 0) {
    // copies that were issued: each stage's last one, and the last query tiles
    for (int i = 0; i < CA_STAGES; ++i)
      if (ctl.last[i])
        mbar_wait(full0 + 8 * i, (uint32_t)ctl.last[i] & 1u, abort_flag, p.err, TC_DRAIN_LIMIT,
                  false);
    if (ctl.qissued > 0)
      mbar_wait(qfull, (uint32_t)((ctl.qissued - 1) & 1), abort_flag, p.err, TC_DRAIN_LIMIT, false);
  }
  __syncthreads();
  if (warp == 20) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// ------------------------------------------------------------------ join

// One block per CTA of the attend kernel: the item that started there and went
// on in the next ones, one warp per row.
__global__ void __launch_bounds__(256) ca_join_kernel(const CaArgs p) {
  pdl_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 e = p.shared[c0];
  if (e.x < 0) return;
  const int4 gi = p.ginfo[2 * e.x];
  const int h = e.y, c1 = e.z;
  const int rows = gi.z * p.G, per_tile = p.TT * p.G;
  for (int i = blockIdx.y * 8 + (threadIdx.x >> 5); i < rows; i += 8 * gridDim.y) {
    const int at = i < per_tile ? i : 128 + i - per_tile;
    auto rec = [&](int c) { return ((size_t)c * 2 + (c == c0 ? 1 : 0)) * 256 + at; };
    auto part = [&](int c) { return c <= c1 ? __ldcg(p.rec_lse + rec(c)) : -INFINITY; };
    const float mine = part(c0 + lane);  // a lane's part of the first 32
    float M = mine;
    for (int c = c0 + 32 + lane; c <= c1; c += 32) M = fmaxf(M, part(c));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b0 = c0; b0 <= c1; b0 += 32) {
      // (fmaxf passed over a part whose LSE is NaN; its factor is NaN)
      const float e = b0 == c0 ? mine : part(b0 + lane);
      const float fl = e == -INFINITY ? 0.f : __expf(e - M);
      for (int c = b0; c <= min(c1, b0 + 31); c += 4) {
        float f[4];
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          f[u] = __shfl_sync(0xffffffffu, fl, c - b0 + u);  // (0 past the last part)
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (f[u] != 0.f)
            v[u] = __ldcg(reinterpret_cast<const float4 *>(p.rec_o + rec(c + u) * CA_D) + lane);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          sum += f[u];
          acc.x = fmaf(f[u], v[u].x, acc.x);
          acc.y = fmaf(f[u], v[u].y, acc.y);
          acc.z = fmaf(f[u], v[u].z, acc.z);
          acc.w = fmaf(f[u], v[u].w, acc.w);
        }
      }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const size_t row = (size_t)(gi.y + i / p.G) * p.Hq + (size_t)h * p.G + i % p.G;
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    if (p.out_bf16)
      reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + row * CA_D)[lane] =
          make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    else
      reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * CA_D)[lane] = acc;
    if (lane == 0 && p.lse != nullptr) p.lse[row] = sum != 0.f ? M + logf(sum) : -INFINITY;
  }
}

// ------------------------------------------------------------------ host

struct CaLayout {
  size_t first, shared, gpre, ginfo, lse, o, part, bytes;
  int Gmax, TT, ctas;
};

CaLayout ca_layout(const qsa_dims &d, int S, int Nq) {
  CaLayout l;
  l.TT = 128 / (d.Hq / d.Hkv);
  l.Gmax = S + Nq / (2 * l.TT);
  l.ctas = device_sm_count();
  auto r = [](size_t x) { return (x + 255) / 256 * 256; };
  l.first = 256;
  l.shared = l.first + r(16 * (size_t)l.ctas);
  l.gpre = l.shared + r(16 * (size_t)l.ctas);
  l.ginfo = l.gpre + r(8 * ((size_t)l.Gmax + 1));
  l.lse = l.ginfo + r(32 * (size_t)l.Gmax);
  l.o = l.lse + r((size_t)l.ctas * 512 * 4);
  l.part = l.o + (size_t)l.ctas * 512 * CA_D * 4;
  l.bytes = l.part + (size_t)l.ctas * 512 * 8;
  return l;
}

}  // namespace

int debug_stall_dense() {
  const char *e = getenv("QSA_DEBUG_STALL_DENSE");
  return e != nullptr ? atoi(e) : -1;
}

size_t chunk_attention_ws_bytes(const qsa_dims &d, int S, int Nq) {
  return ca_layout(d, S, Nq).bytes;
}

cudaError_t launch_chunk_attention(const qsa_dims &d, const qsa_cache &c, int S,
                                   const int32_t *seq_lens, const int32_t *row_start, int Nq,
                                   const void *q, void *out, int out_is_bf16, float *lse,
                                   void *ws, unsigned *err, cudaStream_t st) {
  cudaError_t e;
  EncodeTiledFn enc = encode_tiled_fn(&e);
  if (e != cudaSuccess) return e;
  if (enc == nullptr) return cudaErrorNotSupported;
  const CaLayout l = ca_layout(d, S, Nq);
  char *w = static_cast<char *>(ws);
  CaArgs a;
  a.seq_lens = seq_lens;
  a.row_start = row_start;
  a.hdr = reinterpret_cast<int *>(w);
  a.first = reinterpret_cast<int4 *>(w + l.first);
  a.shared = reinterpret_cast<int4 *>(w + l.shared);
  a.gpre = reinterpret_cast<long long *>(w + l.gpre);
  a.ginfo = reinterpret_cast<int4 *>(w + l.ginfo);
  a.rec_lse = reinterpret_cast<float *>(w + l.lse);
  a.rec_o = reinterpret_cast<float *>(w + l.o);
  a.part = reinterpret_cast<float2 *>(w + l.part);
  a.out = out;
  a.lse = lse;
  a.S = S;
  a.Nq = Nq;
  a.Gmax = l.Gmax;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.G = d.Hq / d.Hkv;
  a.TT = l.TT;
  a.pages = paged_tiles(d, c, err);
  a.out_bf16 = out_is_bf16;
  a.scale = d.scale;
  a.k_tiles = debug_stall_dense();
  a.err = err;

  CUtensorMap q_map, q1_map, k_map, v_map;
  if (!query_map(enc, &q_map, q, d, Nq, a.TT) || !query_map(enc, &q1_map, q, d, Nq, 1) ||
      !pool_map(enc, &k_map, c.k_pool, d, c, a.pages.box) ||
      !pool_map(enc, &v_map, c.v_pool, d, c, a.pages.box))
    return cudaErrorInvalidValue;
  e = launch_pdl(ca_plan_kernel, 1, CA_PLAN_THREADS, 0, st, a, l.ctas);
  if (e != cudaSuccess) return e;
  e = ensure_dynamic_smem(reinterpret_cast<const void *>(ca_attend_kernel), CA_SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(ca_attend_kernel, l.ctas, CA_THREADS, CA_SMEM, st, q_map, q1_map, k_map,
                 v_map, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(ca_join_kernel, dim3(l.ctas, 12), 256, 0, st, a);
}

}  // namespace qsa
