// qsa_qk_norm_rope: RMS norm of every query and key head, then the position
// rotation, in one pass.
//
//   y = x * (sum x^2 / D + eps)^(-1/2) * w        (per head; no weights: y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)  for the rot / 2 pairs
//   (a, b) = (i, i + rot/2), or (2i, 2i + 1) when interleaved
// Norm, weight and rotation stay in fp32 registers; the result is rounded to
// bf16 once, when it is stored.
//
// The work is memory: every head row is read and written once (4 bytes a
// value), next to it a token's rot table entries. D / 16 lanes hold a head,
// two 16-byte vectors each, chosen so that both members of every rotated pair
// are in one lane: the norm costs log2(D / 16) shuffles and the rotation none.
// A pass of a warp so holds 512 / D heads.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace qsa {
namespace {

struct NormRopeArgs {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  const float *q_w, *k_w, *rope;
  const int32_t *pos;
  int64_t q_stride, k_stride;  // elements between tokens
  long long tasks;
  float eps;
  int N, Hq, Hk, rot, max_pos;
  int qp, groups;  // passes over the query heads; task groups per token
  unsigned *err;
};

__device__ __forceinline__ void unpack8(uint4 v, float *f) {
  f[0] = bf16lo(v.x); f[1] = bf16hi(v.x); f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
  f[4] = bf16lo(v.z); f[5] = bf16hi(v.z); f[6] = bf16lo(v.w); f[7] = bf16hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float *f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float *p, float *f) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// A warp's tasks are PPT passes of one token each, grid-stride; the next
// task's rows and position are requested before this one's are used, so that
// a task waits only for its table entries. 3 passes with 2 blocks per SM keep
// the most bytes in flight that the registers allow: 16,381 tokens of 32 + 4
// heads take 57 us (5.4 TB/s), 64 with 2 passes, 69 with 3 blocks, 76 with one
// task per warp and no next one.
constexpr int NR_PPT = 3, NR_BLOCKS = 2;
template <int D, bool INTER, int PPT>
__global__ void __launch_bounds__(256, NR_BLOCKS) norm_rope_kernel(NormRopeArgs a) {
  constexpr int LPH = D / 16;   // lanes per head
  constexpr int HPP = 32 / LPH;  // heads per pass
  const int lane = threadIdx.x & 31;
  const int l = lane % LPH, hl = lane / LPH;
  const int h2 = a.rot / 16;  // lanes of a head that hold rotated pairs
  const bool rotated = l < h2;
  // this lane's two 8-element vectors of its head
  const int ca = !INTER && rotated ? l : 2 * l, cb = !INTER && rotated ? l + h2 : 2 * l + 1;
  const long long stride = (long long)gridDim.x * 8;
  long long task = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  if (task >= a.tasks) return;

  uint4 va[PPT], vb[PPT];
  int pos, tok, p0;
  auto fetch = [&](long long t) {
    tok = (int)(t / a.groups);
    p0 = (int)(t - (long long)tok * a.groups) * PPT;
    pos = a.pos[tok];
#pragma unroll
    for (int u = 0; u < PPT; ++u) {
      const int p = p0 + u;
      const bool is_q = p < a.qp;
      const int h = (is_q ? p : p - a.qp) * HPP + hl;
      va[u] = vb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h < (is_q ? a.Hq : a.Hk)) {
        const __nv_bfloat16 *x = (is_q ? a.q + (size_t)tok * a.q_stride
                                       : a.k + (size_t)tok * a.k_stride) + (size_t)h * D;
        va[u] = *reinterpret_cast<const uint4 *>(x + ca * 8);
        vb[u] = *reinterpret_cast<const uint4 *>(x + cb * 8);
      }
    }
  };
  fetch(task);
  for (;;) {
    uint4 xa[PPT], xb[PPT];
#pragma unroll
    for (int u = 0; u < PPT; ++u) {
      xa[u] = va[u];
      xb[u] = vb[u];
    }
    const int cpos = pos, ctok = tok, cp0 = p0;
    // (pos < 0: padding, nothing is written)
    const bool skip = cpos < 0 || (a.rot > 0 && cpos >= a.max_pos);
    if (skip && cpos >= 0 && lane == 0) raise_err(a.err, ERR_POS);
    float cs[8], sn[8];
    if (rotated && !skip) {
      const float *t = a.rope + (size_t)cpos * a.rot + 8 * l;
      load8(t, cs);
      load8(t + a.rot / 2, sn);
    }
    task += stride;
    const bool more = task < a.tasks;
    if (more) fetch(task);
    else pdl_trigger();
#pragma unroll
    for (int u = 0; u < PPT; ++u) {
      const int p = cp0 + u;
      const bool is_q = p < a.qp;
      const int h = (is_q ? p : p - a.qp) * HPP + hl;
      float x[16];
      unpack8(xa[u], x);
      unpack8(xb[u], x + 8);
      const float *w = is_q ? a.q_w : a.k_w;
      if (w != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + a.eps);
        float wv[16];
        load8(w + ca * 8, wv);
        load8(w + cb * 8, wv + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * inv * wv[i];
      }
      if (rotated) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float &f = INTER ? x[2 * i] : x[i], &g = INTER ? x[2 * i + 1] : x[i + 8];
          const float f0 = f, g0 = g;
          f = f0 * cs[i] - g0 * sn[i];
          g = g0 * cs[i] + f0 * sn[i];
        }
      }
      if (!skip && h < (is_q ? a.Hq : a.Hk)) {
        __nv_bfloat16 *y = (is_q ? a.q_out + (size_t)ctok * a.Hq * D
                                 : a.k_out + (size_t)ctok * a.Hk * D) + (size_t)h * D;
        *reinterpret_cast<uint4 *>(y + ca * 8) = pack8(x);
        *reinterpret_cast<uint4 *>(y + cb * 8) = pack8(x + 8);
      }
    }
    if (!more) break;
  }
}

template <int D, bool INTER, int PPT>
cudaError_t launch_nr(NormRopeArgs a, int passes, cudaStream_t st) {
  a.groups = (passes + PPT - 1) / PPT;
  a.tasks = (long long)a.N * a.groups;
  long long blocks = (a.tasks + 7) / 8;
  if (PPT > 1) blocks = std::min<long long>(blocks, (long long)NR_BLOCKS * device_sm_count());
  return launch_pdl(norm_rope_kernel<D, INTER, PPT>, (unsigned)blocks, 256, 0, st, a);
}

template <int D, bool INTER>
cudaError_t launch_nr_p(NormRopeArgs a, cudaStream_t st) {
  constexpr int HPP = 512 / D;
  a.qp = (a.Hq + HPP - 1) / HPP;
  const int passes = a.qp + (a.Hk + HPP - 1) / HPP;
  // few tokens: one pass per warp and task, for the most warps (up to about a
  // warp's worth of passes per scheduler both take the time of a launch)
  if ((long long)a.N * passes <= 8 * device_sm_count()) return launch_nr<D, INTER, 1>(a, passes, st);
  return launch_nr<D, INTER, NR_PPT>(a, passes, st);
}

}  // namespace

cudaError_t launch_norm_rope(int N, int Hq, int Hk, int D, const int32_t *pos, const void *q,
                             int64_t q_stride, const void *k, int64_t k_stride, const float *q_w,
                             const float *k_w, float eps, const float *rope, int max_pos, int rot,
                             int interleaved, void *q_out, void *k_out, unsigned *err,
                             cudaStream_t st) {
  NormRopeArgs a;
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k);
  a.q_out = static_cast<__nv_bfloat16 *>(q_out);
  a.k_out = static_cast<__nv_bfloat16 *>(k_out);
  a.q_w = q_w;
  a.k_w = k_w;
  a.rope = rope;
  a.pos = pos;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.eps = eps;
  a.N = N;
  a.Hq = Hq;
  a.Hk = Hk;
  a.rot = rot;
  a.max_pos = max_pos;
  a.err = err;
  if (D == 128)
    return interleaved ? launch_nr_p<128, true>(a, st) : launch_nr_p<128, false>(a, st);
  return interleaved ? launch_nr_p<64, true>(a, st) : launch_nr_p<64, false>(a, st);
}

}  // namespace qsa
