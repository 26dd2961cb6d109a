// qsa_chunk_attention: dense causal attention of the rows of appended chunks
// over the paged cache.
//
//   z_t = scale q.K_t for the row's len = L - T + i + 1 first tokens,
//   LSE = ln sum e^(z_t), out = sum e^(z_t - LSE) V_t
// One warp per (row, query head): 4 dims a lane, one token at a time, with
// the running maximum and sum of the softmax in registers.
#include "common.cuh"
#include "launch.h"

namespace qsa {
namespace {

struct ChunkArgs {
  const __nv_bfloat16 *k_pool, *v_pool, *q;
  const int32_t *block_table, *seq_lens, *row_start;
  void *out;
  float *lse;
  int S, Nq, Hq, Hkv, P, max_pages, num_pages, out_bf16;
  float scale;
  unsigned *err;
};

__global__ void __launch_bounds__(256) chunk_attention_kernel(ChunkArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  const int r = (int)(w / a.Hq), h = (int)(w % a.Hq);
  if (r >= a.Nq) return;
  int lo = 0, hi = a.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.row_start[mid] <= r) lo = mid; else hi = mid - 1;
  }
  const int r0 = a.row_start[lo], r1 = a.row_start[lo + 1], L = a.seq_lens[lo];
  if (r < r0 || r >= r1) return;
  if (r0 < 0 || r1 > a.Nq || r1 - r0 > L || (long long)L > (long long)a.max_pages * a.P) {
    if (lane == 0) raise_err(a.err, ERR_LEN);
    return;
  }
  const int len = L - (r1 - r0) + (r - r0) + 1;
  const size_t row = (size_t)r * a.Hq + h;
  const uint2 qv = *reinterpret_cast<const uint2 *>(a.q + row * 128 + lane * 4);
  const float q0 = bf16lo(qv.x), q1 = bf16hi(qv.x), q2 = bf16lo(qv.y), q3 = bf16hi(qv.y);
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
  for (int t = 0; t < len; ++t) {
    const int page = a.block_table[(size_t)lo * a.max_pages + t / a.P];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) raise_err(a.err, ERR_PAGE);
      continue;
    }
    const size_t at = (((size_t)page * a.P + t % a.P) * a.Hkv + h / (a.Hq / a.Hkv)) * 128 + lane * 4;
    const uint2 kv = *reinterpret_cast<const uint2 *>(a.k_pool + at);
    const uint2 vv = *reinterpret_cast<const uint2 *>(a.v_pool + at);
    float z = q0 * bf16lo(kv.x) + q1 * bf16hi(kv.x) + q2 * bf16lo(kv.y) + q3 * bf16hi(kv.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z *= a.scale;
    if (z > m) {
      const float f = __expf(m - z);
      l *= f; o0 *= f; o1 *= f; o2 *= f; o3 *= f;
      m = z;
    }
    const float p = __expf(z - m);
    l += p;
    o0 = fmaf(p, bf16lo(vv.x), o0); o1 = fmaf(p, bf16hi(vv.x), o1);
    o2 = fmaf(p, bf16lo(vv.y), o2); o3 = fmaf(p, bf16hi(vv.y), o3);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  o0 *= inv; o1 *= inv; o2 *= inv; o3 *= inv;
  if (a.out_bf16)
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * 128 + lane * 4) =
        make_uint2(pack_bf16x2(o0, o1), pack_bf16x2(o2, o3));
  else
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * 128 + lane * 4) =
        make_float4(o0, o1, o2, o3);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t chunk_attention_ws_bytes(const qsa_dims &d, int S, int Nq) {
  (void)d; (void)S; (void)Nq;
  return 0;
}

cudaError_t launch_chunk_attention(const qsa_dims &d, const qsa_cache &c, int S,
                                   const int32_t *seq_lens, const int32_t *row_start, int Nq,
                                   const void *q, void *out, int out_is_bf16, float *lse,
                                   void *ws, unsigned *err, cudaStream_t st) {
  (void)ws;
  ChunkArgs a;
  a.k_pool = static_cast<const __nv_bfloat16 *>(c.k_pool);
  a.v_pool = static_cast<const __nv_bfloat16 *>(c.v_pool);
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.block_table = c.block_table;
  a.seq_lens = seq_lens;
  a.row_start = row_start;
  a.out = out;
  a.lse = lse;
  a.S = S;
  a.Nq = Nq;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.P = d.P;
  a.max_pages = c.max_pages_per_seq;
  a.num_pages = c.num_pages;
  a.out_bf16 = out_is_bf16;
  a.scale = d.scale;
  a.err = err;
  const long long warps = (long long)Nq * d.Hq;
  return launch_pdl(chunk_attention_kernel, (unsigned)((warps + 7) / 8), 256, 0, st, a);
}

}  // namespace qsa
