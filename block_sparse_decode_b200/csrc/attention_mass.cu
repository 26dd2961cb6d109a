// qsa_attention_mass: the attention weight that the rows of appended chunks
// gave to each micro-block, summed over rows and heads.
//
//   mass[s, j] = mass_in[s, j] + sum_{t in block j} sum_{rows i of s that see t}
//                sum_h e^(scale q_ih.K_t - LSE_ih)
// One warp per (sequence, micro-block): 4 dims a lane, one (token, row, head)
// product at a time. The sum's order is fixed.
#include "common.cuh"
#include "launch.h"

namespace qsa {
namespace {

struct MassArgs {
  const __nv_bfloat16 *k_pool, *q;
  const int32_t *block_table, *seq_lens, *row_start;
  const float *lse, *mass_in;
  float *mass;
  int S, Nq, Hq, Hkv, P, max_pages, num_pages, ld;
  float scale;
  unsigned *err;
};

__global__ void __launch_bounds__(256) attention_mass_kernel(MassArgs a) {
  const int lane = threadIdx.x & 31, s = blockIdx.y;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  if (j >= a.ld) return;
  const int r0 = a.row_start[s], r1 = a.row_start[s + 1], L = a.seq_lens[s], T = r1 - r0;
  float sum = 0.f;
  if (r0 < 0 || T < 0 || r1 > a.Nq || T > L || (long long)L > (long long)a.max_pages * a.P ||
      (long long)L > 4LL * a.ld) {
    if (j == 0 && lane == 0) raise_err(a.err, ERR_LEN);
  } else {
    const int G = a.Hq / a.Hkv;
    for (int t = 4 * j; t < 4 * j + 4 && t < L; ++t) {
      const int page = a.block_table[(size_t)s * a.max_pages + t / a.P];
      if (page < 0 || page >= a.num_pages) {
        if (T > 0 && lane == 0) raise_err(a.err, ERR_PAGE);
        continue;
      }
      const int i0 = max(0, t - (L - T));
      for (int g = 0; g < a.Hkv; ++g) {
        const uint2 kv = *reinterpret_cast<const uint2 *>(
            a.k_pool + (((size_t)page * a.P + t % a.P) * a.Hkv + g) * 128 + lane * 4);
        const float k0 = bf16lo(kv.x), k1 = bf16hi(kv.x), k2 = bf16lo(kv.y), k3 = bf16hi(kv.y);
        for (int i = i0; i < T; ++i)
          for (int h = g * G; h < g * G + G; ++h) {
            const size_t row = (size_t)(r0 + i) * a.Hq + h;
            const uint2 qv = *reinterpret_cast<const uint2 *>(a.q + row * 128 + lane * 4);
            float z = k0 * bf16lo(qv.x) + k1 * bf16hi(qv.x) + k2 * bf16lo(qv.y) + k3 * bf16hi(qv.y);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            const float e = a.lse[row];
            if (e > -INFINITY) sum += __expf(z * a.scale - e);
          }
      }
    }
  }
  if (lane == 0) {
    const size_t at = (size_t)s * a.ld + j;
    a.mass[at] = (a.mass_in != nullptr ? a.mass_in[at] : 0.f) + sum;
  }
}

}  // namespace

size_t attention_mass_ws_bytes(const qsa_dims &d, int S, int Nq) {
  (void)d; (void)S; (void)Nq;
  return 0;
}

cudaError_t launch_attention_mass(const qsa_dims &d, const qsa_cache &c, int S,
                                  const int32_t *seq_lens, const int32_t *row_start, int Nq,
                                  const void *q, const float *lse, const float *mass_in,
                                  float *mass, int ld, void *ws, unsigned *err, cudaStream_t st) {
  (void)ws;
  MassArgs a;
  a.k_pool = static_cast<const __nv_bfloat16 *>(c.k_pool);
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.block_table = c.block_table;
  a.seq_lens = seq_lens;
  a.row_start = row_start;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass = mass;
  a.S = S;
  a.Nq = Nq;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.P = d.P;
  a.max_pages = c.max_pages_per_seq;
  a.num_pages = c.num_pages;
  a.ld = ld;
  a.scale = d.scale;
  a.err = err;
  return launch_pdl(attention_mass_kernel, dim3((ld + 7) / 8, S), 256, 0, st, a);
}

}  // namespace qsa
