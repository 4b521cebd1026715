// Expanded latent attention, simple form: a CTA per (block of 256 query rows,
// head), one warp a query row at a time, online softmax over groups of 32 keys.
#include "../../include/kda_latent.h"
#include "kda_common.cuh"
#include "kda_latent.cuh"

namespace kda {

__global__ void __launch_bounds__(256) kda_latent_prefill_kernel(const PrefillParams p, int64_t blocks_per_row) {
  __shared__ float qs[8][kQkDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  const int64_t blk = blockIdx.x;
  int64_t q0, k0, lq, lk, r0;
  if (p.cu_q) {
    if (blk >= p.blk_off[p.N]) return;
    int64_t lo = 0, hi = p.N - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) >> 1;
      if (p.blk_off[mid] <= blk) lo = mid; else hi = mid - 1;
    }
    q0 = p.cu_q[lo];
    lq = p.cu_q[lo + 1] - q0;
    k0 = p.cu_k[lo];
    lk = p.cu_k[lo + 1] - k0;
    r0 = (blk - p.blk_off[lo]) * kPrefillRows;
  } else {
    const int64_t n = blk / blocks_per_row;
    q0 = n * p.Tq;
    lq = p.Tq;
    k0 = n * p.Tk;
    lk = p.Tk;
    r0 = (blk - n * blocks_per_row) * kPrefillRows;
  }
  const int64_t r1 = min(lq, r0 + kPrefillRows);
  for (int64_t i = r0 + warp; i < r1; i += 8) {
    const uint16_t* q = p.q + (q0 + i) * p.q_st + h * p.q_sh;
    for (int d = lane; d < kQkDim; d += 32) qs[warp][d] = bf16_to_f(q[d]);
    __syncwarp();
    const int64_t seen = p.causal ? min(lk, i + lk - lq + 1) : lk;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t j0 = 0; j0 < seen; j0 += 32) {
      const int64_t j = j0 + lane;
      float s = -INFINITY;
      if (j < seen) {
        const uint32_t* k = reinterpret_cast<const uint32_t*>(p.k + (k0 + j) * p.k_st + h * p.k_sh);
        const uint32_t* pe = reinterpret_cast<const uint32_t*>(p.k_pe + (k0 + j) * p.pe_st);
        s = 0.f;
        for (int d = 0; d < kQkDim / 2; ++d) {
          const float2 x = unpack_bf16(d < kNope / 2 ? k[d] : pe[d - kNope / 2]);
          s += x.x * qs[warp][2 * d] + x.y * qs[warp][2 * d + 1];
        }
        s *= p.scale_log2;
      }
      float mt = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mn = fmaxf(m, mt), f = ex2(m - mn), e = ex2(s - mn);
      m = mn;
      l = l * f + e;
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[d] *= f;
      const int cnt = (int)min((int64_t)32, seen - j0);
      for (int jj = 0; jj < cnt; ++jj) {
        const float w = __shfl_sync(0xffffffffu, e, jj);
        const uint2 r = reinterpret_cast<const uint2*>(p.v + (k0 + j0 + jj) * p.v_st + h * p.v_sh)[lane];
        const float2 x = unpack_bf16(r.x), y = unpack_bf16(r.y);
        acc[0] += w * x.x;
        acc[1] += w * x.y;
        acc[2] += w * y.x;
        acc[3] += w * y.y;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    const int64_t row = (q0 + i) * p.H + h;
    reinterpret_cast<uint2*>(p.out + row * kVDim)[lane] =
        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    if (lane == 0 && p.lse) p.lse[row] = seen > 0 ? m / kLog2e + logf(l) : -INFINITY;
    __syncwarp();
  }
}

bool launch_latent_prefill(const PrefillParams& p, cudaStream_t s) {
  const int64_t per = (p.Tq + kPrefillRows - 1) / kPrefillRows;
  const int64_t blocks = p.cu_q ? p.Tq / kPrefillRows + p.N : p.B * per;
  kda_latent_prefill_kernel<<<dim3((unsigned)blocks, (unsigned)p.H), 256, 0, s>>>(p, per);
  return true;
}

}  // namespace kda
