// Absorbed latent attention over the paged cache, simple form: one warp a
// query row, online softmax over groups of 32 cached rows (lane = cached row
// for the scores, lane = 16 output values for the products).
#include "../../include/kda_latent.h"
#include "kda_common.cuh"
#include "kda_latent.cuh"

namespace kda {

__global__ void __launch_bounds__(128) kda_latent_decode_kernel(const DecodeParams p) {
  __shared__ float qs[4][kLatRow];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = p.R * p.H;
  const int64_t item = (int64_t)blockIdx.x * 4 + warp;
  if (item >= (int64_t)p.B * rows) return;
  const int b = (int)(item / rows), i = (int)(item % rows) / p.H;
  int64_t len = p.lens[b];
  const int64_t cap = p.max_pages * p.page_size;
  if (len < 0 || len > cap) {
    if (lane == 0) atomicExch(p.status, KDA_ERR_BAD_LENGTHS);
    len = len < 0 ? 0 : cap;
  }
  const int64_t seen = len - (p.R - 1 - i);
  for (int d = lane; d < kLatRow; d += 32) qs[warp][d] = bf16_to_f(p.q[item * kLatRow + d]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int d = 0; d < 16; ++d) acc[d] = 0.f;
  for (int64_t j0 = 0; j0 < seen; j0 += 32) {
    const int64_t j = j0 + lane;
    const uint16_t* row = nullptr;
    float s = -INFINITY;
    if (j < seen) {
      const int64_t page = p.table[b * p.table_stride + j / p.page_size];
      s = 0.f;
      if (page < 0 || page >= p.num_pages) {
        atomicExch(p.status, KDA_ERR_BAD_PAGE);
      } else {
        row = p.cache + page * p.page_stride + (j % p.page_size) * p.token_stride;
        for (int d = 0; d < kLatRow; d += 2) {
          const float2 x = unpack_bf16(*reinterpret_cast<const uint32_t*>(row + d));
          s += x.x * qs[warp][d] + x.y * qs[warp][d + 1];
        }
      }
      s *= p.scale_log2;
    }
    float mt = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    const float mn = fmaxf(m, mt), f = ex2(m - mn);
    const float e = ex2(s - mn);
    m = mn;
    l = l * f + e;
#pragma unroll
    for (int d = 0; d < 16; ++d) acc[d] *= f;
    const int cnt = (int)min((int64_t)32, seen - j0);
    for (int jj = 0; jj < cnt; ++jj) {
      const float w = __shfl_sync(0xffffffffu, e, jj);
      const uint64_t r = __shfl_sync(0xffffffffu, (unsigned long long)row, jj);
      if (!r) continue;
      const uint32_t* v = reinterpret_cast<const uint32_t*>(r) + lane;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const float2 x = unpack_bf16(v[32 * d]);
        acc[2 * d] += w * x.x;
        acc[2 * d + 1] += w * x.y;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + item * kLat) + lane;
#pragma unroll
  for (int d = 0; d < 8; ++d) out[32 * d] = pack_bf16(acc[2 * d] * inv, acc[2 * d + 1] * inv);
  if (lane == 0 && p.lse) p.lse[item] = seen > 0 ? m / kLog2e + logf(l) : -INFINITY;
}

size_t decode_workspace_bytes(const DecodeParams&) { return 0; }

bool launch_latent_decode(const DecodeParams& p, cudaStream_t s) {
  const int64_t items = (int64_t)p.B * p.R * p.H;
  kda_latent_decode_kernel<<<(unsigned)((items + 3) / 4), 128, 0, s>>>(p);
  return true;
}

}  // namespace kda
