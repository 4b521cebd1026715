// Expanded latent attention of few queries and many keys: items shared out by key
// tiles, and their parts joined.  (A file of its own, so that it is compiled beside
// the unsplit form.)
#include "kda_latent_prefill.cuh"

namespace kda {

// Adds up the parts of the items that several shares hold: o = sum_k w_k o_k,
// w_k = 2^(lse_k - lse), in the shares' order.  A warp a row, 16 rows a CTA; bound by
// the partial rows' bytes (in L2 mostly).
template <bool kPair>
__global__ void __launch_bounds__(512) kda_latent_prefill_join_kernel(const PrefillParams p, int64_t per,
                                                                      const PrefillSplit sp) {
  constexpr int kRows = (kPair ? 4 : 2) * kPreRows;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  __shared__ PreItem shared_it;
  __shared__ int64_t shared_at[2];
  if (threadIdx.x == 0) {  // (divisions of 64 bits: once a CTA)
    PreItem it;
    int64_t first = 0;  // where the item's first key tile lies
    it.n0 = it.n1 = 0;
    if (p.items) {
      const uint32_t e = blockIdx.x / (uint32_t)p.H, h = blockIdx.x - e * (uint32_t)p.H;
      if (e < (uint32_t)*p.count) {
        PreWalk<kPair>::listed(p, e, it);
        it.h = (int)h;
        first = (int64_t)p.items[e].start * p.H + (int64_t)h * (it.nt() + kPreItemCost) + kPreItemCost;
      }
    } else {
      const uint32_t bh = (uint32_t)(p.B * p.H), back = blockIdx.x / bh, x = blockIdx.x - back * bh;
      for (uint32_t b = 0; b < back; ++b) {
        PreWalk<kPair>::dense(p, per, b, 0, it);
        first += (int64_t)bh * (it.nt() + kPreItemCost);
      }
      PreWalk<kPair>::dense(p, per, back, x, it);
      first += (int64_t)x * (it.nt() + kPreItemCost) + kPreItemCost;
    }
    const int64_t size = split_size(p, sp);
    shared_it = it;
    shared_at[0] = first / size;
    shared_at[1] = (first + it.nt() - 1) / size;
  }
  __syncthreads();
  const PreItem it = shared_it;
  const int nt = it.nt();
  const int64_t s0 = shared_at[0], s1 = shared_at[1];
  const int local = blockIdx.y * 16 + (threadIdx.x >> 5), row = it.r0 + local, lane = threadIdx.x & 31;
  if (nt == 0 || s0 == s1 || row >= it.lq) return;
  const int parts = (int)(s1 - s0) + 1;
  auto slot = [&](int k) { return (2 * (s0 + k) + (k == 0 ? 1 : 0)) * kRows + local; };
  float top = -INFINITY;
  for (int k = lane; k < parts; k += 32) top = fmaxf(top, sp.part_lse[slot(k)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.f : top;
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const int64_t from = slot(k);
    const float w = ex2(sp.part_lse[from] - base);
    const float4 x = reinterpret_cast<const float4*>(sp.part + from * kVDim)[lane];
    sum += w;
    if (w != 0.f) {
      acc[0] += w * x.x;
      acc[1] += w * x.y;
      acc[2] += w * x.z;
      acc[3] += w * x.w;
    }
  }
  const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
  const int64_t at = ((int64_t)it.q0 + row) * p.H + it.h;
  reinterpret_cast<uint2*>(p.out + at * kVDim)[lane] =
      make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
  if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
}

namespace {

template <bool kPair>
bool launch_both(const PrefillParams& p, const PrefillSplit& sp, int sms, cudaStream_t s) {
  if (!launch_prefill<kPair, true>(p, sp, sms, s)) return false;
  const int rows = kPair ? 2 * kPrefillRows : kPrefillRows;
  const int64_t per = (p.Tq + rows - 1) / rows, items = (p.items ? p.Tq / rows + p.N : p.B * per) * p.H;
  return launch_overlapped(kda_latent_prefill_join_kernel<kPair>, dim3((unsigned)items, (unsigned)(rows / 16)), 512, 0, s, 1,
                           p, per, sp);
}

}  // namespace

bool launch_prefill_split(const PrefillParams& p, const PrefillSplit& sp, int sms, cudaStream_t s) {
  return p.pairs ? launch_both<true>(p, sp, sms, s) : launch_both<false>(p, sp, sms, s);
}

}  // namespace kda
