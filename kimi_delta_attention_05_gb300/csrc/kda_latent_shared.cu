// Decoding behind shared prefixes: the launches, and the join of the parts that the
// shared pass (kda_latent_prefix.cu) and the requests' own pass (kda_latent_decode.cu)
// leave.
//
// Only whole tiles of a prefix are shared (128 tokens), and only by requests all of
// whose new tokens see them; the rest of the prefix, up to 127 tokens, belongs to the
// requests' own passes, as do requests that see less and groups of one.  So the
// shared pass has no masks and the own pass has those of kda_latent_decode.  The own
// pass starts on SMs that the shared pass leaves, or has no use for.
#include <algorithm>

#include "../../include/kda_latent.h"
#include "kda_common.cuh"
#include "kda_latent.cuh"

namespace kda {

// What the own pass has not finished: out = sum_k w_k o_k, w_k = 2^(lse_k - lse), over
// a row's parts: the prefix's in the order of its shares, then the request's own.  A
// warp a row, 16 dimensions a lane; a CTA looks through `chunk` blocks of N rows.
__global__ void __launch_bounds__(256) kda_latent_shared_join_kernel(const SharedParams p, const int chunk) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const DecodeParams& d = p.d;
  const int lane = threadIdx.x & 31, rows = d.R * d.H, blocks = d.B * p.own_row_blocks;
  const int64_t all = (int64_t)d.B * rows, cap = d.max_pages * d.page_size;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);  // row of a block of N
  const int first = blockIdx.x * chunk;
  int4 info = make_int4(-1, 0, 0, 0);
  if (lane < chunk && first + lane < blocks) info = p.split[first + lane];
  uint32_t left = __ballot_sync(0xffffffffu, info.x >= 0);
  while (left) {
    const int from = __ffs(left) - 1;
    left &= left - 1;
    const int req = __shfl_sync(0xffffffffu, info.x, from), own_first = __shfl_sync(0xffffffffu, info.y, from);
    const int own_last = __shfl_sync(0xffffffffu, info.z, from), group = __shfl_sync(0xffffffffu, info.w, from);
    const int own_block = (first + from) % p.own_row_blocks, row = own_block * p.own_n + r;
    if (r >= p.own_n || row >= rows) continue;  // (the whole warp)
    const int64_t at = (int64_t)req * rows + row;
    int pre = 0;
    int64_t second = 0;
    if (group >= 0) {
      const int64_t c = p.groups.cu[group];
      const int tokens = shared_tokens(c, p.groups.cu[group + 1], p.groups.prefix[group], cap);
      pre = prefix_parts(p.line[group], p.head->size, tokens, (int)(at - c * rows), all, second);
    }
    const int parts = pre + own_last - own_first + 1;
    // the place of part k: a row's first at its own, the others with their shares
    auto place = [&](int k) {
      if (k < pre) return k == 0 ? at : second + (int64_t)(k - 1) * kPfxRows;
      k -= pre;
      return k == 0 ? at : all + ((int64_t)(own_first + k) * p.own_row_blocks + own_block) * p.own_n + r;
    };
    float top = -INFINITY;
    for (int k = lane; k < parts; k += 32) top = fmaxf(top, (k < pre ? p.pre_lse : p.own_lse)[place(k)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float acc[16], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const int64_t at_k = place(k);
      const float w = ex2((k < pre ? p.pre_lse : p.own_lse)[at_k] - base);
      const float4* src = reinterpret_cast<const float4*>((k < pre ? p.pre_part : p.own_part) + at_k * kLat) + lane;
      sum += w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = src[32 * i];
        if (w != 0.f) {
          acc[4 * i] += w * x.x;
          acc[4 * i + 1] += w * x.y;
          acc[4 * i + 2] += w * x.z;
          acc[4 * i + 3] += w * x.w;
        }
      }
    }
    const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
    uint2* dst = reinterpret_cast<uint2*>(d.out + at * kLat) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dst[32 * i] = make_uint2(pack_bf16(acc[4 * i] * inv, acc[4 * i + 1] * inv),
                               pack_bf16(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv));
    if (lane == 0 && d.lse) d.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
  }
}

namespace {

// Sizes and places of a call's workspace; returns its bytes.
size_t shared_layout(SharedParams& p) {
  const OwnLayout own = own_layout(p.d);
  const size_t rows = (size_t)p.d.B * p.d.R * p.d.H;
  p.own_n = own.n;
  p.own_row_blocks = own.row_blocks;
  // (tables shorter than a tile have nothing to share)
  p.pairs = p.d.num_pages > 0 && p.d.max_pages * p.d.page_size >= kPfxTile ? std::max(1, device_sm_count() / 2) : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* x = p.d.ws + at;
    at += (bytes + 255) / 256 * 256;
    return x;
  };
  p.head = reinterpret_cast<SharedHead*>(take(sizeof(SharedHead)));
  p.line = reinterpret_cast<int64_t*>(take((size_t)p.groups.G * 8));
  p.split = reinterpret_cast<int4*>(take((size_t)p.d.B * own.row_blocks * sizeof(int4)));
  const size_t pre_rows = p.pairs > 0 ? rows + (size_t)p.pairs * kPfxRows : 0, own_rows = rows + (size_t)own.ctas * own.n;
  p.pre_lse = reinterpret_cast<float*>(take(pre_rows * 4));
  p.own_lse = reinterpret_cast<float*>(take(own_rows * 4));
  p.pre_part = reinterpret_cast<float*>(take(pre_rows * kLat * 4));
  p.own_part = reinterpret_cast<float*>(take(own_rows * kLat * 4));
  return at;
}

}  // namespace

size_t shared_workspace_bytes(const DecodeParams& d, int64_t G) {
  SharedParams p = {};
  p.d = d;
  p.d.ws = nullptr;
  p.groups.G = (int)G;
  return shared_layout(p);
}

bool launch_latent_shared(const DecodeParams& d, const SharedGroups& groups, cudaStream_t s) {
  SharedParams p = {};
  p.d = d;
  p.groups = groups;
  shared_layout(p);
  if (d.num_pages == 0) p.d.max_pages = 0;  // no cache: every length is taken as 0
  if (p.pairs > 0 && !launch_latent_prefix(p, s)) return false;
  if (!launch_latent_own(p, s)) return false;
  const int64_t blocks = (int64_t)d.B * p.own_row_blocks;
  const int chunk = (int)std::min<int64_t>(32, (blocks + 1023) / 1024);
  const dim3 grid((unsigned)((blocks + chunk - 1) / chunk), (unsigned)((std::min(p.own_n, d.R * d.H) + 7) / 8));
  return launch_overlapped(kda_latent_shared_join_kernel, grid, 256, 0, s, 1, p, chunk);
}

}  // namespace kda
