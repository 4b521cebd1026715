// Decoding behind shared prefixes: the list of groups, and the join of the parts
// that the shared pass (kda_latent_prefix.cu) and the requests' own pass
// (kda_latent_decode.cu) leave.
//
// Only whole tiles of a prefix are shared (128 tokens), and only by requests all of
// whose new tokens see them; the rest of the prefix, up to 127 tokens, belongs to the
// requests' own passes, as do requests that see less and groups of one.  So the
// shared pass has no masks and the own pass has those of kda_latent_decode.
#include <algorithm>

#include "../../include/kda_latent.h"
#include "kda_common.cuh"
#include "kda_latent.cuh"

namespace kda {

constexpr int kGroupThreads = 1024;

// Sum over the threads before this one; `total` gets that over all.
__device__ __forceinline__ int64_t scan_block(int64_t x, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kGroupThreads / 32; ++w) {
    const int64_t s = sums[w];
    if (w < warp) before += s;
    total += s;
  }
  __syncthreads();  // sums are read
  return before + upto - x;
}

// The groups that share tiles, in order, and their items' place on the line of
// costs.  One CTA, `width` lanes a group (a power of two up to 32): latency of three
// or four dependent loads a round of 1024 / width groups.
__global__ void __launch_bounds__(kGroupThreads) kda_latent_groups_kernel(const SharedParams p, const int width) {
  __shared__ int64_t sums[kGroupThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const DecodeParams& d = p.d;
  const int tid = threadIdx.x;
  int bad = 0;
  for (int g = tid; g <= p.G; g += kGroupThreads) {
    const int64_t c = p.cu[g];
    bad |= (g == 0 && c != 0) || (g == p.G && c != d.B) || c < 0 || c > d.B || (g > 0 && c < p.cu[g - 1]);
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (tid == 0) atomicExch(d.status, KDA_ERR_BAD_SEQLENS);
    for (int b = tid; b < d.B; b += kGroupThreads) {
      p.start[b] = 0;
      p.of[b] = -1;
    }
  }
  const int64_t cap = d.max_pages * d.page_size;
  const int lane = tid & (width - 1), rows = d.R * d.H;
  int64_t active = 0, cost = 0;
  for (int g0 = 0; g0 < p.G && !bad; g0 += kGroupThreads / width) {
    const int g = g0 + tid / width;
    int first = 0, end = 0, tiles = 0;
    if (g < p.G) {
      first = (int)p.cu[g];
      end = (int)p.cu[g + 1];
      const int64_t len = p.prefix[g];
      if ((len < 0 || len > cap) && first < end && lane == 0) atomicExch(d.status, KDA_ERR_BAD_LENGTHS);
      tiles = (int)(min(max(len, (int64_t)0), cap) / kPfxTile);
    }
    // requests all of whose new tokens see the tiles: how many, and the first
    auto sees = [&](int b) { return min(max((int64_t)d.lens[b], (int64_t)0), cap) - (d.R - 1) >= (int64_t)tiles * kPfxTile; };
    int count = 0, source = d.B;
    if (tiles > 0)
      for (int b = first + lane; b < end; b += width)
        if (sees(b)) {
          ++count;
          source = min(source, b);
        }
    for (int o = width >> 1; o > 0; o >>= 1) {
      count += __shfl_xor_sync(0xffffffffu, count, o);
      source = min(source, __shfl_xor_sync(0xffffffffu, source, o));
    }
    if (count < 2) tiles = 0;
    const int group_rows = (end - first) * rows;
    const int64_t blocks = (group_rows + kPfxRows - 1) / kPfxRows;
    const bool leads = lane == 0 && tiles > 0;
    int64_t more, more_cost;
    // (the groups of a round, for all lanes of each)
    const int64_t k = __shfl_sync(0xffffffffu, active + scan_block(leads, sums, more), 0, width);
    const int64_t at =
        cost + scan_block(leads ? blocks * (kPfxItemCost + (int64_t)tiles * kPfxTileCost) : 0, sums, more_cost);
    if (leads) {
      p.groups[k] = {tiles, source, first * rows, group_rows};
      p.line[k] = at;
    }
    for (int b = first + lane; b < end; b += width) {
      const bool in = tiles > 0 && sees(b);
      p.start[b] = in ? tiles * kPfxTile : 0;
      p.of[b] = in ? (int)k : -1;
    }
    active += more;
    cost += more_cost;
  }
  // the shares, at least a tile each, and the item in which each begins
  const int64_t size = max((int64_t)kPfxTileCost, (cost + p.pairs - 1) / p.pairs);
  if (tid == 0) *p.head = {cost, size, (int32_t)active, 0};
  __syncthreads();
  for (int s = tid; s < p.pairs; s += kGroupThreads) {
    const int64_t u = s * size;
    if (u >= cost) continue;
    int lo = 0, hi = (int)active - 1;  // last group that begins at u or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.line[mid] <= u) lo = mid; else hi = mid - 1;
    }
    const int64_t item = kPfxItemCost + (int64_t)p.groups[lo].tiles * kPfxTileCost;
    p.first[s] = make_int2(lo, (int)((u - p.line[lo]) / item));
  }
}

// out = sum_k w_k o_k, w_k = 2^(lse_k - lse), over a row's parts: the prefix's in the
// order of its shares, then the request's own.  A warp a row, 16 dimensions a lane.
__global__ void __launch_bounds__(256) kda_latent_shared_join_kernel(const SharedParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const DecodeParams& d = p.d;
  const int lane = threadIdx.x & 31, rows = d.R * d.H;
  const int64_t all = (int64_t)d.B * rows, at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (at >= all) return;
  const int b = (int)((uint32_t)at / (uint32_t)rows), row = (int)(at - (int64_t)b * rows);
  const int of = p.of[b], own_block = row / p.own_n;
  const int4 own = p.split[b * p.own_row_blocks + own_block];
  int64_t pre_first = 0, pre_more = 0;  // first share, and the place of the second's part
  int pre = 0;
  if (of >= 0) {
    const SharedGroup g = p.groups[of];
    const int64_t size = p.head->size;
    const int in = (int)(at - g.row0), block = in / kPfxRows;
    const int64_t item = p.line[of] + block * (kPfxItemCost + (int64_t)g.tiles * kPfxTileCost);
    pre_first = prefix_share(item, 0, size);
    pre = (int)(prefix_share(item, g.tiles - 1, size) - pre_first) + 1;
    pre_more = all + (pre_first + 1) * kPfxRows + in % kPfxRows;
  }
  const int parts = pre + own.z - own.y + 1;
  // the place of part k: a row's first at its own, the others with their shares
  auto place = [&](int k) {
    if (k < pre) return k == 0 ? at : pre_more + (int64_t)(k - 1) * kPfxRows;
    k -= pre;
    return k == 0 ? at : all + ((int64_t)(own.y + k) * p.own_row_blocks + own_block) * p.own_n + row % p.own_n;
  };
  auto lse_of = [&](int k) { return (k < pre ? p.pre_lse : p.own_lse)[place(k)]; };
  float top = -INFINITY;
  for (int k = lane; k < parts; k += 32) top = fmaxf(top, lse_of(k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.f : top;
  float acc[16], sum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const int64_t from = place(k);
    const float w = ex2((k < pre ? p.pre_lse : p.own_lse)[from] - base);
    const float4* src = reinterpret_cast<const float4*>((k < pre ? p.pre_part : p.own_part) + from * kLat) + lane;
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

namespace {

// Sizes and places of a call's workspace; returns its bytes.
size_t shared_layout(SharedParams& p) {
  const OwnLayout own = own_layout(p.d);
  const size_t rows = (size_t)p.d.B * p.d.R * p.d.H;
  p.own_n = own.n;
  p.own_row_blocks = own.row_blocks;
  p.pairs = std::max(1, device_sm_count() / 2);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* x = p.d.ws + at;
    at += (bytes + 255) / 256 * 256;
    return x;
  };
  p.head = reinterpret_cast<SharedHead*>(take(sizeof(SharedHead)));
  p.first = reinterpret_cast<int2*>(take((size_t)p.pairs * sizeof(int2)));
  p.start = reinterpret_cast<int32_t*>(take((size_t)p.d.B * 4));
  p.of = reinterpret_cast<int32_t*>(take((size_t)p.d.B * 4));
  p.groups = reinterpret_cast<SharedGroup*>(take((size_t)p.G * sizeof(SharedGroup)));
  p.line = reinterpret_cast<int64_t*>(take((size_t)p.G * 8));
  p.split = reinterpret_cast<int4*>(take((size_t)p.d.B * own.row_blocks * sizeof(int4)));
  const size_t pre_rows = rows + (size_t)p.pairs * kPfxRows, own_rows = rows + (size_t)own.ctas * own.n;
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
  p.G = (int)G;
  return shared_layout(p);
}

bool launch_latent_shared(const DecodeParams& d, const int64_t* cu, const int32_t* prefix, int64_t G, cudaStream_t s) {
  SharedParams p = {};
  p.d = d;
  p.cu = cu;
  p.prefix = prefix;
  p.G = (int)G;
  shared_layout(p);
  if (d.num_pages == 0) p.d.max_pages = 0;  // no cache: every length is taken as 0
  // lanes a group: as many as it has requests on average
  int width = 1;
  while (width < 32 && (int64_t)width * G < d.B) width *= 2;
  if (!launch_overlapped(kda_latent_groups_kernel, dim3(1), kGroupThreads, 0, s, 1, p, width)) return false;
  // (tables shorter than a tile have nothing to share)
  if (p.d.max_pages * p.d.page_size >= kPfxTile && !launch_latent_prefix(p, s)) return false;
  if (!launch_latent_own(p, s)) return false;
  const int64_t rows = (int64_t)d.B * d.R * d.H;
  return launch_overlapped(kda_latent_shared_join_kernel, dim3((unsigned)((rows + 7) / 8)), 256, 0, s, 1, p);
}

}  // namespace kda
