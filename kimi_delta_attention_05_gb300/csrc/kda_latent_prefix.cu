// Absorbed latent attention of many query rows over prefixes that they share, on
// CTA pairs.
//
// The rows of a group's requests lie side by side in q, and all of them see all of
// the prefix's whole tiles: no masks, and each cached row is read once a block of
// 128 query rows.  That is bound by the tensor cores (2 * 1088 flops a query row and
// cached row of 1152 bytes), or at 128 rows about equally by HBM.
//
// Products of a pair (cta_group::2, M = 128: 64 query rows a CTA, full rate):
//   S [128 rows x 128 tokens] = Q (64 rows a CTA) . K^T (64 tokens a CTA)
//   O [128 rows x 512]       += P (64 rows a CTA) . V  (128 tokens, 256 dims a CTA)
// With M = 128 a CTA's 64 rows x N columns lie on its 128 tensor-memory lanes as two
// halves of N / 2 columns, so O takes 256 columns and two S 128.  Rows on the M side
// keep their softmax within the CTA, four threads a row, and P needs no exchange;
// the pair halves what each SM holds of Q (73.7 KB) and V.
//
// Shared memory: Q, the tile as keys (64 tokens x 576, three column parts), as values
// (128 tokens x 256, two halves; a second copy from L2, as the token that a product
// counts as its k-th has to be the same in both CTAs) and P fill it: 229 KB, each once.
// Parts are refilled as soon as the products that read them are done, and needed
// again some 1800 cycles later, which covers the copies.  128 tokens a tile rather than
// 64 with two stages: a product of N = 64 takes 25 cycles for 16 of arithmetic, as Q's
// 2 KB are read for each (N = 128: 32 for 32).
//
// Work: the tiles of all items (group, block of 128 rows) in one line, cut into
// equal shares, one CTA pair a share.  Every piece leaves its normalised rows and
// their lse in fp32; the join adds them in the order of the tiles.
//
// Roles: warps 0-7 softmax and output, warp 8 queries and keys, warp 9 products
// (first CTA), warp 10 values.  Every wait is bounded.
#include <cstring>
#include <numeric>

#include "../../include/kda_latent.h"
#include "kda_latent.cuh"
#include "kda_latent_tc.cuh"

namespace kda {

constexpr int kPfxThreads = 352;
constexpr int kPfxKeyWarp = 8, kPfxMmaWarp = 9, kPfxValueWarp = 10;
constexpr int kPfxKeyPart = 64 * 3 * 128;        // 64 tokens of three 64-column blocks
constexpr int kPfxValuePart = 64 * 4 * 128;      // 64 tokens of four
constexpr int kPfxQ = 0;                         // [9 blocks][64 rows][128 bytes]
constexpr int kPfxQBytes = 9 * 64 * 128;
constexpr int kPfxK = kPfxQ + kPfxQBytes;        // 3 x [8 groups of 8 tokens][3 blocks][8 x 128 bytes]
constexpr int kPfxV = kPfxK + 3 * kPfxKeyPart;   // 2 x [8 groups of 8 tokens][4 blocks][8 x 128 bytes]
constexpr int kPfxP = kPfxV + 2 * kPfxValuePart; // [2 blocks of 64 tokens][64 rows][128 bytes]
constexpr int kPfxMax = kPfxP + 2 * 64 * 128;    // fp32 [4][64]: maxima, then sums, of a row's four threads
constexpr int kPfxBar = kPfxMax + 4 * 64 * 4;
// (those that the products wait for are the first CTA's)
constexpr int kFKeys = 0, kFValues = 3, kEKeys = 5, kEValues = 8, kFQ = 10, kEQ = 11, kFS = 12, kFP = 14, kFO = 15,
              kPfxBars = 16;
constexpr int kPfxTmem = kPfxBar + 8 * kPfxBars;
constexpr int kPfxAbort = kPfxTmem + 8;
constexpr int kPfxSmem = kPfxAbort + 8;
static_assert(kPfxK % 1024 == 0 && kPfxV % 1024 == 0 && kPfxP % 1024 == 0 && kPfxKeyPart % 1024 == 0,
              "operand images need 1024-byte alignment");
static_assert(kPfxSmem <= 232448, "exceeds the opt-in shared memory of one CTA");
constexpr int kPfxLeast = 2 * kPfxTileCost;  // least cost of a share: two tiles
constexpr float kPfxSlack = 8.0f;  // log2 growth of a maximum that is let pass

struct PrefixMaps {
  CUtensorMap q, keys, values;
};

// The pieces with tiles of one share [u0, u1) of the line of costs, in order.
struct PrefixPieces {
  SharedGroups groups;
  int64_t cap, u0, u1, pre;  // tokens that a table can hold; the share; start of the next item
  int g, block, row_heads;   // next item; R H
  // the current piece: its group, the group's first query row and their number, the piece's first row within it,
  // tiles [t0, t1), whether it is its item's first on the line
  int of, row0, rows, row, t0, t1, leads;
  // Called by whole warps; the values are broadcast, so that the compiler knows them as uniform.
  __device__ __forceinline__ bool next() {
    bool more = false;
    while (!more && g < groups.G && pre < u1) {
      const int64_t first = groups.cu[g], end = groups.cu[g + 1];
      const int tokens = shared_tokens(first, end, groups.prefix[g], cap);
      of = g;
      row0 = (int)first * row_heads;
      rows = tokens > 0 ? (int)(end - first) * row_heads : 0;
      row = block * kPfxRows;
      ++block;
      if (row + kPfxRows >= rows) {
        block = 0;
        ++g;
      }
      if (rows == 0) continue;
      const int tiles = tokens / kPfxTile;
      auto before = [&](int64_t u) {
        const int64_t d = u - pre - kPfxItemCost;
        return d <= 0 ? 0 : (int)min((int64_t)tiles, (d + kPfxTileCost - 1) / kPfxTileCost);
      };
      const int a = before(u0), b = before(u1);
      leads = a == 0;
      // An item lies on the line from its last tile to its first: a share that ends one item and begins another
      // takes the one's first tiles, then the other's last, and so do the others at the same time (read from
      // DRAM for 48 requests of three tokens behind two prefixes of 49152: 254 MB, the other way round 1010).
      t0 = tiles - b;
      t1 = tiles - a;
      pre += prefix_item_cost(tokens);
      more = t0 < t1;
    }
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    if (!same(more)) return false;
    of = same(of);
    row0 = same(row0);
    rows = same(rows);
    row = same(row);
    t0 = same(t0);
    t1 = same(t1);
    leads = same(leads);
    return true;
  }
};

__device__ __forceinline__ void tma_pair_5d(uint32_t dst, const void* map, int x, int y, int z, int w, int v, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(mbar)
      : "memory");
}

__global__ void __launch_bounds__(kPfxThreads, 1)
    kda_latent_prefix_kernel(const SharedParams sp, const int box, const __grid_constant__ PrefixMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const DecodeParams& p = sp.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank(), share = blockIdx.x >> 1;
  const uint32_t sb = smem_u32(smem), bars = sb + kPfxBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  auto lead = [&](int i) { return map_rank(bar(i), 0); };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kPfxAbort);

  if (warp == kPfxKeyWarp && lane == 0) {
    for (int i = 0; i < kPfxBars; ++i)
      mbar_init(bar(i), i == kFP ? 16 : i == kFQ || (i >= kFKeys && i < kEKeys) ? 2 : 1);
    *s_abort = (sb & 1023) ? 1 : 0;
    if (sb & 1023) atomicExch(p.status, KDA_ERR_DEVICE_TIMEOUT);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    prefetch_map(&maps.q);
    prefetch_map(&maps.keys);
    prefetch_map(&maps.values);
  }
  if (warp == kPfxMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sb + kPfxTmem), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
  }
  // (set up while the kernel before this one ends)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kPfxTmem);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // ---- this pair's share of the line of items: each thread sums a run of groups ----
  PrefixPieces it;
  it.groups = sp.groups;
  it.cap = p.max_pages * p.page_size;
  it.row_heads = p.R * p.H;
  {
    int64_t* scan = reinterpret_cast<int64_t*>(smem + kPfxMax);  // sums of the warps; then the share's first item
    const int G = sp.groups.G, run = (G + kPfxThreads - 1) / kPfxThreads;
    const int g0 = min(G, tid * run), g1 = min(G, g0 + run);
    int bad = 0;
    int64_t mine = 0;
    auto cost_of = [&](int g) {
      const int64_t first = sp.groups.cu[g], end = sp.groups.cu[g + 1];
      bad |= first < 0 || end < first || end > p.B || (g == 0 && first != 0) || (g == G - 1 && end != p.B);
      const int tokens = shared_tokens(first, end, sp.groups.prefix[g], it.cap);
      if (tokens == 0 || bad) return (int64_t)0;
      return ((end - first) * it.row_heads + kPfxRows - 1) / kPfxRows * prefix_item_cost(tokens);
    };
    for (int g = g0; g < g1; ++g) mine += cost_of(g);
    int64_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    if (lane == 31) scan[warp] = before;
    before -= mine;
    const bool refused = __syncthreads_or(bad);  // (the requests' own pass reports it)
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kPfxThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    if (refused) total = 0;
    const int64_t size = max((int64_t)kPfxLeast, div_costs(total + sp.pairs - 1, sp.pairs));
    it.u0 = min(total, share * size);
    it.u1 = min(total, it.u0 + size);
    const bool writes = blockIdx.x == 0;
    if (writes && tid == 0) *sp.head = {total, size};
    if (writes || (it.u0 >= before && it.u0 < before + mine)) {
      int64_t pre = before;
      for (int g = g0; g < g1; ++g) {
        const int64_t cost = cost_of(g);
        if (writes) sp.line[g] = pre;
        if (it.u0 >= pre && it.u0 < pre + cost) {
          const int64_t item = prefix_item_cost(shared_tokens(sp.groups.cu[g], sp.groups.cu[g + 1], sp.groups.prefix[g], it.cap));
          const int64_t block = div_costs(it.u0 - pre, item);
          scan[12] = g;
          scan[13] = block;
          scan[14] = pre + block * item;
        }
        pre += cost;
      }
    }
    __syncthreads();
    const bool any = it.u0 < it.u1;
    it.g = any ? (int)scan[12] : G;
    it.block = any ? (int)scan[13] : 0;
    it.pre = any ? scan[14] : 0;
    __syncthreads();  // the place goes to the softmax
  }
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (mbar_try_wait(b, parity) || *s_abort) return;
    if (!mbar_wait_bounded(b, parity)) {
      atomicExch(p.status, KDA_ERR_DEVICE_TIMEOUT);
      *s_abort = 1;
    }
  };
  auto stop = [&]() {
    __syncwarp();
    return __any_sync(0xffffffffu, *s_abort != 0) != 0;
  };
  // After a timeout: copies still in flight land in memory of this CTA, which stays until the
  // cluster's last barrier; they are few and unconditional, so a bounded pause is enough.
  auto pause = [&]() {
    const long long t0 = clock64();
    while (clock64() - t0 < (1LL << 22)) {
    }
  };
  // The request of a piece's group whose row of the table is read: the first that sees the shared tokens; -1: none
  // does, and what is read does not count.
  auto source_of = [&]() {
    const int64_t first = sp.groups.cu[it.of], end = sp.groups.cu[it.of + 1];
    const int tokens = shared_tokens(first, end, sp.groups.prefix[it.of], it.cap);
    for (int64_t b = first; b < end; b += 32) {
      const uint32_t in =
          __ballot_sync(0xffffffffu, b + lane < end && sees_shared(p.lens[min(b + lane, end - 1)], it.cap, p.R, tokens));
      if (in) return (int)b + __ffs(in) - 1;
    }
    return -1;
  };
  // Page and 8-token group of the run of `box` tokens that starts at a token of the prefix.
  auto place = [&](int source, int64_t token, int& group) {
    const uint32_t in_table = (uint32_t)token / (uint32_t)p.page_size;
    int page = source < 0 ? (int)p.num_pages : p.table[source * p.table_stride + in_table];
    group = (int)((uint32_t)token - in_table * (uint32_t)p.page_size) >> 3;
    if (source >= 0 && (page < 0 || page >= p.num_pages)) {
      atomicExch(p.status, KDA_ERR_BAD_PAGE);
      page = (int)p.num_pages;  // past the map: reads as zeros
    }
    return page;
  };

  if (warp == kPfxKeyWarp) {
    // ---- a piece's query rows, and this CTA's 64 tokens of each tile as keys ----
    const int runs = 64 / box;
    int n = 0, q = 0;
    bool gone = false;
    while (!gone && it.next()) {
      const int source = source_of();
      for (int t = it.t0; t < it.t1 && !gone; ++t, ++n) {
        int page = 0, group = 0;
        if (lane < runs) page = place(source, (int64_t)t * kPfxTile + rank * 64 + lane * box, group);
        if (t == it.t0) {
          if (q > 0) wait(bar(kEQ), (uint32_t)((q - 1) & 1));
          if ((gone = stop())) break;
          if (lane == 0) {
            const uint32_t full = lead(kFQ);
            mbar_expect_tx_cluster(full, kPfxQBytes);
            tma_pair_3d(sb + kPfxQ, &maps.q, 0, it.row0 + it.row + rank * 64, 0, full);
          }
          ++q;
        }
        for (int c = 0; c < 3; ++c) {
          if (n > 0) wait(bar(kEKeys + c), (uint32_t)((n - 1) & 1));
          if ((gone = stop())) break;
          const uint32_t full = lead(kFKeys + c);
          if (lane == 0) mbar_expect_tx_cluster(full, kPfxKeyPart);
          __syncwarp();
          if (lane < runs)
            tma_pair_5d(sb + kPfxK + c * kPfxKeyPart + lane * box * (3 * 128), &maps.keys, 0, 0, 3 * c, group, page, full);
        }
      }
    }
    if (gone && lane == 0) pause();
  } else if (warp == kPfxValueWarp) {
    // ---- all 128 tokens of each tile, this CTA's half of the value dimensions ----
    const int runs = 64 / box;
    int n = 0;
    bool gone = false;
    while (!gone && it.next()) {
      const int source = source_of();
      for (int t = it.t0; t < it.t1 && !gone; ++t, ++n) {
        int page = 0, group = 0;
        if (lane < 2 * runs) page = place(source, (int64_t)t * kPfxTile + lane * box, group);
        for (int h = 0; h < 2; ++h) {
          if (n > 0) wait(bar(kEValues + h), (uint32_t)((n - 1) & 1));
          if ((gone = stop())) break;
          const uint32_t full = lead(kFValues + h);
          if (lane == 0) mbar_expect_tx_cluster(full, kPfxValuePart);
          __syncwarp();
          const int run = lane - h * runs;
          if (run >= 0 && run < runs)
            tma_pair_5d(sb + kPfxV + h * kPfxValuePart + run * box * (4 * 128), &maps.values, 0, 0, 4 * rank, group, page, full);
        }
      }
    }
    if (gone && lane == 0) pause();
  } else if (warp == kPfxMmaWarp) {
    // ---- products of the pair, issued by its first CTA: a tile's scores, then the values of the tile before ----
    if (rank == 0) {
      const uint32_t id_s = idesc_bf16(128, kPfxTile, false, false), id_o = idesc_bf16(128, 256, false, true);
      const uint64_t d_q = smem_desc(sb + kPfxQ, 16, 1024), d_k = smem_desc(sb + kPfxK, 16, 3 * 1024);
      const uint64_t d_p = smem_desc(sb + kPfxP, 16, 1024), d_v = smem_desc(sb + kPfxV, 1024, 4 * 1024);
      auto ready = [&](int b, int n) {
        wait(bar(b), (uint32_t)(n & 1));
        __syncwarp();
        tc_fence_after();
      };
      int n = 0, q = 0;      // tiles whose scores are on the way, pieces
      bool fresh = false;    // the tile before is the first of its piece
      auto values = [&](int m, bool first) {
        ready(kFP, m);
        const uint32_t more = first ? 0u : 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ready(kFValues + h, m);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_ss<true>(tmem + 128 * j, d_p + (uint64_t)((h * 8192 + ks * 32) >> 4),
                             d_v + (uint64_t)((h * kPfxValuePart + ks * 8192 + j * 2048) >> 4), id_o, h + ks > 0 ? 1u : more);
            mma_commit<true>(bar(kEValues + h));
            if (h == 1) mma_commit<true>(bar(kFO));
          }
          __syncwarp();
        }
      };
      while (it.next()) {
        for (int t = it.t0; t < it.t1; ++t, ++n) {
          if (t == it.t0) ready(kFQ, q++);
          const uint32_t s = tmem + 256 + 64 * (n & 1);
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            ready(kFKeys + c, n);
            if (elect_one()) {
#pragma unroll
              for (int b = 0; b < 3; ++b)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  mma_ss<true>(s, d_q + (uint64_t)(((3 * c + b) * 8192 + ks * 32) >> 4),
                               d_k + (uint64_t)((c * kPfxKeyPart + b * 1024 + ks * 32) >> 4), id_s, c + b + ks > 0);
              mma_commit<true>(bar(kEKeys + c));
              if (c == 2) {
                mma_commit<true>(bar(kFS + (n & 1)));
                if (t + 1 == it.t1) mma_commit<true>(bar(kEQ));
              }
            }
            __syncwarp();
          }
          if (n > 0) values(n - 1, fresh);
          fresh = t == it.t0;
        }
      }
      if (n > 0) {
        values(n - 1, fresh);
        mbar_wait_bounded(bar(kFO), (uint32_t)((n - 1) & 1));  // before tensor memory is freed
      }
    }
  } else {
    // ---- softmax and output: lane 32 w .. of tensor memory is row 32 (w % 2) .. with the tokens (dimensions) of
    //      half w / 2 of a product; warps 4-7 take the second half of the columns ----
    const int w4 = warp & 3, right = warp >> 2, side = w4 >> 1;
    const int r = 32 * (w4 & 1) + lane;  // query row of this CTA's 64
    const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
    float* wmax = reinterpret_cast<float*>(smem + kPfxMax);
    const int quarter = 2 * side + right;
    const uint32_t p_row = sb + kPfxP + side * 8192 + r * 128;
    int n = 0;
    while (it.next()) {
      float m = -INFINITY, l = 0.f;
      for (int t = it.t0; t < it.t1; ++t, ++n) {
        wait(bar(kFS + (n & 1)), (uint32_t)((n >> 1) & 1));
        __syncwarp();
        tc_fence_after();
        float v[32];
        tc_ld32(tmem + lane_base + 256 + 64 * (n & 1) + 32 * right, v);
        float x = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          v[i] *= p.scale_log2;
          x = fmaxf(x, v[i]);
        }
        // the running maximum moves only when it grows by more than 2^8 (exact: the result is divided by the sum
        // taken with the same maximum), so that O is rarely rescaled
        if (named_bar_or(1, 256, x > m + kPfxSlack)) {
          wmax[quarter * 64 + r] = x;
          named_bar(1, 256);
          x = fmaxf(fmaxf(wmax[r], wmax[64 + r]), fmaxf(wmax[128 + r], wmax[192 + r]));
          float f = 1.0f;
          if (x > m + kPfxSlack) {
            f = ex2(m - x);
            m = x;
            l *= f;
          }
          if (t > it.t0) {  // O of the tiles so far to the new maxima
            wait(bar(kFO), (uint32_t)((n - 1) & 1));
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              float o[16];
              tc_ld16(tmem + lane_base + 128 * right + c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tc_st16(tmem + lane_base + 128 * right + c, o);
            }
            tc_st_wait();
          }
          named_bar(1, 256);  // wmax is read
        }
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          v[i] = ex2(v[i] - base);
          l += v[i];
        }
        if (n > 0) wait(bar(kFO), (uint32_t)((n - 1) & 1));  // P of the tile before is read
        __syncwarp();
        // weights rounded to bf16, the operands' type; the sums are taken before it
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = p_row + (((4 * right + i) ^ (r & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(pack_bf16(v[8 * i], v[8 * i + 1])),
                       "r"(pack_bf16(v[8 * i + 2], v[8 * i + 3])), "r"(pack_bf16(v[8 * i + 4], v[8 * i + 5])),
                       "r"(pack_bf16(v[8 * i + 6], v[8 * i + 7]))
                       : "memory");
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(kFP));
      }
      // ---- the piece's rows ----
      wmax[quarter * 64 + r] = l;
      named_bar(1, 256);
      const float sum = (wmax[r] + wmax[64 + r]) + (wmax[128 + r] + wmax[192 + r]);
      const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
      const int row = it.row + 64 * rank + r;  // of the group
      const bool there = row < it.rows;
      // a row's first part at its own place, a later one at this share's
      const int64_t at = it.leads ? (int64_t)it.row0 + row
                                  : (int64_t)p.B * p.R * p.H + (int64_t)share * kPfxRows + 64 * rank + r;
      if (quarter == 0 && there) sp.pre_lse[at] = sum == 0.f ? -INFINITY : m + __log2f(sum);
      wait(bar(kFO), (uint32_t)((n - 1) & 1));
      __syncwarp();
      tc_fence_after();
      // A warp turns 32 rows x 16 dimensions in 2 KB of P's place (its own: the last products have read it) and
      // stores 64 bytes of 8 rows at a time; a thread's own row at a time, each store touched 32 lines and the
      // 128 KB took 12000 cycles.
      const uint32_t turn = sb + kPfxP + warp * 2048;
      const int64_t first = at - r + 32 * (w4 & 1);  // this warp's first row; all of one part are side by side
      const int rows_there = it.rows - (it.row + 64 * rank + 32 * (w4 & 1));
      float* dst = sp.pre_part + first * kLat + 256 * side + 128 * right;
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        float o[16];
        tc_ld16(tmem + lane_base + 128 * right + c, o);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(turn + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)),
                       "f"(o[4 * i] * inv), "f"(o[4 * i + 1] * inv), "f"(o[4 * i + 2] * inv), "f"(o[4 * i + 3] * inv)
                       : "memory");
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row_of = 8 * k + (lane >> 2), piece = lane & 3;
          float4 x;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                       : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                       : "r"(turn + row_of * 64 + ((piece ^ (row_of >> 1 & 3)) << 4))
                       : "memory");
          if (row_of < rows_there) *reinterpret_cast<float4*>(dst + row_of * kLat + c + 4 * piece) = x;
        }
        __syncwarp();
      }
      tc_fence_before();
      named_bar(1, 256);  // wmax is read
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of this pair reaches a CTA that has left
  tc_fence_after();
  if (warp == kPfxMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
}

bool launch_latent_prefix(const SharedParams& sp, cudaStream_t s) {
  const DecodeParams& p = sp.d;
  PrefixMaps maps;
  memset(&maps, 0, sizeof(maps));
  const int box = (int)std::gcd<int64_t, int64_t>(p.page_size, 64);
  const int64_t rows = (int64_t)p.B * p.R * p.H;
  {  // query rows as [64 values][rows][9 blocks]: one copy brings 64 rows
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, 9};
    const cuuint64_t strides[2] = {kLatRow * 2, 128};
    const cuuint32_t shape[3] = {64, 64, 9};
    if (!encode_map_bf16(&maps.q, p.q, 3, dims, strides, shape)) return false;
  }
  if (p.num_pages > 0) {  // the cache as [64 values][8 tokens][9 blocks][8-token groups of a page][pages]
    const cuuint64_t dims[5] = {64, 8, 9, (cuuint64_t)p.page_size / 8, (cuuint64_t)p.num_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)p.token_stride * 2, 128, (cuuint64_t)p.token_stride * 16,
                                   (cuuint64_t)p.page_stride * 2};
    cuuint32_t shape[5] = {64, 8, 3, (cuuint32_t)box / 8, 1};
    if (!encode_map_bf16(&maps.keys, p.cache, 5, dims, strides, shape)) return false;
    shape[2] = 4;
    if (!encode_map_bf16(&maps.values, p.cache, 5, dims, strides, shape)) return false;
  }
  static std::once_flag once[64];
  static cudaError_t rc[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::call_once(once[dev], [&] {
    rc[dev] = cudaFuncSetAttribute(kda_latent_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPfxSmem);
  });
  if (rc[dev] != cudaSuccess) return false;
  return launch_overlapped(kda_latent_prefix_kernel, dim3(2 * sp.pairs), kPfxThreads, kPfxSmem, s, 2, sp, box, maps);
}

}  // namespace kda
