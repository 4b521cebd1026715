// Absorbed latent attention of a batch whose requests share prefixes, on CTA pairs;
// parts joined by a second small kernel.
//
// The query rows of a group's requests lie side by side in q.  An item is 128 of
// them: its tiles are the prefix's (128 tokens, whole ones that all new tokens of a
// request see), read once for all rows, then each request's own, of which the other
// requests' rows see nothing.  So a cached row of the prefix crosses HBM once a
// group and L2 once an item, and a request's own once: bound by the tensor cores (2 *
// 1088 flops a query row and cached row of 1152 bytes) where many rows share, else by
// HBM.  An own tile costs a whole one whatever the rows that see it and the tokens it
// has, 1.1 us for up to 128 tokens on two SMs: less than HBM takes for 128 with all SMs
// at it, more where a request has few tokens of its own.
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
// 2 KB are read for each (N = 128: 32 for 32).  A tile behind another takes 2190
// cycles, the products' own time.
//
// Work: the tiles of all items in one line, cut into equal shares, one CTA pair a
// share, or an item a share where none is much longer than that.  A piece that is its
// whole item writes its rows; the others leave normalised rows and their lse in fp32,
// which the join adds in the order of the tiles.
//
// Rows that are not finite: with weight 0 they make NaN of the O of rows that do not see
// them, whose weights are finite; those rows are marked, and the join computes them anew.
//
// Measured: 48 requests of three tokens behind two prefixes of 49152, 32 heads, 274 us or
// 1.81 PFLOP/s, tensor pipe 86 % active; 256 requests of up to 512 own tokens behind 4096,
// 32 heads, 74 us, of which 7 pass before a share's first scores (its plan 3.5, first
// copies and first product); 24 prefixes of up to 8192, 16 heads, 82 us: a tile takes 3400
// cycles, as most come from HBM, at 5 TB/s while there are any, and a piece's 128 KB of
// fp32 output a CTA 4 to 6 us, the join 5.
//
// Roles: warps 0-7 softmax and output, warp 8 queries and keys, warp 9 products
// (first CTA), warp 10 values.  Every wait is bounded.
#include <algorithm>
#include <cstring>
#include <numeric>

#include "../../include/kda_latent.h"
#include "kda_latent.cuh"
#include "kda_latent_tc.cuh"

namespace kda {

constexpr int kShTile = 128;       // cached rows of a tile
constexpr int kShRows = 128;       // query rows of an item, a CTA pair's
constexpr int kShThreads = 352, kShWarps = kShThreads / 32;
constexpr int kShKeyWarp = 8, kShMmaWarp = 9, kShValueWarp = 10;
// The line's costs: 4 a tile, and what an item's set-up and output take (8, 12, 14, 16 and 20 measured: 82.8, 81.9, 81.6,
// 82.1 and 82.4 us on 24 prefixes of up to 8192); least cost of a share.  (A request's own tiles, which come from HBM, take
// longer than the prefix's, but at 6 they made the shares less even: 95.8 against 89.4 at 4, with an item's cost of 8 and
// more fixed cost than now.)
constexpr int kShTileCost = 4, kShItemCost = 16, kShLeast = 2 * kShTileCost;
constexpr int kShWhole = 16;       // cost that cuts add, beside that which grows with the items
constexpr float kShSlack = 8.0f;   // log2 growth of a maximum that is let pass

// The join: CTAs of the grid an SM, rows of a CTA at a time, and how many such an item has.  Three CTAs are resident (80
// registers), the fourth begins as another ends: 2, 3, 4 and 6 an SM took 85.5, 85.1, 82.0 and 82.0 us on 24 prefixes of up to
// 8192, and 285, 280, 274 and 275 on 48 requests behind two of 49152.  (128 threads: 86.7 against 82.3; a CTA for every 8 rows
// that an item could have, most of them empty: 83.1.)
constexpr int kShJoinThreads = 256, kShJoinCtas = 4;
constexpr int kShJoinRows = kShJoinThreads / 32, kShJoinUnits = kShRows / kShJoinRows;

constexpr int kShKeyPart = 64 * 3 * 128;      // 64 tokens of three 64-column blocks
constexpr int kShValuePart = 64 * 4 * 128;    // 64 tokens of four
constexpr int kShQ = 0;                       // [9 blocks][64 rows][128 bytes]
constexpr int kShQBytes = 9 * 64 * 128;
constexpr int kShK = kShQ + kShQBytes;        // 3 x [8 groups of 8 tokens][3 blocks][8 x 128 bytes]
constexpr int kShV = kShK + 3 * kShKeyPart;   // 2 x [8 groups of 8 tokens][4 blocks][8 x 128 bytes]
constexpr int kShP = kShV + 2 * kShValuePart; // [2 blocks of 64 tokens][64 rows][128 bytes]
constexpr int kShMax = kShP + 2 * 64 * 128;   // fp32 [4][64]: maxima, then sums, of a row's four threads
constexpr int kShBar = kShMax + 4 * 64 * 4;
// (those that the products wait for are the first CTA's; kFTail is each CTA's own)
constexpr int kFKeys = 0, kFValues = 3, kEKeys = 5, kEValues = 8, kFQ = 10, kEQ = 11, kFS = 12, kFP = 14, kFO = 15,
              kFTail = 16, kShBars = 17;
constexpr int kShTmem = kShBar + 8 * kShBars;
constexpr int kShAbort = kShTmem + 8;
constexpr int kShItems = (kShAbort + 8 + 15) / 16 * 16;  // the share's first items
constexpr int kShKept = 32;
constexpr int kShSmem = kShItems + 32 * kShKept;
static_assert(kShK % 1024 == 0 && kShV % 1024 == 0 && kShP % 1024 == 0 && kShKeyPart % 1024 == 0,
              "operand images need 1024-byte alignment");
static_assert(kShSmem <= 232448, "exceeds the opt-in shared memory of one CTA");
static_assert((KDA_LATENT_SHARED_GROUPS + 1) * 4 <= kShP, "the groups' first items lie in the operands' place");

// 128 query rows of a group, and their place on the line of costs.
struct SharedItem {
  int row, rows;      // the group's first row, and its rows
  int block;          // of these
  int common;         // tiles of the prefix
  int64_t start;      // on the line
  int tiles;          // all
  int pad;
};
static_assert(sizeof(SharedItem) == 32, "read as two 16-byte pieces");

struct SharedHead {
  int64_t size;       // cost of a share
  int items, cut;     // all, and those that shares may have cut: all or none
};

struct SharedParams {
  DecodeParams d;
  SharedGroups groups;
  int pairs;                   // CTA pairs, a share each
  // workspace
  SharedHead* head;
  SharedItem* items;           // written by the first CTA (all) and by each whose share they are in (the same)
  int* spoilt;                 // [2 * pairs], of each CTA: whether it has found a row that another request's rows spoilt
  float *part, *part_lse;      // fp32 rows and their lse (log2): a row's first part at its own place, those that begin
                               // within a share behind them; [B R H + pairs * kShRows]
};

struct SharedMaps {
  CUtensorMap q, keys, values;
};

// a / b of numbers that are not negative, in 32 bits where they fit (a 64-bit division takes some 100 instructions)
__device__ __forceinline__ int64_t div_costs(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t item_cost(int tiles) { return kShItemCost + (int64_t)tiles * kShTileCost; }

// What one call's groups and lengths mean, in 32 bits (offsets that do not fit are found before they are used): the code
// of the set-up runs once, and every instruction of it is fetched for that.
struct SharedView {
  const int64_t* cu;
  const int32_t *prefix, *lens;
  int B, R, H, rows_of;        // rows_of: R H, the rows of a request
  int cap;                     // tokens that a table can hold
  bool alone;                  // offsets that do not fit: all requests are one group without a prefix
  __device__ __forceinline__ int first(int g) const { return alone ? 0 : (int)cu[g]; }
  __device__ __forceinline__ int end(int g) const { return alone ? B : (int)cu[g + 1]; }
  // tokens of the prefix that are shared: whole tiles, of groups of two and more
  __device__ __forceinline__ int tokens(int g, int requests) const {
    return alone || requests < 2 ? 0 : min(max(prefix[g], 0), cap) / kShTile * kShTile;
  }
  __device__ __forceinline__ int len(int b) const { return min(max(lens[b], 0), cap); }
  // first token that a request takes on its own: behind the shared ones if all its new tokens see them
  __device__ __forceinline__ int own_from(int n, int shared) const { return shared > 0 && n - (R - 1) >= shared ? shared : 0; }
  __device__ __forceinline__ int own_tiles(int b, int shared) const {
    const int n = len(b);
    return (n - own_from(n, shared) + kShTile - 1) / kShTile;
  }
  // the request that has a row (or, within a group, the number of one)
  __device__ __forceinline__ int request(int row) const { return (int)((uint32_t)row / (uint32_t)rows_of); }
};

__device__ __forceinline__ SharedView shared_view(const SharedParams& p) {
  return {p.groups.cu, p.groups.prefix, p.d.lens, p.d.B, p.d.R, p.d.H, p.d.R * p.d.H, (int)(p.d.max_pages * p.d.page_size),
          false};
}

// The pieces of one share [u0, u1) of the line of costs, in order.
struct SharedPieces {
  const SharedItem *items, *kept;  // all; the share's first ones in shared memory
  int next_item, first_item, end_item;  // (items outside [first_item, end_item) may not have been written yet)
  int64_t u0, u1;
  // the current piece: its item's (with what is needed of its group, which saves two loads, 0.3 us, before the first copies),
  // the tiles [t0, t1) of all, whether it is the item's first on the line
  int row, rows, block, common, tiles, t0, t1, leads;
  // Called by whole warps; the values are broadcast, so that the compiler knows them as uniform.
  __device__ __forceinline__ bool next() {
    bool more = false;
    while (!more && next_item < end_item) {
      const SharedItem* from = next_item - first_item < kShKept ? kept + (next_item - first_item) : items + next_item;
      const int4 a = *reinterpret_cast<const int4*>(from), b = *(reinterpret_cast<const int4*>(from) + 1);
      const int64_t start = (int64_t)(uint32_t)b.x | (int64_t)b.y << 32;
      ++next_item;
      row = a.x;
      rows = a.y;
      block = a.z;
      common = a.w;
      tiles = b.z;
      auto before = [&](int64_t u) {
        const int64_t d = u - start - kShItemCost;
        return d <= 0 ? 0 : (int)min((int64_t)tiles, (d + kShTileCost - 1) / kShTileCost);
      };
      const int x = before(u0), y = before(u1);
      leads = x == 0;
      // An item lies on the line from its last tile to its first: a share that ends one item and begins another
      // takes the one's first tiles, then the other's last, and so do the others at the same time (read from
      // DRAM for 48 requests of three tokens behind two prefixes of 49152: 285 MB, the other way round 1010).
      t0 = tiles - y;
      t1 = tiles - x;
      more = t0 < t1 || (tiles == 0 && start >= u0);  // (an item without tiles: rows that see nothing)
    }
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    if (!same(more)) return false;
    row = same(row);
    rows = same(rows);
    block = same(block);
    common = same(common);
    tiles = same(tiles);
    t0 = same(t0);
    t1 = same(t1);
    leads = same(leads);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t1 - t0 == tiles; }
};

// A walk over a piece's tiles, the prefix's and own ones: whose tokens each has, and which.
struct SharedTile {
  int request;      // whose own tokens, or -1: the prefix's
  int token, valid; // first token, and how many
  int first, last;  // the item's requests
  int left;         // tiles of this request behind the current one
  int shared;       // tokens of the prefix that are shared
  int turn;         // the tile at which the prefix begins: the piece's first, or behind its own ones where it takes those first
  __device__ __forceinline__ void own(const SharedView& v, int b, int skip) {
    for (;; ++b) {
      const int n = b <= last ? v.own_tiles(b, shared) : INT32_MAX;  // (no tile is asked for behind the last request's)
      if (skip < n) {
        left = n - skip - 1;
        break;
      }
      skip -= n;
    }
    request = b;
    const int n = v.len(min(b, last));
    token = v.own_from(n, shared) + skip * kShTile;
    valid = min(kShTile, n - token);
  }
  __device__ __forceinline__ void prefix(const SharedPieces& it) {
    request = -1;
    token = it.t0 * kShTile;
    valid = kShTile;
  }
  __device__ __forceinline__ void start(const SharedView& v, const SharedPieces& it) {
    const int row = it.block * kShRows;
    shared = it.common * kShTile;  // (0 where none of the requests sees all of the prefix)
    first = v.request(it.row + row);
    last = v.request(it.row + min(it.rows, row + kShRows) - 1);
    // Own tiles come from HBM, the prefix's from L2 where the group has several items: every second one takes its own
    // first, so that not all wait for HBM at the same time (256 requests of up to 512 own tokens behind 4096: 75.7 -> 73.5 us).
    turn = it.t0;
    if (it.t0 < it.common && it.t1 > it.common && (it.block & 1) && it.rows > 4 * kShRows) turn += it.t1 - it.common;
    prefix(it);
    if ((it.t0 >= it.common && it.t0 < it.t1) || turn > it.t0) own(v, first, max(0, it.t0 - it.common));
  }
  // The request whose row of the table names the prefix: the first that takes it as shared, where there is one.
  __device__ __forceinline__ int source(const SharedView& v) const {
    int b = first;
    while (b < last && v.own_from(v.len(b), shared) == 0) ++b;
    return b;
  }
  // to tile t of the piece, which has one
  __device__ __forceinline__ void advance(const SharedView& v, const SharedPieces& it, int t) {
    if (t == turn) {
      prefix(it);
    } else if (request < 0 && token + kShTile < it.common * kShTile) {
      token += kShTile;
    } else if (request < 0) {
      own(v, first, 0);
    } else if (left > 0) {
      --left;
      token += kShTile;
      valid = min(kShTile, v.len(request) - token);
    } else {
      own(v, request + 1, 0);
    }
  }
};

__device__ __forceinline__ void tma_pair_5d(uint32_t dst, const void* map, int x, int y, int z, int w, int v, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(mbar)
      : "memory");
}

__global__ void __launch_bounds__(kShThreads, 1)
    kda_latent_shared_kernel(const SharedParams sp, const int box, const __grid_constant__ SharedMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const DecodeParams& p = sp.d;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank(), share = blockIdx.x >> 1;
  const uint32_t sb = smem_u32(smem), bars = sb + kShBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  auto lead = [&](int i) { return map_rank(bar(i), 0); };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kShAbort);
  volatile int* s_spoilt = s_abort + 1;

  if (warp == kShKeyWarp && lane == 0) {
    for (int i = 0; i < kShBars; ++i)
      mbar_init(bar(i), i == kFP ? 16 : i == kFQ || (i >= kFKeys && i < kEKeys) ? 2 : 1);
    *s_abort = (sb & 1023) ? 1 : 0;
    *s_spoilt = 0;
    if (sb & 1023) atomicExch(p.status, KDA_ERR_DEVICE_TIMEOUT);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    prefetch_map(&maps.q);
    if (p.num_pages > 0) {
      prefetch_map(&maps.keys);
      prefetch_map(&maps.values);
    }
  }
  if (warp == kShMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sb + kShTmem), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();  // (waited for behind the plan)
  // (set up while the kernel before this one ends)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  // ---- this pair's share of the line: every CTA finds the items and their costs for itself ----
  SharedPieces it;
  SharedView view = shared_view(sp);
  {
    int* first_item = reinterpret_cast<int*>(smem);                // [G] items before each group
    int64_t* scan = reinterpret_cast<int64_t*>(smem + kShMax);     // sums of the warps; then the share's first item
    const bool writes = blockIdx.x == 0;
    auto prefix_sum = [&](auto x, auto& total) {                   // over the threads before this one
      auto upto = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const auto y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) scan[warp] = upto;
      __syncthreads();
      upto -= x;
      total = 0;
#pragma unroll 1
      for (int w = 0; w < kShWarps; ++w) {
        const auto s = (decltype(x))scan[w];
        if (w < warp) upto += s;
        total += s;
      }
      __syncthreads();  // sums are read
      return upto;
    };
    // groups: a run a thread
    int G = sp.groups.G;
    const int run = (G + kShThreads - 1) / kShThreads, g0 = min(G, tid * run), g1 = min(G, g0 + run);
    int bad = 0, far = 0, mine = 0;
    auto blocks_of = [&](int requests) { return (int)(((uint32_t)(requests * view.rows_of) + kShRows - 1) / kShRows); };
    for (int g = g0; g < g1; ++g) {
      const int64_t first = view.cu[g], end = view.cu[g + 1];
      const int len = view.prefix[g];
      bad |= first < 0 || end < first || end > p.B || (g == 0 && first != 0) || (g == G - 1 && end != p.B);
      if (!bad) mine += blocks_of((int)(end - first));
      far |= end > first && (len < 0 || len > view.cap);
    }
    bad = __syncthreads_or(bad);
    if (writes && far) atomicExch(p.status, KDA_ERR_BAD_LENGTHS);
    if (bad) {  // (a group without a prefix: every request on its own)
      if (writes && tid == 0) atomicExch(p.status, KDA_ERR_BAD_SEQLENS);
      view.alone = true;
      G = 1;
      mine = tid == 0 ? blocks_of(p.B) : 0;
    }
    int items, at = prefix_sum(mine, items);
    if (bad) {
      if (tid == 0) first_item[0] = 0;
    } else {
      for (int g = g0; g < g1; ++g) {
        first_item[g] = at;
        at += blocks_of(view.end(g) - view.first(g));
      }
    }
    __syncthreads();
    // items: a run a thread
    const int per = (items + kShThreads - 1) / kShThreads;
    const int i0 = min(items, tid * per), i1 = min(items, i0 + per);
    int odd = 0, group = 0;
    auto look = [&](int i, int& g, SharedItem& x) {  // item i, g being the group of the one before
      while (g + 1 < G && first_item[g + 1] <= i) ++g;
      x.block = i - first_item[g];
      const int first = view.first(g), n = view.end(g) - first, row = x.block * kShRows;
      x.row = first * view.rows_of;
      x.rows = n * view.rows_of;
      const int shared = view.tokens(g, n);
      const int b0 = first + view.request(row), b1 = first + view.request(min(n * view.rows_of, row + kShRows) - 1);
      x.common = 0;
      x.tiles = 0;
#pragma unroll 4
      for (int b = b0; b <= b1; ++b) {
        const int raw = view.lens[b], len = min(max(raw, 0), view.cap), from = view.own_from(len, shared);
        odd |= raw != len;
        if (from > 0) x.common = shared / kShTile;
        x.tiles += (len - from + kShTile - 1) / kShTile;
      }
      x.tiles += x.common;
    };
    {
      int lo = 0, hi = G - 1;  // last group that begins at item i0 or before
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_item[mid] <= i0) lo = mid; else hi = mid - 1;
      }
      group = lo;
    }
    SharedItem x = {};
    int64_t cost = 0;
    int most = 0;  // tiles of an item
    for (int i = i0, g = group; i < i1; ++i) {
      look(i, g, x);
      cost += item_cost(x.tiles);
      most = max(most, x.tiles);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int* mosts = reinterpret_cast<int*>(scan + 16);
    if (lane == 0) mosts[warp] = most;
    if (writes && odd) atomicExch(p.status, KDA_ERR_BAD_LENGTHS);
    int64_t total, start = prefix_sum(cost, total);
    for (int w = 0; w < kShWarps; ++w) most = max(most, mosts[w]);
    int64_t size = max((int64_t)kShLeast, div_costs(total + sp.pairs - 1, sp.pairs));
    // No more items than pairs, and none that takes much longer than an equal share would with what cuts add, fp32 parts to
    // write, read and join, which grows with the items: every item is a share, and writes its rows.  Whole and cut, us: 64
    // items of 36 to 48 tiles 76 and 79, of 12 to 24 45 and 52, 72 of 12 to 16 37 and 49; 50 of 36 to 48 72 and 67, 32 of 12
    // 32.7 and 31.4, of 20 to 32 51 and 40, 16 of 12 to 16 34 and 25.
    const bool whole = items <= sp.pairs && item_cost(most) <= size + kShWhole + items * 3 / 4;
    if (whole) size = total + 1;  // (the join finds no cut)
    it.u0 = whole ? 0 : min(total, share * size);
    it.u1 = min(total, it.u0 + size);  // (whole items: those of the line that the pair takes are set below)
    it.items = sp.items;
    it.kept = reinterpret_cast<const SharedItem*>(smem + kShItems);
    if (writes && tid == 0) *sp.head = {size, items, whole ? 0 : items};
    const bool has = start < it.u1 && start + cost > it.u0;  // some of the share
    if (has) {  // its first and its last item
      int64_t begin = start;
      for (int i = i0, g = group; i < i1; ++i) {
        if (per > 1) look(i, g, x);
        const int64_t end = begin + item_cost(x.tiles);
        if (begin <= it.u0 && end > it.u0) scan[12] = i;
        if (begin < it.u1 && end >= it.u1) scan[13] = i;
        begin = end;
      }
    }
    __syncthreads();
    it.next_item = it.first_item = it.u0 < it.u1 ? (int)scan[12] : 0;
    it.end_item = it.u0 < it.u1 ? (int)scan[13] + 1 : 0;
    if (whole) {
      it.next_item = it.first_item = share;
      it.end_item = min(items, share + 1);
    }
    if (writes || has) {
      for (int i = i0, g = group; i < i1; ++i) {
        if (per > 1) look(i, g, x);
        x.start = start;
        const int64_t end = start + item_cost(x.tiles);
        if (writes || (start < it.u1 && end > it.u0)) sp.items[i] = x;
        if (start < it.u1 && end > it.u0 && i >= it.first_item && i - it.first_item < kShKept)
          reinterpret_cast<SharedItem*>(smem + kShItems)[i - it.first_item] = x;
        start = end;
      }
    }
    fence_proxy_async_smem();  // (the place of first_item goes to the tensor copies)
    __syncthreads();           // (and that of scan to the softmax)
  }
  cluster_wait();  // the other CTA's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kShTmem);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

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
  // Page and 8-token group of the run of `box` tokens that starts at a token of a request.
  auto place = [&](int request, int token, int& group) {
    const uint32_t in_table = (uint32_t)token / (uint32_t)p.page_size;
    int page = p.table[request * p.table_stride + in_table];
    group = (int)((uint32_t)token - in_table * (uint32_t)p.page_size) >> 3;
    if (page < 0 || page >= p.num_pages) {
      atomicExch(p.status, KDA_ERR_BAD_PAGE);
      page = (int)p.num_pages;  // past the map: reads as zeros
    }
    return page;
  };

  if (warp == kShKeyWarp) {
    // ---- a piece's query rows, and this CTA's 64 tokens of each tile as keys ----
    int n = 0, q = 0;
    bool gone = false;
    SharedTile tile;
    while (!gone && it.next()) {
      if (it.t0 == it.t1) continue;
      if (q > 0) wait(bar(kEQ), (uint32_t)((q - 1) & 1));
      if ((gone = stop())) break;
      if (lane == 0) {
        const uint32_t full = lead(kFQ);
        mbar_expect_tx_cluster(full, kShQBytes);
        tma_pair_3d(sb + kShQ, &maps.q, 0, it.row + it.block * kShRows + rank * 64, 0, full);
      }
      ++q;
      tile.start(view, it);
      const int source = it.t0 < it.common ? tile.source(view) : 0;
      int runs, page, group;  // of this CTA's 64 tokens; what is not copied is masked
      auto look = [&]() {
        runs = (min(64, max(0, tile.valid - rank * 64)) + box - 1) / box;
        page = group = 0;
        if (lane < runs) page = place(tile.request < 0 ? source : tile.request, tile.token + rank * 64 + lane * box, group);
      };
      look();
      for (int t = it.t0; t < it.t1 && !gone; ++t, ++n) {
        for (int c = 0; c < 3; ++c) {
          if (n > 0) wait(bar(kEKeys + c), (uint32_t)((n - 1) & 1));
          if ((gone = stop())) break;
          const uint32_t full = lead(kFKeys + c);
          if (lane == 0) mbar_expect_tx_cluster(full, runs * box * (3 * 128));
          __syncwarp();
          if (lane < runs)
            tma_pair_5d(sb + kShK + c * kShKeyPart + lane * box * (3 * 128), &maps.keys, 0, 0, 3 * c, group, page, full);
        }
        if (t + 1 < it.t1) {  // the next tile's places while this one's copies run
          tile.advance(view, it, t + 1);
          look();
        }
      }
    }
    if (gone && lane == 0) pause();
  } else if (warp == kShValueWarp) {
    // ---- all 128 tokens of each tile, this CTA's half of the value dimensions ----
    const int runs_of_half = 64 / box;
    int n = 0, tails = 0;
    bool gone = false;
    SharedTile tile;
    while (!gone && it.next()) {
      if (it.t0 == it.t1) continue;
      tile.start(view, it);
      const int source = it.t0 < it.common ? tile.source(view) : 0;
      for (int t = it.t0; t < it.t1 && !gone; ++t, ++n) {
        if (t > it.t0) tile.advance(view, it, t);
        int page = 0, group = 0;
        if (lane < 2 * runs_of_half && lane * box < tile.valid)
          page = place(tile.request < 0 ? source : tile.request, tile.token + lane * box, group);
        for (int h = 0; h < 2; ++h) {
          if (n > 0) wait(bar(kEValues + h), (uint32_t)((n - 1) & 1));
          if ((gone = stop())) break;
          const uint32_t full = lead(kFValues + h);
          const uint32_t dst = sb + kShV + h * kShValuePart;
          const int run = lane - h * runs_of_half, valid = min(64, max(0, tile.valid - h * 64));
          if (valid == 64) {
            if (lane == 0) mbar_expect_tx_cluster(full, kShValuePart);
            __syncwarp();
            if (run >= 0 && run < runs_of_half)
              tma_pair_5d(dst + run * box * (4 * 128), &maps.values, 0, 0, 4 * rank, group, page, full);
            continue;
          }
          // what lies behind the length takes part in the product with weight 0: it has to be finite.  The rows land
          // on a barrier of this CTA's own, those behind are cleared, and only then is the half handed over
          const int runs = (valid + box - 1) / box;
          if (runs > 0) {
            if (lane == 0) mbar_expect_tx(bar(kFTail), runs * box * (4 * 128));
            __syncwarp();
            if (run >= 0 && run < runs)
              tma_load_5d(dst + run * box * (4 * 128), &maps.values, 0, 0, 4 * rank, group, page, bar(kFTail));
            ++tails;
            wait(bar(kFTail), (uint32_t)((tails - 1) & 1));
            if ((gone = stop())) break;
          }
          for (int x = lane; x < (64 - valid) * 32; x += 32) {  // 16-byte pieces: 8 of a row's 128 bytes, 4 blocks
            const int row = valid + (x >> 5), blk = x >> 3 & 3;
            *reinterpret_cast<uint4*>(smem + kShV + h * kShValuePart + (row >> 3) * 4096 + blk * 1024 + (row & 7) * 128 +
                                      (x & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_release_shared_cluster(full);
        }
      }
    }
    if (gone && lane == 0) pause();
  } else if (warp == kShMmaWarp) {
    // ---- products of the pair, issued by its first CTA: a tile's scores, then the values of the tile before ----
    if (rank == 0) {
      const uint32_t id_s = idesc_bf16(128, kShTile, false, false), id_o = idesc_bf16(128, 256, false, true);
      const uint64_t d_q = smem_desc(sb + kShQ, 16, 1024), d_k = smem_desc(sb + kShK, 16, 3 * 1024);
      const uint64_t d_p = smem_desc(sb + kShP, 16, 1024), d_v = smem_desc(sb + kShV, 1024, 4 * 1024);
      auto ready = [&](int b, int n) {
        wait(bar(b), (uint32_t)(n & 1));
        __syncwarp();
        tc_fence_after();
      };
      // what the second CTA's threads wrote to its shared memory is acquired at cluster scope (42 cycles)
      auto ready_of_both = [&](int b, int n) {
        wait(bar(b), (uint32_t)(n & 1));
        mbar_try_wait_cluster(bar(b), (uint32_t)(n & 1));
        __syncwarp();
        tc_fence_after();
      };
      int n = 0, q = 0;    // tiles whose scores are on the way, pieces
      bool fresh = false;  // the tile before is the first of its piece
      auto values = [&](int m, bool first) {
        ready_of_both(kFP, m);
        const uint32_t more = first ? 0u : 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ready_of_both(kFValues + h, m);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_ss<true>(tmem + 128 * j, d_p + (uint64_t)((h * 8192 + ks * 32) >> 4),
                             d_v + (uint64_t)((h * kShValuePart + ks * 8192 + j * 2048) >> 4), id_o, h + ks > 0 ? 1u : more);
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
                               d_k + (uint64_t)((c * kShKeyPart + b * 1024 + ks * 32) >> 4), id_s, c + b + ks > 0);
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
    float* wmax = reinterpret_cast<float*>(smem + kShMax);
    const int quarter = 2 * side + right;
    const uint32_t p_row = sb + kShP + side * 8192 + r * 128;
    int n = 0;
    SharedTile tile;
    while (it.next()) {
      // this thread's row: its request, the tokens that it sees, whether it sees the shared ones
      tile.start(view, it);
      const int row = it.block * kShRows + 64 * rank + r, rows = it.rows;  // of the group
      int request = -2, seen = 0;
      bool sees = false;
      if (row < rows) {
        request = view.request(it.row + row);
        const int len = view.len(request);
        seen = len - (view.R - 1 - (int)((uint32_t)(it.row + row - request * view.rows_of) / (uint32_t)view.H));
        sees = view.own_from(len, tile.shared) > 0;
      }
      float m = -INFINITY, l = 0.f;
      for (int t = it.t0; t < it.t1; ++t, ++n) {
        if (t > it.t0) tile.advance(view, it, t);
        // how many of the thread's 32 tokens its row sees
        const int in = tile.request < 0 ? (sees ? 32 : 0)
                                        : tile.request == request ? seen - tile.token - 64 * side - 32 * right : 0;
        wait(bar(kFS + (n & 1)), (uint32_t)((n >> 1) & 1));
        __syncwarp();
        tc_fence_after();
        float v[32];
        tc_ld32(tmem + lane_base + 256 + 64 * (n & 1) + 32 * right, v);
        float x = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= p.scale_log2;
        if (in < 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i >= in) v[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) x = fmaxf(x, v[i]);
        // the running maximum moves only when it grows by more than 2^8 (exact: the result is divided by the sum
        // taken with the same maximum), so that O is rarely rescaled
        if (named_bar_or(1, 256, x > m + kShSlack)) {
          wmax[quarter * 64 + r] = x;
          named_bar(1, 256);
          x = fmaxf(fmaxf(wmax[r], wmax[64 + r]), fmaxf(wmax[128 + r], wmax[192 + r]));
          float f = 1.0f;
          if (x > m + kShSlack) {
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
        // (the proxy fence orders the weights before the products' reads in this CTA, the release before the first CTA's
        // thread that issues them; a release of all memory took 1700 to 2700 cycles, with copies in flight)
        if (lane == 0) mbar_release_shared_cluster(lead(kFP));
      }
      // ---- the piece's rows ----
      wmax[quarter * 64 + r] = l;
      named_bar(1, 256);
      const float sum = (wmax[r] + wmax[64 + r]) + (wmax[128 + r] + wmax[192 + r]);
      const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
      const bool whole = it.whole(), there = row < rows;
      const float lse2 = sum == 0.f ? -INFINITY : m + __log2f(sum);
      // the row in q, and of a part: a row's first at its own place, a later one at this share's
      const int64_t at = whole || it.leads ? (int64_t)it.row + row
                                           : (int64_t)p.B * view.rows_of + (int64_t)share * kShRows + 64 * rank + r;
      if (quarter == 0 && there) {
        sp.part_lse[at] = lse2;
        if (whole && p.lse) p.lse[at] = lse2 * 0.6931471805599453f;
      }
      if (it.t0 < it.t1) {
        wait(bar(kFO), (uint32_t)((n - 1) & 1));
        __syncwarp();
        tc_fence_after();
      }
      // A warp turns 32 rows in 2 KB of P's place (its own: the last products have read it) and stores 64 bytes of 8
      // rows at a time; a thread's own row at a time, each store touched 32 lines and the 128 KB took 12000 cycles.
      const uint32_t turn = sb + kShP + warp * 2048;
      const int64_t warp_row = at - r + 32 * (w4 & 1);  // this warp's first row; all of one part are side by side
      const int rows_there = rows - (row - lane);
      const int dims = 256 * side + 128 * right;
      auto turned = [&](const uint32_t (&x)[16], auto store) {  // 64 bytes of a row a lane
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(turn + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)),
                       "r"(x[4 * i]), "r"(x[4 * i + 1]), "r"(x[4 * i + 2]), "r"(x[4 * i + 3])
                       : "memory");
        __syncwarp();
        uint4 y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row_of = 8 * k + (lane >> 2);
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                       : "=r"(y[k].x), "=r"(y[k].y), "=r"(y[k].z), "=r"(y[k].w)
                       : "r"(turn + row_of * 64 + (((lane & 3) ^ (row_of >> 1 & 3)) << 4))
                       : "memory");
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (8 * k + (lane >> 2) < rows_there) store(8 * k + (lane >> 2), y[k]);
        __syncwarp();
      };
      float spoilt = 0.f;  // NaN with an o that is not finite
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        float o[32];
        if (it.t0 < it.t1) {
          tc_ld32(tmem + lane_base + 128 * right + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) spoilt = fmaf(o[i], 0.f, spoilt);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = inv == 0.f ? 0.f : o[i] * inv;
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        uint32_t x[16];
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
          uint16_t* dst = p.out + warp_row * kLat + dims + c + 8 * (lane & 3);
          turned(x, [&](int row_of, const uint4& y) { *reinterpret_cast<uint4*>(dst + row_of * kLat) = y; });
        } else {
          float* dst = sp.part + warp_row * kLat + dims + c + 4 * (lane & 3);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(o[16 * h + i]);
            turned(x, [&](int row_of, const uint4& y) { *reinterpret_cast<uint4*>(dst + 16 * h + row_of * kLat) = y; });
          }
        }
      }
      tc_fence_before();
      named_bar(1, 256);  // wmax is read
      // A row whose weights are finite and whose o is not: rows of another request, with weight 0, were not finite (or its
      // own gave infinities that it did not see).  The join computes it anew.
      if (there && sum > 0.f && spoilt != 0.f) {
        sp.part_lse[at] = __int_as_float(0x7fffffff);
        *s_spoilt = 1;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) sp.spoilt[blockIdx.x] = *s_spoilt;
  cluster_sync();  // nothing of this pair reaches a CTA that has left
  tc_fence_after();
  if (warp == kShMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
}

// A row by its own request's tokens alone, by a warp, 16 dimensions a lane: for rows that what their request does not see
// spoilt, so that no request's rows touch another's result.  (32 requests of 5100 tokens with one such row: 3.8 ms instead
// of 0.05.)
__device__ __forceinline__ void shared_row_alone(const SharedParams& p, int64_t row) {
  const DecodeParams& d = p.d;
  const int lane = threadIdx.x & 31, rows_of = d.R * d.H;
  const int b = (int)(row / rows_of), i = (int)(row - (int64_t)b * rows_of) / d.H;
  const int page = (int)d.page_size, cap = (int)(d.max_pages * d.page_size);
  const int seen = min(max(d.lens[b], 0), cap) - (d.R - 1 - i);
  auto load = [&](const uint16_t* from, uint32_t (&x)[9]) {  // latents 16 lane .., and two of the 64 others
    const uint4 a = reinterpret_cast<const uint4*>(from)[2 * lane], c = reinterpret_cast<const uint4*>(from)[2 * lane + 1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = c.x, x[5] = c.y, x[6] = c.z, x[7] = c.w;
    x[8] = reinterpret_cast<const uint32_t*>(from + kLat)[lane];
  };
  uint32_t q[9];
  load(d.q + row * kLatRow, q);
  float acc[16] = {}, m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int j = 0; j < seen; j += 2) {
    uint32_t x[2][9];
    float v[2], top = m;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = min(j + u, seen - 1), at = t / page, id = d.table[b * d.table_stride + at];
      if (id >= 0 && id < d.num_pages) {
        load(d.cache + id * d.page_stride + (int64_t)(t - at * page) * d.token_stride, x[u]);
      } else {  // (flagged already; reads as zeros)
#pragma unroll
        for (int k = 0; k < 9; ++k) x[u][k] = 0;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      v[u] = 0.f;
#pragma unroll
      for (int k = 0; k < 9; ++k) {
        const float2 a = unpack_bf16(q[k]), c = unpack_bf16(x[u][k]);
        v[u] = fmaf(a.x, c.x, fmaf(a.y, c.y, v[u]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
      v[u] = j + u < seen ? v[u] * d.scale_log2 : -INFINITY;
      top = fmaxf(top, v[u]);
    }
    const float base = top == -INFINITY ? 0.f : top, f = ex2(m - base);
    m = top;
    l *= f;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] *= f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (j + u >= seen) continue;
      const float w = ex2(v[u] - base);
      l += w;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 c = unpack_bf16(x[u][k]);
        acc[2 * k] = fmaf(w, c.x, acc[2 * k]);
        acc[2 * k + 1] = fmaf(w, c.y, acc[2 * k + 1]);
      }
    }
  }
  const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
  uint32_t y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = l == 0.f ? 0 : pack_bf16(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(d.out + row * kLat) + 2 * lane;
  dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
  dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
  if (lane == 0 && d.lse) d.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
}

// The rows of items that several shares hold: out = sum_k w_k o_k, w_k = 2^(lse_k - lse), in the order of the shares.  A
// warp a row, 16 dimensions a lane; parts are in L2.
__global__ void __launch_bounds__(kShJoinThreads, 3) kda_latent_shared_join_kernel(const SharedParams p) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const DecodeParams& d = p.d;
  const int lane = threadIdx.x & 31;
  const SharedHead head = *p.head;
  int spoilt = 0;
  for (int i = lane; i < 2 * p.pairs; i += 32) spoilt |= p.spoilt[i];
  const int64_t all = (int64_t)d.B * d.R * d.H;
  for (int unit = blockIdx.x; unit < head.cut * kShJoinUnits; unit += gridDim.x) {
    const SharedItem item = p.items[unit / kShJoinUnits];
    // its tiles' places on the line, hence the shares that hold them
    const int64_t first = div_costs(item.start + kShItemCost, head.size);
    const int64_t last = item.start + item_cost(max(0, item.tiles - 1));
    const int parts = (int)(div_costs(last, head.size) - first) + 1;
    if (parts == 1) continue;
    const int r = unit % kShJoinUnits * kShJoinRows + (threadIdx.x >> 5), row = item.block * kShRows + r;
    if (row >= item.rows) continue;
    const int64_t at = item.row + row;
    auto place = [&](int k) { return k == 0 ? at : all + (first + k) * kShRows + r; };
    auto piece = [&](int k) { return reinterpret_cast<const float4*>(p.part + place(k) * kLat) + lane; };
    float4 x[2][4];  // the first two parts, on their way while the weights are found
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[k][i] = piece(k)[32 * i];
    float top = -INFINITY;
    for (int k = lane; k < parts; k += 32) top = fmaxf(top, p.part_lse[place(k)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float acc[16], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    auto add = [&](int k, const float4 (&y)[4]) {
      const float w = ex2(p.part_lse[place(k)] - base);
      sum += w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (w != 0.f) {
          acc[4 * i] += w * y[i].x;
          acc[4 * i + 1] += w * y[i].y;
          acc[4 * i + 2] += w * y[i].z;
          acc[4 * i + 3] += w * y[i].w;
        }
      }
    };
    add(0, x[0]);
    add(1, x[1]);
#pragma unroll 2
    for (int k = 2; k < parts; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[0][i] = piece(k)[32 * i];
      add(k, x[0]);
    }
    const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
    uint2* dst = reinterpret_cast<uint2*>(d.out + at * kLat) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dst[32 * i] = make_uint2(pack_bf16(acc[4 * i] * inv, acc[4 * i + 1] * inv),
                               pack_bf16(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv));
    if (lane == 0 && d.lse) d.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
  }
  if (!__any_sync(0xffffffffu, spoilt)) return;
  // (behind the others, by the same warps: asked for as each row is joined, and in a call, it took 2 us more)
  __syncwarp();
#pragma unroll 1
  for (int unit = blockIdx.x; unit < head.items * kShJoinUnits; unit += gridDim.x) {
    const SharedItem item = p.items[unit / kShJoinUnits];
    const int64_t first = div_costs(item.start + kShItemCost, head.size);
    const int64_t last = item.start + item_cost(max(0, item.tiles - 1));
    const int parts = (int)(div_costs(last, head.size) - first) + 1;
    const int r = unit % kShJoinUnits * kShJoinRows + (threadIdx.x >> 5), row = item.block * kShRows + r;
    if (row >= item.rows) continue;
    int found = 0;
    for (int k = lane; k < parts; k += 32)
      found |= isnan(p.part_lse[k == 0 ? (int64_t)item.row + row : all + (first + k) * kShRows + r]);
    if (__any_sync(0xffffffffu, found)) shared_row_alone(p, item.row + row);
  }
}

namespace {

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return sms;
}

// At most one item a group more than the rows fill.
int64_t most_items(const SharedParams& p) { return (int64_t)p.d.B * p.d.R * p.d.H / kShRows + p.groups.G; }

// Sizes and places of a call's workspace; returns its bytes.
size_t shared_layout(SharedParams& p) {
  const size_t rows = (size_t)p.d.B * p.d.R * p.d.H;
  p.pairs = std::max(1, sm_count() / 2);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* x = p.d.ws + at;
    at += (bytes + 255) / 256 * 256;
    return x;
  };
  p.head = reinterpret_cast<SharedHead*>(take(sizeof(SharedHead)));
  p.items = reinterpret_cast<SharedItem*>(take((size_t)most_items(p) * sizeof(SharedItem)));
  p.spoilt = reinterpret_cast<int*>(take((size_t)p.pairs * 8));
  const size_t parts = rows + (size_t)p.pairs * kShRows;
  p.part_lse = reinterpret_cast<float*>(take(parts * 4));
  p.part = reinterpret_cast<float*>(take(parts * kLat * 4));
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
  SharedParams sp = {};
  sp.d = d;
  sp.groups = groups;
  shared_layout(sp);
  DecodeParams& p = sp.d;
  SharedMaps maps;
  memset(&maps, 0, sizeof(maps));
  const int box = (int)std::gcd<int64_t, int64_t>(p.page_size, 64);
  const int64_t rows = (int64_t)p.B * p.R * p.H;
  {  // query rows as [64 values][rows][9 blocks]: one copy brings 64 rows
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, 9};
    const cuuint64_t strides[2] = {kLatRow * 2, 128};
    const cuuint32_t shape[3] = {64, 64, 9};
    if (!encode_map_bf16(&maps.q, p.q, 3, dims, strides, shape)) return false;
  }
  if (p.num_pages == 0) {
    p.max_pages = 0;  // no cache: every length is taken as 0, and nothing is copied
  } else {  // the cache as [64 values][8 tokens][9 blocks][8-token groups of a page][pages]
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
    rc[dev] = cudaFuncSetAttribute(kda_latent_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShSmem);
  });
  if (rc[dev] != cudaSuccess) return false;
  if (!launch_overlapped(kda_latent_shared_kernel, dim3(2 * sp.pairs), kShThreads, kShSmem, s, 2, sp, box, maps)) return false;
  const unsigned ctas = (unsigned)std::min<int64_t>(most_items(sp) * kShJoinUnits, sp.pairs * 2 * kShJoinCtas);
  return launch_overlapped(kda_latent_shared_join_kernel, dim3(ctas), kShJoinThreads, 0, s, 1, sp);
}

}  // namespace kda
