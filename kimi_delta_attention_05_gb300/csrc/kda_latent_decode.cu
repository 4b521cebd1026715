// Absorbed latent attention over the paged cache on the 5th-generation tensor
// cores: split over the cache's length, joined by a second small kernel.
//
// Per query row (token i of a request, head h) with cached rows x_j = [c_j | pe_j]:
//   s_j = scale q . x_j,   o = sum_j softmax(s)_j c_j,   lse = ln sum_j e^{s_j}
// Every row of a request reads the same x_j, and c_j serves as key and value,
// so a cached row crosses HBM once: 1152 bytes against 2 * 1088 flops a query
// row.  Up to about 64 rows that is bound by HBM.
//
// Products, transposed so that the tensor core's fixed 64 / 128 rows are
// cached tokens and value dimensions, and its free width N the query rows
// (16, 32 or 64): few heads then cost few columns instead of empty rows.
//   S^T [64 tokens x N]      = X (64 x 576, K-major)              . Q^T
//   O^T [4 x 128 dims x N]  += C^T (128 x 64, the same tile read MN-major) . P^T
// The tile of 64 cached rows lies in shared memory once, as [8 groups of 8
// tokens][9 blocks of 64 columns][8 tokens][128 bytes] with the 128-byte
// swizzle: pages of any multiple of 8 tokens arrive in whole rows, as one
// copy a run of gcd(page_size, 64) tokens.  Tensor memory:
// O^T 4 N columns, S^T twice N.
//
// Softmax: four warps for each half of the query rows read S^T as 16 x 8
// fragments (a thread holds two tokens of N / 8 rows), reduce the maximum over tokens with shuffles, and write P^T
// as the next product's operand with transposing matrix stores.  The running
// maximum of a row moves only when it grows by more than 2^8 (exact: the
// result is divided by the sum taken with the same maximum), so O^T is rarely
// rescaled; whether any row moves is one reducing barrier.
//
// Work: the tiles of all requests in one line, cut into equal shares, one CTA
// a share; a CTA's share is a few pieces (request, tile range).  A piece that
// is not its whole request writes its normalised rows and their lse in fp32 to
// the workspace, and the join kernel weights them in the order of the tiles,
// so results do not depend on timing.  With more than 64 query rows the CTAs
// form groups, one a block of rows, that walk the same shares at the same
// time, so the cache is read from HBM by one of them and from L2 by the others.
//
// Measured: 256 requests of up to 4096 tokens, 32 rows, 117 us or 5.3 TB/s of cache;
// 8 of up to 131072, 16 rows, 109 us or 5.7 TB/s; 48 of up to 8192, 192 rows in three
// blocks, 140 us or 588 TFLOP/s, where what bounds is the chain of a tile: 2900 cycles
// from its request to its landing, 1400 scores, 1200 softmax, 900 values, with two
// tiles at a time, as shared memory holds no third.  One request of 8192 tokens: 16.3 us,
// latency of set-up, two tiles and the join.
//
// Roles: warps 0-7 softmax and output, warp 8 copies, warp 9 products.
// Every wait is bounded; a CTA that gives up sets the status word.
#include <algorithm>
#include <cstring>
#include <numeric>

#include "../../include/kda_latent.h"
#include "kda_latent.cuh"
#include "kda_latent_tc.cuh"

namespace kda {

constexpr int kDecTile = 64;                     // cached rows of a tile
constexpr int kDecChunks = kLatRow / 64;         // 64-column blocks of a row
constexpr int kDecStages = 2;
constexpr int kDecAtom = 8 * 128;                // 8 tokens of a 64-column block
constexpr int kDecGroup = kDecChunks * kDecAtom; // 8 tokens: 9216 bytes
constexpr int kDecStage = 8 * kDecGroup;         // 73728
constexpr int kDecThreads = 320;
constexpr int kDecCopyWarp = 8, kDecMmaWarp = 9;
// A share's cost: 4 a tile and 6 a request (query block, first wait, output),
// which together are about one and a half tiles' time (2, 4 and 6 measured: 121.2,
// 120.7 and 120.3 us on 256 requests of up to 4096 tokens, 53.4, 52.9 and 50.0 on 203 of up to 1400).
constexpr int kDecTileCost = 4, kDecReqCost = 6;
static_assert(kDecTileCost == 4, "tiles_before shifts by it");
constexpr float kDecSlack = 8.0f;                // log2 growth of a maximum that is let pass

struct DecodeMaps {
  CUtensorMap q, cache;
};

struct DecodePlan {
  int row_blocks;      // groups of CTAs
  int shares;          // CTAs of a group
  int box_rows;        // cached rows of one tensor copy: gcd(page_size, 64)
  int min_tiles;       // least tiles of a share
  int whole;           // requests are not split: the share that holds a request's start has all of it
  float* part;         // [row_blocks * shares * 2][N][512] normalised partial rows
  float* part_lse;     // [row_blocks * shares * 2][N] their lse, log2
  int by_request;      // the join works by request (fewer than shares), else by share
  int4* split;         // [requests or shares][row_blocks]: (request or -1, first share, last share)
};

template <int N>
struct DecCfg {
  static constexpr int kQBufs = N <= 32 ? 2 : 1;
  static constexpr int kQBytes = kDecChunks * N * 128;
  static constexpr int kQ = kDecStages * kDecStage;
  static constexpr int kP = kQ + kQBufs * kQBytes;          // [N][64 tokens] bf16
  static constexpr int kWmax = kP + N * 128;                // fp32 [4][N]: maxima, then sums, of the warps
  static constexpr int kFac = kWmax + 16 * N;               // fp32 [N]
  static constexpr int kBar = kFac + 4 * N;
  // full[2], empty[2], qfull[2], qempty[2], sfull[2], pready, pvdone
  static constexpr int kFull = 0, kEmpty = 2, kQFull = 4, kQEmpty = 6, kSFull = 8, kPReady = 10, kPvDone = 11,
                       kBars = 12;
  static constexpr int kScan = kBar + 8 * kBars;            // int64 [10] sums of the warps, [2] first request and its start
  static constexpr int kTmem = kScan + 96;
  static constexpr int kAbort = kTmem + 8;
  static constexpr int kSmem = kAbort + 8;
  static constexpr uint32_t kCols = N == 16 ? 128 : N == 32 ? 256 : 512;  // 6 N rounded up
  static_assert(kP % 1024 == 0 && kQ % 1024 == 0 && kDecStage % 1024 == 0, "operand images need 1024-byte alignment");
  static_assert(kSmem <= 232448, "exceeds the opt-in shared memory of one CTA");
};

// A request's length, clamped to what its table can hold.
__device__ __forceinline__ int dec_len(const DecodeParams& p, int b) {
  const int64_t len = p.lens[b], cap = p.max_pages * p.page_size;
  return (int)(len < 0 ? 0 : (len > cap ? cap : len));
}
__device__ __forceinline__ int dec_tiles(int len) { return len > 0 ? (len - 1) / kDecTile + 1 : 0; }
__device__ __forceinline__ int64_t dec_cost(int tiles) { return (int64_t)tiles * kDecTileCost + kDecReqCost; }

// a / b of non-negative numbers, in 32 bits where they fit
__device__ __forceinline__ int64_t div_fast(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The pieces of one share [u0, u1) of the line of costs, in order.  Request b
// takes [pre, pre + cost) of it; its tile k starts at pre + kDecReqCost + k
// kDecTileCost and belongs to the share that holds that point; a request
// without tiles, or one that is not split, belongs to the share that holds pre.
struct DecPieces {
  int unsplit;
  int64_t u0, u1, pre;  // the share; start of request b
  int b;
  // the current piece: request, its length, tiles [t0, t1) of its `tiles`
  int req, len, t0, t1, tiles;
  __device__ __forceinline__ int tiles_before(int64_t u) const {
    const int64_t d = u - pre - kDecReqCost;
    return d <= 0 ? 0 : (int)min((int64_t)tiles, (d + kDecTileCost - 1) >> 2);
  }
  __device__ __forceinline__ bool next(const DecodeParams& p) {
    while (b < p.B && pre < u1) {
      req = b;
      len = dec_len(p, b);
      tiles = dec_tiles(len);
      t0 = tiles_before(u0);
      t1 = tiles_before(u1);
      if (unsplit && pre >= u0) t1 = tiles;  // (and t0 is 0)
      const bool mine = tiles > 0 && !unsplit ? t0 < t1 : pre >= u0;
      pre += dec_cost(tiles);
      ++b;
      if (mine) return true;
    }
    return false;
  }
  __device__ __forceinline__ int count() const { return t1 - t0; }
  __device__ __forceinline__ bool whole() const { return t1 - t0 == tiles; }
};

// A walk over the tiles of a share.
struct DecCursor {
  DecPieces it;
  int tile;
  int piece;  // index of the piece among those with tiles
  bool ok;
  __device__ __forceinline__ void start(const DecPieces& s, const DecodeParams& p) {
    it = s;
    piece = -1;
    ok = true;
    piece_with_tiles(p);
  }
  __device__ __forceinline__ void piece_with_tiles(const DecodeParams& p) {
    do {
      ok = it.next(p);
    } while (ok && it.count() == 0);
    tile = it.t0;
    ++piece;
  }
  __device__ __forceinline__ void advance(const DecodeParams& p) {
    if (++tile >= it.t1) piece_with_tiles(p);
  }
  __device__ __forceinline__ bool first() const { return tile == it.t0; }
  __device__ __forceinline__ bool last() const { return tile + 1 == it.t1; }
};

template <int N>
__global__ void __launch_bounds__(kDecThreads, 1)
    kda_latent_decode_kernel(const DecodeParams p, const DecodePlan pl, const __grid_constant__ DecodeMaps maps) {
  using C = DecCfg<N>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rblk = blockIdx.x % pl.row_blocks, share = blockIdx.x / pl.row_blocks;
  const int rows = p.R * p.H, row0 = rblk * N;
  const uint32_t sb = smem_u32(smem);
  const uint32_t bars = sb + C::kBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kAbort);
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + C::kScan);

  // ---- set-up: barriers, tensor memory, this CTA's share of the tiles ----
  // (by the last warps: the first ones fetch the lengths meanwhile)
  if (warp == kDecCopyWarp && lane == 0) {
    for (int i = 0; i < C::kBars; ++i) mbar_init(bar(i), i == C::kPReady ? 8 : 1);
    *s_abort = (sb & 1023) ? 1 : 0;
    s_scan[10] = 0;
    s_scan[11] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kDecMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sb + C::kTmem),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  if (warp == kDecCopyWarp && lane == 0) {
    prefetch_map(&maps.q);
    prefetch_map(&maps.cache);
  }
  // (set up while the kernel before this one ends; nothing it wrote is read until here)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  // each thread sums a run of requests; a scan over threads gives the total
  // (hence the shares' size) and the run that holds this share's first tile
  const int run = (p.B + kDecThreads - 1) / kDecThreads;
  const int b0 = min(p.B, tid * run), b1 = min(p.B, b0 + run);
  int64_t mine = 0;
  bool odd = false;
  for (int b = b0; b < b1; ++b) {
    const int raw = p.lens[b], len = dec_len(p, b);
    odd |= raw != len;
    mine += dec_cost(dec_tiles(len));
  }
  if (odd && blockIdx.x == 0) atomicExch(p.status, KDA_ERR_BAD_LENGTHS);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kDecThreads / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int64_t size = max((int64_t)pl.min_tiles * kDecTileCost, div_fast(total + pl.shares - 1, pl.shares));
  const int64_t u0 = min(total, share * size), u1 = min(total, u0 + size);
  before += incl - mine;
  if (u0 < u1 && u0 >= before && u0 < before + mine) {
    int64_t pre = before;
    for (int b = b0; b < b1; ++b) {
      const int64_t t = dec_cost(dec_tiles(dec_len(p, b)));
      if (u0 < pre + t) {
        s_scan[10] = b;
        s_scan[11] = pre;
        break;
      }
      pre += t;
    }
  }
  __syncthreads();
  DecPieces pieces;
  pieces.unsplit = pl.whole;
  pieces.u0 = u0;
  pieces.u1 = u1;
  pieces.b = u0 < u1 ? (int)s_scan[10] : p.B;
  pieces.pre = s_scan[11];
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::kTmem);
  if (*s_abort && tid == 0) atomicExch(p.status, KDA_ERR_DEVICE_TIMEOUT);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  auto wait = [&](uint32_t b, uint32_t parity) {
    if (mbar_try_wait(b, parity) || *s_abort) return;
    if (!mbar_wait_bounded(b, parity)) {
      atomicExch(p.status, KDA_ERR_DEVICE_TIMEOUT);
      *s_abort = 1;
    }
  };

  if (warp == kDecCopyWarp) {
    // ---- copies: the tiles of the share into the stages, the query rows of each piece ----
    const int box = pl.box_rows;
    DecCursor c;
    c.start(pieces, p);
    int it = 0, qi = 0;  // tiles and query blocks issued
    bool gone = false;
    while (c.ok && !gone) {
      const int s = it & 1;
      const int valid = min(kDecTile, c.it.len - c.tile * kDecTile);
      const int segs = (valid + box - 1) / box;
      // page of this lane's run of box rows (lanes below segs), fetched before the wait
      int page = 0, off = 0;
      if (lane < segs) {
        const uint32_t j = (uint32_t)(c.tile * kDecTile + lane * box), in_table = j / (uint32_t)p.page_size;
        page = p.table[c.it.req * p.table_stride + in_table];
        off = (int)(j - in_table * (uint32_t)p.page_size);
        if (page < 0 || page >= p.num_pages) {
          atomicExch(p.status, KDA_ERR_BAD_PAGE);
          page = (int)p.num_pages;  // past the map: reads as zeros
        }
      }
      const uint32_t dst = sb + s * kDecStage, full = bar(C::kFull + s);
      if (it >= kDecStages) wait(bar(C::kEmpty + s), (uint32_t)(((it >> 1) & 1) ^ 1));
      __syncwarp();
      gone = __any_sync(0xffffffffu, *s_abort != 0);
      if (gone) break;
      if (lane == 0) mbar_expect_tx(full, (uint32_t)(segs * box * (kDecGroup / 8)));
      __syncwarp();
      if (lane < segs)
        tma_load_5d(dst + lane * box * (kDecGroup / 8), &maps.cache, 0, 0, 0, off >> 3, page, full);
      if (c.first()) {
        const int qb = qi % C::kQBufs;
        if (qi >= C::kQBufs) wait(bar(C::kQEmpty + qb), (uint32_t)(((qi / C::kQBufs) & 1) ^ 1));
        __syncwarp();
        gone = __any_sync(0xffffffffu, *s_abort != 0);
        if (!gone && lane == 0) {
          mbar_expect_tx(bar(C::kQFull + qb), C::kQBytes);
          tma_load_4d(sb + C::kQ + qb * C::kQBytes, &maps.q, 0, row0, 0, c.it.req, bar(C::kQFull + qb));
        }
        if (!gone) ++qi;
      }
      ++it;  // (also where the query block was given up: the tile's copies are in flight)
      c.advance(p);
    }
    // After a timeout: let the copies still in flight land before leaving.
    if (gone && lane == 0) {
      for (int t = max(0, it - kDecStages); t < it; ++t)
        mbar_wait_bounded(bar(C::kFull + (t & 1)), (uint32_t)((t >> 1) & 1));
      for (int t = max(0, qi - C::kQBufs); t < qi; ++t)
        mbar_wait_bounded(bar(C::kQFull + t % C::kQBufs), (uint32_t)((t / C::kQBufs) & 1));
    }
  } else if (warp == kDecMmaWarp) {
    // ---- products ----
    const uint32_t id_s = idesc_bf16(64, N, false, false), id_o = idesc_bf16(128, N, true, false);
    const uint64_t d_x = smem_desc(sb, 16, kDecGroup), d_c = smem_desc(sb, kDecAtom, kDecGroup);
    const uint64_t d_q = smem_desc(sb + C::kQ, 16, 1024), d_p = smem_desc(sb + C::kP, 16, 1024);
    const uint32_t t_s = tmem + 4 * N;
    DecCursor cs, co;
    cs.start(pieces, p);
    co = cs;
    int is = 0, io = 0;  // tiles of the scores and of the values
    // One place each for the two products (a second copy of the unrolled issue
    // loops costs microseconds of instruction fetches on a cold start), written
    // out in full (with a block index of run time the operands leave the uniform
    // registers and an issue costs 120 cycles instead of 35).  The next tile's
    // scores go first if it has landed, so that the softmax of one tile overlaps
    // the products of the other; else they follow this tile's values.  Barriers
    // are read as seldom as possible: while the tensor core streams its operands
    // a shared-memory access takes some 250 cycles.
    for (;;) {
      bool go = cs.ok && is == io;
      if (cs.ok && is == io + 1)
        go = __all_sync(0xffffffffu, mbar_test(bar(C::kFull + (is & 1)), (uint32_t)((is >> 1) & 1)));
      if (go) {  // S^T of tile `is` into its half of the score columns
        const int s = is & 1, qb = cs.piece % C::kQBufs;
        const uint64_t a = d_x + (uint64_t)((s * kDecStage) >> 4), b = d_q + (uint64_t)((qb * C::kQBytes) >> 4);
        if (cs.first()) wait(bar(C::kQFull + qb), (uint32_t)((cs.piece / C::kQBufs) & 1));
        wait(bar(C::kFull + s), (uint32_t)((is >> 1) & 1));
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ch = 0; ch < kDecChunks; ++ch)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss<false>(t_s + N * s, a + (uint64_t)((ch * kDecAtom + ks * 32) >> 4),
                            b + (uint64_t)((ch * N * 128 + ks * 32) >> 4), id_s, ch + ks > 0);
          mma_commit<false>(bar(C::kSFull + s));
          if (cs.last()) mma_commit<false>(bar(C::kQEmpty + qb));
        }
        __syncwarp();
        ++is;
        cs.advance(p);
        continue;
      }
      if (!co.ok) break;
      // O^T += C^T P^T of tile `io`
      const int s = io & 1;
      wait(bar(C::kPReady), (uint32_t)(io & 1));
      const int valid = min(kDecTile, co.it.len - co.tile * kDecTile);
      if (valid < kDecTile) {
        // what lies behind the length takes part in the product with weight 0: it has to be finite
        for (int t = valid; t < kDecTile; ++t)
          for (int i = lane; i < kLat / 8; i += 32)
            *reinterpret_cast<uint4*>(smem + s * kDecStage + (t >> 3) * kDecGroup + (i >> 3) * kDecAtom + (t & 7) * 128 +
                                      (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      tc_fence_after();
      const uint64_t a = d_c + (uint64_t)((s * kDecStage) >> 4);
      const uint32_t start = co.first() ? 0u : 1u;
      if (elect_one()) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss<false>(tmem + mt * N, a + (uint64_t)((mt * 2 * kDecAtom + ks * 2 * kDecGroup) >> 4),
                          d_p + (uint64_t)((ks * 32) >> 4), id_o, ks > 0 ? 1u : start);
        mma_commit<false>(bar(C::kEmpty + s));
        mma_commit<false>(bar(C::kPvDone));
      }
      __syncwarp();
      ++io;
      co.advance(p);
    }
    if (io > 0) mbar_wait_bounded(bar(C::kPvDone), (uint32_t)((io - 1) & 1));  // before tensor memory is freed
  } else {
    // ---- softmax and output: warps 0-3 the first half of the query rows, 4-7 the
    //      second; warp w of the four holds tokens 16 w .. 16 w + 15 of a tile, then value
    //      dimensions 32 w .. of each 128 ----
    constexpr int kH = N / 2;   // query rows of this half
    constexpr int kV = kH / 2;  // scores of a thread: 8-column group g, v[4 g + 2 r + e] = row 8 g + 2 (lane % 4) + e
    constexpr int kM = kH / 4;  //   of token lane / 4 + 8 r; maxima and sums m[2 g + e]
    const int half = warp >> 2, w4 = warp & 3, h0 = half * kH, bar_id = 1 + half;
    float* wmax = reinterpret_cast<float*>(smem + C::kWmax) + h0;
    float* fac = reinterpret_cast<float*>(smem + C::kFac) + h0;
    const uint32_t lane_base = ((uint32_t)(w4 * 32) << 16) + h0;
    const int tok = 16 * w4 + (lane >> 2);
    const int c0 = 2 * (lane & 3);
    // this lane's address for the transposing stores: matrix lane / 8, row lane % 8
    const int st_head = h0 + 8 * (lane >> 4) + (lane & 7), st_chunk = 2 * w4 + ((lane >> 3) & 1);
    const uint32_t st_addr = sb + C::kP + st_head * 128 + ((st_chunk ^ (lane & 7)) << 4);
    int it = 0;
    while (pieces.next(p)) {
      const int nt = pieces.count();
      const bool whole = pieces.whole();
      float m[kM], l[kM];
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
      }
      for (int tile = pieces.t0; tile < pieces.t0 + nt; ++tile, ++it) {
        const int s = it & 1;
        wait(bar(C::kSFull + s), (uint32_t)((it >> 1) & 1));
        __syncwarp();
        tc_fence_after();
        float v[kV];
        tc_ld16x256(tmem + lane_base + 4 * N + N * s, v);
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] *= p.scale_log2;
        const int j = tile * kDecTile + tok;
        if ((tile + 1) * kDecTile > pieces.len - (p.R - 1)) {
          // the last tiles: row (token i, head) sees j < len - (R - 1 - i)
#pragma unroll
          for (int i = 0; i < kM; ++i) {
            const int row = row0 + h0 + 8 * (i >> 1) + c0 + (i & 1);
            const int seen = pieces.len - max(0, p.R - 1 - row / p.H);
            if (j >= seen) v[4 * (i >> 1) + (i & 1)] = -INFINITY;
            if (j + 8 >= seen) v[4 * (i >> 1) + 2 + (i & 1)] = -INFINITY;
          }
        }
        float mx[kM];
        bool grow = false;
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          float x = fmaxf(v[4 * (i >> 1) + (i & 1)], v[4 * (i >> 1) + 2 + (i & 1)]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mx[i] = x;
          grow |= x > m[i] + kDecSlack;
        }
        const bool first = tile == pieces.t0;
        if (named_bar_or(bar_id, 128, grow)) {
          if (lane < 4) {
#pragma unroll
            for (int i = 0; i < kM; ++i) wmax[w4 * N + 8 * (i >> 1) + c0 + (i & 1)] = mx[i];
          }
          named_bar(bar_id, 128);
          float f[kM];
#pragma unroll
          for (int i = 0; i < kM; ++i) {
            const int c = 8 * (i >> 1) + c0 + (i & 1);
            const float x = fmaxf(fmaxf(wmax[c], wmax[N + c]), fmaxf(wmax[2 * N + c], wmax[3 * N + c]));
            f[i] = 1.0f;
            if (x > m[i] + kDecSlack) {
              f[i] = ex2(m[i] - x);
              m[i] = x;
              l[i] *= f[i];
            }
          }
          if (!first) {  // O^T of the tiles so far to the new maxima
            if (w4 == 0 && lane < 4) {
#pragma unroll
              for (int i = 0; i < kM; ++i) fac[8 * (i >> 1) + c0 + (i & 1)] = f[i];
            }
            wait(bar(C::kPvDone), (uint32_t)((it - 1) & 1));
            named_bar(bar_id, 128);
            tc_fence_after();
#pragma unroll 1
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
              for (int r = 0; r < kH; r += 8) {
                float o[8];
                tc_ld8_nowait(tmem + lane_base + mt * N + r, o);
                tc_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] *= fac[r + i];
                tc_st8(tmem + lane_base + mt * N + r, o);
              }
            }
            tc_st_wait();
          }
        }
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          const float base = m[i] == -INFINITY ? 0.f : m[i];
          float& x = v[4 * (i >> 1) + (i & 1)];
          float& y = v[4 * (i >> 1) + 2 + (i & 1)];
          x = ex2(x - base);
          y = ex2(y - base);
          l[i] += x + y;
        }
        if (it > 0) wait(bar(C::kPvDone), (uint32_t)((it - 1) & 1));  // P^T of the tile before is read
        __syncwarp();
        // weights rounded to bf16, the operands' type; the sums are taken before it (256 requests of up
        // to 4096 tokens: relative RMS against 64 bits 0.0021, of which 0.0017 are the output's rounding)
        if constexpr (kH == 8) {
          stsm_x2_t(st_addr, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
#pragma unroll
          for (int g = 0; g < kH / 8; g += 2)
            stsm_x4_t(st_addr + g * 1024, pack_bf16(v[4 * g], v[4 * g + 1]), pack_bf16(v[4 * g + 2], v[4 * g + 3]),
                      pack_bf16(v[4 * g + 4], v[4 * g + 5]), pack_bf16(v[4 * g + 6], v[4 * g + 7]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kPReady));
      }
      // ---- the piece's rows ----
      named_bar(bar_id, 128);  // wmax and fac of the last tile are read
#pragma unroll
      for (int i = 0; i < kM; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
        if (lane < 4) wmax[w4 * N + 8 * (i >> 1) + c0 + (i & 1)] = l[i];
      }
      named_bar(bar_id, 128);
      const int slot = 2 * blockIdx.x + (pieces.t0 > 0 ? 0 : 1);
      if (w4 == 0 && lane < 4) {
#pragma unroll
        for (int i = 0; i < kM; ++i) {
          const int c = 8 * (i >> 1) + c0 + (i & 1);
          const float sum = (wmax[c] + wmax[N + c]) + (wmax[2 * N + c] + wmax[3 * N + c]);
          fac[c] = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
          const float lse2 = sum == 0.f ? -INFINITY : m[i] + __log2f(sum);
          if (!whole) {
            pl.part_lse[(int64_t)slot * N + h0 + c] = lse2;
          } else if (p.lse && row0 + h0 + c < rows) {
            p.lse[(int64_t)pieces.req * rows + row0 + h0 + c] = lse2 * 0.6931471805599453f;
          }
        }
      }
      if (nt > 0) {
        wait(bar(C::kPvDone), (uint32_t)((it - 1) & 1));
        __syncwarp();
      }
      named_bar(bar_id, 128);
      tc_fence_after();
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        const int dim = mt * 128 + w4 * 32;  // this warp's 32 dimensions of the block of 128
        float o[kH];
        if (nt > 0) {
#pragma unroll
          for (int r = 0; r < kH; r += 8) tc_ld8_nowait(tmem + lane_base + mt * N + r, o + r);
          tc_ld_wait();
        } else {
#pragma unroll
          for (int r = 0; r < kH; ++r) o[r] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < kH; r += 4) {
          const float4 f = *reinterpret_cast<const float4*>(fac + r);
          o[r] = f.x == 0.f ? 0.f : o[r] * f.x;
          o[r + 1] = f.y == 0.f ? 0.f : o[r + 1] * f.y;
          o[r + 2] = f.z == 0.f ? 0.f : o[r + 2] * f.z;
          o[r + 3] = f.w == 0.f ? 0.f : o[r + 3] * f.w;
        }
        const int left = rows - row0 - h0;  // query rows there are from this half's first
        if (!whole) {
          float* dst = pl.part + ((int64_t)slot * N + h0) * kLat + dim + lane;
#pragma unroll
          for (int r = 0; r < kH; ++r)
            if (r < left) dst[r * kLat] = o[r];
        } else {
          // two rows at a time: even lanes store two dimensions of the first, odd lanes of the second
          uint16_t* dst = p.out + ((int64_t)pieces.req * rows + row0 + h0) * kLat + dim + (lane & ~1);
#pragma unroll
          for (int r = 0; r < kH; r += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? o[r] : o[r + 1], 1);
            const uint32_t w = (lane & 1) ? pack_bf16(other, o[r + 1]) : pack_bf16(o[r], other);
            const int at = r + (lane & 1);
            if (at < left) *reinterpret_cast<uint32_t*>(dst + at * kLat) = w;
          }
        }
      }
      named_bar(bar_id, 128);  // fac is read
    }
    tc_fence_before();
  }
  if (tid == 0 && !pl.whole) {
    // what the join kernel has to do, by request or by the share a request starts in
    if (!pl.by_request) pl.split[blockIdx.x] = make_int4(-1, 0, 0, 0);
    DecPieces each = pieces;
    each.b = u0 < u1 ? (int)s_scan[10] : p.B;
    each.pre = s_scan[11];
    while (each.next(p)) {
      if (each.t0 > 0) continue;
      // (the request's last tile starts kDecTileCost before the next request)
      const int4 info = each.whole() ? make_int4(-1, 0, 0, 0)
                                     : make_int4(each.req, share, (int)div_fast(each.pre - kDecTileCost, size), 0);
      if (pl.by_request) pl.split[each.req * pl.row_blocks + rblk] = info;
      else if (!each.whole()) pl.split[blockIdx.x] = info;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kDecMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(C::kCols));
}

// Joins the parts of a request that several shares hold: out = sum_k w_k o_k,
// w_k = 2^(lse_k - lse), in the shares' order.  kWide: a CTA a row, four groups
// of 128 threads (4 dimensions each) over quarters of the parts, for few
// requests in many parts; else a warp a row (16 dimensions a lane).  Bound by
// latency, as the parts are in L2: about 4 us behind the main kernel.
template <bool kWide>
__global__ void __launch_bounds__(512) kda_latent_join_kernel(const DecodeParams p, const DecodePlan pl, int n) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int4 info = pl.split[blockIdx.x];
  if (info.x < 0) return;
  const int tid = threadIdx.x, lane = tid & 31, rblk = blockIdx.x % pl.row_blocks, first = info.y;
  const int r = kWide ? blockIdx.y : blockIdx.y * 16 + (tid >> 5);  // row of the block of n
  const int rows = p.R * p.H, row = rblk * n + r;
  if (r >= n || row >= rows) return;  // (kWide: the whole CTA)
  const int parts = info.z - first + 1;
  const int64_t at = (int64_t)info.x * rows + row;
  auto slot = [&](int k) {  // the first part is its share's second slot, the others their shares' first
    return (int64_t)(2 * ((first + k) * pl.row_blocks + rblk) + (k == 0 ? 1 : 0)) * n + r;
  };
  // every warp takes the maximum over all parts for itself
  float top = -INFINITY;
  for (int k = lane; k < parts; k += 32) top = fmaxf(top, pl.part_lse[slot(k)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = top == -INFINITY ? 0.f : top;
  if constexpr (kWide) {
    __shared__ float part[4][kLat];
    __shared__ float wts[4];
    const int quarter = tid >> 7, t = tid & 127;
    const int k0 = parts * quarter / 4, k1 = parts * (quarter + 1) / 4;
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll 8
    for (int k = k0; k < k1; ++k) {
      const int64_t from = slot(k);
      const float w = ex2(pl.part_lse[from] - base);
      const float4 x = reinterpret_cast<const float4*>(pl.part + from * kLat)[t];
      sum += w;
      if (w != 0.f) {
        acc[0] += w * x.x;
        acc[1] += w * x.y;
        acc[2] += w * x.z;
        acc[3] += w * x.w;
      }
    }
    reinterpret_cast<float4*>(part[quarter])[t] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (t == 0) wts[quarter] = sum;
    __syncthreads();
    const float total = (wts[0] + wts[1]) + (wts[2] + wts[3]);
    const float inv = total > 0.f ? 1.0f / total : (total == 0.f ? 0.f : total);
    const float o = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    reinterpret_cast<__nv_bfloat16*>(p.out)[at * kLat + tid] = __float2bfloat16_rn(o * inv);
    if (tid == 0 && p.lse) p.lse[at] = total == 0.f ? -INFINITY : (top + __log2f(total)) * 0.6931471805599453f;
  } else {
    float acc[16], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 2
    for (int k = 0; k < parts; ++k) {
      const int64_t from = slot(k);
      const float w = ex2(pl.part_lse[from] - base);
      const float4* src = reinterpret_cast<const float4*>(pl.part + from * kLat) + lane;
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
    uint2* dst = reinterpret_cast<uint2*>(p.out + at * kLat) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      dst[32 * i] = make_uint2(pack_bf16(acc[4 * i] * inv, acc[4 * i + 1] * inv),
                               pack_bf16(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv));
    if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
  }
}

namespace {

int device_sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return sms;
}

// Columns of the products: the query rows of a request rounded up to 16, 32 or
// 64; blocks of 64 beyond that.
int dec_width(const DecodeParams& p) {
  const int rows = p.R * p.H;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

struct DecLayout {
  DecodePlan plan;
  int n, joins;
  size_t lse_at, split_at, bytes;
};

DecLayout dec_layout(const DecodeParams& p) {
  DecLayout d;
  memset(&d, 0, sizeof(d));
  d.n = dec_width(p);
  const int sms = std::max(1, device_sm_count());
  const int rows = p.R * p.H;
  d.plan.row_blocks = (rows + d.n - 1) / d.n;
  const int64_t most = (int64_t)p.B * ((p.max_pages * p.page_size + kDecTile - 1) / kDecTile + 1);
  d.plan.min_tiles = 2;
  // Tables of up to four tiles: a split and its join cost more than they save (one
  // request of 256 tokens and 32 rows: 12.4 us split, 11.3 whole; 256 such: 30.4 and 26.3).
  d.plan.whole = p.max_pages * p.page_size <= 4 * kDecTile;
  const int64_t units = d.plan.whole ? p.B : (most + d.plan.min_tiles - 1) / d.plan.min_tiles;
  d.plan.shares = (int)std::max<int64_t>(1, std::min<int64_t>(sms / d.plan.row_blocks, units));
  d.plan.box_rows = (int)std::gcd<int64_t, int64_t>(p.page_size, kDecTile);
  if (d.plan.whole) return d;  // no parts: no workspace
  const size_t ctas = (size_t)d.plan.row_blocks * d.plan.shares;
  d.lse_at = ctas * 2 * d.n * kLat * 4;
  d.split_at = d.lse_at + ctas * 2 * d.n * 4;
  d.plan.by_request = p.B <= d.plan.shares;
  d.joins = (int)(std::min<int64_t>(p.B, d.plan.shares) * d.plan.row_blocks);
  d.bytes = (d.split_at + (size_t)d.joins * sizeof(int4) + 255) / 256 * 256;
  return d;
}

template <int N>
bool launch_dec(const DecodeParams& p, const DecLayout& d, const DecodeMaps& maps, cudaStream_t s) {
  const unsigned ctas = (unsigned)(d.plan.row_blocks * d.plan.shares);
  static std::once_flag once[64];
  static cudaError_t rc[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::call_once(once[dev], [&] {
    rc[dev] = cudaFuncSetAttribute(kda_latent_decode_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   DecCfg<N>::kSmem);
  });
  if (rc[dev] != cudaSuccess) return false;
  if (!launch_overlapped(kda_latent_decode_kernel<N>, dim3(ctas), kDecThreads, DecCfg<N>::kSmem, s, 1, p, d.plan, maps))
    return false;
  if (d.plan.whole) return true;  // nothing to join
  // a row a CTA where a request is in more than four parts on average, else a row a warp
  const bool wide = (int64_t)p.B * 4 < d.plan.shares;
  const int most = std::min(N, p.R * p.H);
  const dim3 grid((unsigned)d.joins, (unsigned)(wide ? most : (most + 15) / 16));
  return launch_overlapped(wide ? kda_latent_join_kernel<true> : kda_latent_join_kernel<false>, grid, 512, 0, s, 1, p,
                           d.plan, N);
}

}  // namespace

size_t decode_workspace_bytes(const DecodeParams& p) { return dec_layout(p).bytes; }

bool launch_latent_decode(const DecodeParams& args, cudaStream_t s) {
  DecodeParams p = args;
  DecLayout d = dec_layout(p);
  d.plan.part = reinterpret_cast<float*>(p.ws);
  d.plan.part_lse = reinterpret_cast<float*>(p.ws + d.lse_at);
  d.plan.split = reinterpret_cast<int4*>(p.ws + d.split_at);
  DecodeMaps maps;
  memset(&maps, 0, sizeof(maps));
  const int rows = p.R * p.H;
  {  // query rows [B][rows][576] as [64 values][rows][9 blocks][B]: one copy brings N rows of a request
    const cuuint64_t dims[4] = {64, (cuuint64_t)rows, (cuuint64_t)kDecChunks, (cuuint64_t)p.B};
    const cuuint64_t strides[3] = {kLatRow * 2, 128, (cuuint64_t)rows * kLatRow * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)d.n, (cuuint32_t)kDecChunks, 1};
    if (!encode_map_bf16(&maps.q, p.q, 4, dims, strides, box)) return false;
  }
  if (p.num_pages == 0) {
    p.max_pages = 0;  // no cache: every length is taken as 0, and nothing is copied
  } else {  // the cache as [64 values][8 tokens][9 blocks][8-token groups of a page][pages]
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)kDecChunks, (cuuint64_t)p.page_size / 8, (cuuint64_t)p.num_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)p.token_stride * 2, 128, (cuuint64_t)p.token_stride * 16,
                                   (cuuint64_t)p.page_stride * 2};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)kDecChunks, (cuuint32_t)d.plan.box_rows / 8, 1};
    if (!encode_map_bf16(&maps.cache, p.cache, 5, dims, strides, box)) return false;
  }
  switch (d.n) {
    case 16: return launch_dec<16>(p, d, maps, s);
    case 32: return launch_dec<32>(p, d, maps, s);
    default: return launch_dec<64>(p, d, maps, s);
  }
}

}  // namespace kda
