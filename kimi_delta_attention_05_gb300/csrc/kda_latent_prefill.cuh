// Expanded latent attention on the 5th-generation tensor cores: persistent
// CTAs walk (block of 256 query rows, head) items, two 128-row tiles in turn.
//
//   s_ij = scale (q_i . [k_j | pe_j]),  o_i = sum_j softmax(s_i)_j v_j
// over the keys a row sees (causal: j <= i + Lk - Lq).  The 64 shared key
// channels are loaded from k_pe for every head; nothing is expanded in memory.
//
// Per tile of 128 keys and each of the two query tiles:
//   S [128 x 128]  = Q (128 x 192, shared memory) . [K | pe]^T
//   O [128 x 128] += P (128 x 128, bf16 in tensor memory, over S) . V
// 2 (192 + 128) flops a (row, key) pair: bound by the tensor cores, so the aim
// is that they never wait.  While one tile's softmax runs, the other tile's
// products do: the issue order is S0(i), O1(i-1), S1(i), O0(i).  A thread owns
// a row of S (32x32b loads), so row maximum and sum need no exchange; the
// running maximum moves only when it grows by more than 2^8 (exact: the result
// is divided by the sum taken with the same maximum), so O is rarely rescaled.
//
// Shared memory: Q 96 KB, and a ring of eight 16 KB slots ([128 keys][64
// channels], 128-byte swizzle) that takes a tile's three key blocks and two
// value blocks in the order they are used and is refilled as soon as their
// products are done.  Keys and values of a tile have one barrier each: while
// the tensor core streams its operands a shared-memory access takes some 150
// to 300 cycles, and the issuing warp has about 400 cycles of queued products
// to spend on waits (one barrier a slot: 528 us on the 8192-token prompt, 454
// with one for the keys and one for the values).  The first key block has its
// own, as its slot is free a product earlier than the others'.  Tensor memory: S0, S1,
// O0, O1, 128 columns each.
//
// What bounds this is shared memory: each 128 x 128 x 16 product of S reads 8 KB
// of operands, about 78 cycles of its bandwidth against 64 of arithmetic.  So
// long sequences go to the paired form: two CTAs on neighbouring SMs share one
// product of 256 rows (cta_group::2), each holds its own 128 query rows of a
// tile and half of every key and value tile, and an operand of 6 KB is read in
// its place; loads from L2 halve too.  Items are then 512 rows, whose causal
// edge wastes more, so short sequences keep single CTAs.
//
// Measured, passes back to back in a graph: one prompt of 8192 tokens, 32 heads, in pairs:
// 361 to 377 us by board and power, 1.82 to 1.90 PFLOP/s (0.95 to 0.99 of cuBLAS's burst
// rate), tensor cores active 86% of the time; called on new inputs each time 420 us, 1.63
// PFLOP/s (0.85 of that rate, 0.95 of cuBLAS's sustained one).  Two pieces of 1024 behind
// 15360 cached, 16 heads: 186 to 194 us, 93% active on the 128 SMs of 152 that have an item;
// 24 packed sequences of up to 2048, 16 heads, in single CTAs: 161 to 190 us by process, 59%
// active: an item of 11 tiles pays about 8000 cycles for its first loads and its output.
//
// Roles: warps 0-3 and 4-7 softmax and output of the two tiles, warp 8 copies,
// warp 9 products (of the pair: in its first CTA), warp 10 the list of items, one
// more only fills its warpgroup.  Every wait is bounded; a CTA that gives up sets the status word.
#pragma once

#include <algorithm>
#include <cstring>

#include "../../include/kda_latent.h"
#include "kda_latent.cuh"
#include "kda_latent_tc.cuh"

namespace kda {

constexpr int kPreRows = 128;                    // query rows of a tile in one CTA
constexpr int kPreQ = 0;                         // two tiles of three [128 rows][64 channels] blocks
constexpr int kPreQTile = 3 * kPreRows * 128;
constexpr int kPreRing = 2 * kPreQTile;          // key and value blocks
constexpr int kPreThreads = 384;
// Registers: 168 a thread at launch; the warpgroup of copies and products gives
// up 64 of its share, the two of the softmax take 32 each (a row of scores and
// its weights in registers): 128 (104 + 2 x 200) = 384 x 168.
constexpr int kPreRegsFew = 104, kPreRegsMany = 200;
static_assert(128 * (kPreRegsFew + 2 * kPreRegsMany) == kPreThreads * 168, "register split");
// Keys of a tile whose weights a pair hands over first: its round from scores to
// values is the longer one, and the products of these keys start meanwhile (none,
// 64 and 96 of the 128 measured: 391, 380 and 395 us on the 8192-token prompt;
// single CTAs gain nothing).
constexpr int kPreFirst = 64;
constexpr float kPreSlack = 8.0f;                // log2 growth of a maximum that is let pass
// single CTAs: ring of [128 keys][64 channels] slots
constexpr int kPreSlots = 8;
constexpr int kPreSlot = kPreKeys * 128;
// pairs: stages of this CTA's 64 keys (three blocks) and its 64 value channels of 128 keys
constexpr int kPairStages = 3;
constexpr int kPairK = 64 * 128;                 // a key block
constexpr int kPairStage = 3 * kPairK + kPreSlot;
constexpr int kPreBar = kPreRing + (kPreSlots * kPreSlot > kPairStages * kPairStage ? kPreSlots * kPreSlot
                                                                                    : kPairStages * kPairStage);
// full and empty of a tile's first key block, other key blocks and value blocks
// (by the tile's parity), q full and empty, sfull[2], pready[2], pvdone[2]
constexpr int kPbFullK0 = 0, kPbFullK = 2, kPbFullV = 4, kPbEmptyK = 6, kPbEmptyV = 8, kPbQ = 10, kPbQEmpty = 11,
              kPbS = 12, kPbP = 14, kPbPv = 16;
// pairs: by stage; then a barrier for value tiles that end behind the sequence, and for the other weights
constexpr int kPpFullK = 18, kPpFullV = 21, kPpEmptyK = 24, kPpEmptyV = 27, kPpTail = 30, kPbP2 = 31;
// the next item: written, and read by every role
constexpr int kPbItem = 33, kPbItemRead = 34, kPbars = 35;
constexpr int kPreItem = (kPreBar + 8 * kPbars + 15) / 16 * 16;
constexpr int kPreTmem = kPreItem + 48;
constexpr int kPreAbort = kPreTmem + 8;
constexpr int kPreSmem = kPreAbort + 8;
static_assert(kPreRing % 1024 == 0 && kPairStage % 1024 == 0 && kPreSmem <= 232448, "shared memory");

struct PrefillMaps {
  CUtensorMap q, k, pe, v;
};

// 32 columns of this thread's lane, without waiting for the data.
__device__ __forceinline__ void tc_ld32_nowait(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One item as every role sees it: a block of rows of a sequence and a head.
struct PreItem {
  int q0, k0, lq, lk;  // first query and key of the sequence, its lengths
  int r0, h;           // the block's first row; head, or -1 behind the last item
  int n0, n1;          // ends of the two query tiles' key tiles (0 where a tile has no row or its rows see nothing)
  int i0, slot;        // first key tile; where the partial rows go, or -1 (split calls)
  __device__ __forceinline__ int nt() const { return max(n0, n1); }
};

// A split call: few long items leave SMs idle, so the items lie in a line of costs
// (kPreItemCost and one a key tile), which is cut into equal shares, one CTA or pair a
// share.  A share that holds a part of an item writes its rows (normalised) and their
// lse in fp32 to its first or second slot, and the join kernel adds the parts up.
struct PrefillSplit {
  int shares;       // 0: not split
  int64_t size;     // of a share (packed: found on the device)
  float* part;      // [2 shares][rows of an item][128]
  float* part_lse;  // [2 shares][rows of an item], log2
};
constexpr int kSplitLeast = 8 + kPreItemCost;  // least share
__device__ __forceinline__ int64_t split_size(const PrefillParams& p, const PrefillSplit& sp) {
  if (!p.items) return sp.size;
  const int64_t total = (int64_t)p.count[2] * p.H;
  return max((int64_t)kSplitLeast, (total + sp.shares - 1) / sp.shares);
}

// The items of a CTA or pair, most work first: every grid-th of the list, each
// second round backwards, so that the work of all is nearly the same.  Packed
// sequences' single CTAs take them as they come instead, by a counter behind the
// list's length: an item's time is its tiles' and about two tiles' more, which the
// order does not know, and the CTAs ended 20% apart (24 sequences of up to 2048
// tokens, 16 heads: 186 us in the fixed order, 167 by the counter).
template <bool kPair>
struct PreWalk {
  static constexpr int kTileRows = kPair ? 2 * kPreRows : kPreRows;
  int64_t round, total;
  // Block `back` from the end of a causal sequence (later ones see more keys and go first), x = sequence * H + head.
  static __device__ __forceinline__ void dense(const PrefillParams& p, int64_t per, uint32_t back, uint32_t x, PreItem& it) {
    const uint32_t n = x / (uint32_t)p.H;
    it.h = (int)(x - n * (uint32_t)p.H);
    it.q0 = (int)(n * p.Tq);
    it.k0 = (int)(n * p.Tk);
    it.lq = (int)p.Tq;
    it.lk = (int)p.Tk;
    it.r0 = (int)(per - 1 - back) * 2 * kTileRows;
    block_tiles(it.lq, it.lk, p.causal, it.r0, kTileRows, it.n0, it.n1);
  }
  // An entry of the list (without its head).
  static __device__ __forceinline__ void listed(const PrefillParams& p, uint32_t e, PreItem& it) {
    const int4 a = *reinterpret_cast<const int4*>(p.items + e);
    it.q0 = a.x;
    it.k0 = a.y;
    it.lq = a.z;
    it.lk = a.w;
    it.r0 = p.items[e].r0;
    block_tiles(it.lq, it.lk, p.causal, it.r0, kTileRows, it.n0, it.n1);
  }
  __device__ __forceinline__ void start(const PrefillParams& p, int64_t blocks) {
    round = 0;
    total = (p.items ? (int64_t)*p.count : blocks) * p.H;
  }
  __device__ __forceinline__ bool next(const PrefillParams& p, int64_t per, PreItem& it) {
    const int64_t wide = kPair ? gridDim.x >> 1 : gridDim.x, mine = kPair ? blockIdx.x >> 1 : blockIdx.x;
    const int64_t base = round * wide;
    int64_t idx = base + ((round & 1) ? wide - 1 - mine : mine);
    if (!kPair && p.items && round > 0) {  // (all lanes of a warp are here)
      int next = 0;
      if ((threadIdx.x & 31) == 0) next = atomicAdd(p.count + 1, 1);
      idx = wide + __shfl_sync(0xffffffffu, next, 0);
    }
    ++round;
    if (idx >= total) return false;
    if (p.items) {
      const uint32_t e = (uint32_t)idx / (uint32_t)p.H;
      it.h = (int)((uint32_t)idx - e * (uint32_t)p.H);
      listed(p, e, it);
    } else {
      const uint32_t bh = (uint32_t)(p.B * p.H), back = (uint32_t)idx / bh;
      dense(p, per, back, (uint32_t)idx - back * bh, it);
    }
    return true;
  }
};

// The items and parts of items of one share.  A block is one of a dense call's `per`
// from the end, with its sequences and heads, or an entry of the list with its heads.
template <bool kPair>
struct PreShare {
  int64_t u0, u1, pre, cost;  // the share; start and cost of the next item
  uint32_t blocks, wide, back, x;
  PreItem block;
  __device__ __forceinline__ void at_block(const PrefillParams& p, int64_t per) {
    if (p.items) PreWalk<kPair>::listed(p, back, block);
    else PreWalk<kPair>::dense(p, per, back, 0, block);
    cost = block.nt() + kPreItemCost;
  }
  // (all lanes of a warp are here)
  __device__ __forceinline__ void start(const PrefillParams& p, int64_t per, const PrefillSplit& sp, int64_t share) {
    const int64_t size = split_size(p, sp);
    u0 = share * size;
    u1 = u0 + size;
    pre = 0;
    x = 0;
    blocks = p.items ? (uint32_t)*p.count : (uint32_t)per;
    wide = p.items ? (uint32_t)p.H : (uint32_t)(p.B * p.H);
    if (p.items) {
      const int lane = threadIdx.x & 31;
      for (back = 0; back < blocks; back += 32) {
        const PrefillItem* e = p.items + min(back + lane, blocks - 1);
        const int64_t from = (int64_t)e->start * p.H, to = from + (int64_t)(e->tiles + kPreItemCost) * p.H;
        const unsigned here = __ballot_sync(0xffffffffu, back + lane < blocks && from <= u0 && u0 < to);
        if (here) {
          const int at = __ffs(here) - 1;
          back += at;
          pre = __shfl_sync(0xffffffffu, from, at);
          break;
        }
      }
      if (back < blocks) at_block(p, per);
    } else {
      for (back = 0; back < blocks; ++back) {
        at_block(p, per);
        if (pre + wide * cost > u0) break;
        pre += wide * cost;
      }
    }
    if (back < blocks) {
      x = (uint32_t)((u0 - pre) / cost);
      pre += x * cost;
    }
  }
  __device__ __forceinline__ bool next(const PrefillParams& p, int64_t per, int share, PreItem& it) {
    while (back < blocks && pre < u1) {
      if (p.items) {
        it = block;
        it.h = (int)x;
      } else {
        PreWalk<kPair>::dense(p, per, back, x, it);
      }
      const int64_t nt = it.nt(), first = pre + kPreItemCost;  // key tile k lies at first + k
      const int t0 = (int)max((int64_t)0, min(nt, u0 - first)), t1 = (int)max((int64_t)0, min(nt, u1 - first));
      const bool mine = nt > 0 ? t0 < t1 : pre >= u0;
      it.i0 = t0;
      it.slot = t0 == 0 && t1 == nt ? -1 : 2 * share + (t0 > 0 ? 0 : 1);
      it.n0 = min(it.n0, t1);
      it.n1 = min(it.n1, t1);
      pre += cost;
      if (++x == wide) {
        x = 0;
        if (++back < blocks) at_block(p, per);
      }
      if (mine) return true;
    }
    return false;
  }
};

template <bool kPair, bool kSplit>
__global__ void __launch_bounds__(kPreThreads, 1)
    kda_latent_prefill_kernel(const PrefillParams p, int64_t per, const PrefillSplit sp,
                              const __grid_constant__ PrefillMaps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sb = smem_u32(smem), bars = sb + kPreBar;
  auto bar = [&](int i) { return bars + 8 * i; };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kPreAbort);
  const uint32_t rank = kPair ? cta_rank() : 0;
  if (tid == 0) {
    for (int i = 0; i < kPbars; ++i) {
      uint32_t n = 1;
      if (i == kPbP || i == kPbP + 1 || i == kPbP2 || i == kPbP2 + 1) n = kPair ? 8 : 4;               // the softmax warps of a tile
      if (kPair && (i == kPbQ || (i >= kPpFullK && i < kPpFullK + 2 * kPairStages))) n = 2;  // both CTAs' copies
      if (i == kPbItemRead) n = kPair && rank ? 9 : 10;  // warps of softmax, copies and, where it issues, products
      mbar_init(bar(i), n);
    }
    *s_abort = (sb & 1023) ? 1 : 0;
    if (sb & 1023) atomicExch(p.status, KDA_ERR_DEVICE_TIMEOUT);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 9) {
    if constexpr (kPair) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sb + kPreTmem), "r"(512u));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(sb + kPreTmem), "r"(512u));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
  }
  if (warp == 8 && lane == 0) {
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
    prefetch_map(&maps.pe);
    prefetch_map(&maps.v);
  }
  // (set up while the kernel before this one ends; packed, that is the one that lists the blocks)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // the other CTA's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kPreTmem);
  if (kSplit) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (mbar_try_wait(b, parity) || *s_abort) return;
    if (!mbar_wait_bounded(b, parity)) {
      atomicExch(p.status, KDA_ERR_DEVICE_TIMEOUT);
      *s_abort = 1;
    }
  };
  // barriers that the issuing CTA waits on, as both CTAs' copies and warps reach them
  auto lead = [&](int i) { return kPair ? map_rank(bar(i), 0) : bar(i); };
  // The waits for items last as long as an item, which may be longer than one wait is
  // allowed to; a timeout of another ends them.
  auto wait_long = [&](uint32_t b, uint32_t parity) {
    bool there = mbar_try_wait(b, parity);
    for (int k = 0; k < 512 && !there && !*s_abort; ++k) there = mbar_wait_bounded(b, parity);
    return __all_sync(0xffffffffu, there) != 0;
  };
  // The next item, for all lanes of a warp; false behind the last one or after a timeout.
  uint32_t taken = 0;
  // Broadcast, so that the compiler knows the values as uniform (the products are then issued without moves to
  // uniform registers: 368 -> 361 us on the 8192-token prompt, 191 -> 185 on two pieces of 1024 behind 15360).
  auto take = [&](PreItem& it) {
    if (!wait_long(bar(kPbItem), taken & 1)) return false;
    ++taken;
    const int4* from = reinterpret_cast<const int4*>(smem + kPreItem);
    const int4 a = from[0], b = from[1];
    const int2 c = kSplit ? *reinterpret_cast<const int2*>(from + 2) : make_int2(0, -1);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kPbItemRead));
    auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    it = {same(a.x), same(a.y), same(a.z), same(a.w), same(b.x), same(b.y), same(b.z), same(b.w),
          kSplit ? same(c.x) : 0, kSplit ? same(c.y) : -1};
    return it.h >= 0;
  };
  PreItem it;
  int g = 0;  // key tiles so far, over all items

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kPreRegsFew));
  if (kPair && warp == 8) {
    // ---- copies of a pair: this CTA's half of the keys and of the value channels, its query rows ----
    bool gone = false;
    int keys = 0, values = 0, tails = 0, q = 0;  // tiles and items on the way
    auto stop = [&]() {
      __syncwarp();
      gone = __any_sync(0xffffffffu, *s_abort != 0);
      return gone;
    };
    int s = 0;
    uint32_t ph = 1;  // parity of the stage's use before
    while (!gone && take(it)) {
      const int nt = it.nt();
      for (int i = it.i0; i < nt && !gone; ++i, ++g) {
        const int key = it.k0 + i * kPreKeys;
        const uint32_t dst = sb + kPreRing + s * kPairStage;
        if (g >= kPairStages) wait(bar(kPpEmptyK + s), ph);
        if (stop()) break;
        if (lane == 0) {
          const uint32_t full = lead(kPpFullK + s);
          const int own = key + 64 * (int)rank;
          mbar_expect_tx_cluster(full, 3 * kPairK);
          tma_pair_3d(dst, &maps.k, 0, it.h, own, full);
          tma_pair_3d(dst + kPairK, &maps.k, 64, it.h, own, full);
          tma_pair_2d(dst + 2 * kPairK, &maps.pe, 0, own, full);
        }
        ++keys;
        if (i == it.i0) {
          if (q > 0) wait(bar(kPbQEmpty), (uint32_t)((q - 1) & 1));
          if (stop()) break;
          if (lane == 0) {
            const uint32_t full = lead(kPbQ);
            mbar_expect_tx_cluster(full, 2 * kPreQTile);
            for (int t = 0; t < 2; ++t)
              for (int b = 0; b < 3; ++b)
                tma_pair_3d(sb + kPreQ + t * kPreQTile + b * kPreRows * 128, &maps.q, 64 * b, it.h,
                            (int)(it.q0 + it.r0 + (2 * t + (int)rank) * kPreRows), full);
          }
          ++q;
        }
        if (g >= kPairStages) wait(bar(kPpEmptyV + s), ph);
        if (stop()) break;
        const int valid = it.lk - i * kPreKeys;
        const uint32_t full = lead(kPpFullV + s);
        if (valid >= kPreKeys) {
          if (lane == 0) {
            mbar_expect_tx_cluster(full, kPreSlot);
            tma_pair_3d(dst + 3 * kPairK, &maps.v, 64 * (int)rank, it.h, key, full);
          }
        } else {
          // rows behind the sequence take part with weight 0: they have to be finite.  The tile
          // lands on a barrier of this CTA's own, is cleared, and only then handed over
          if (lane == 0) {
            mbar_expect_tx(bar(kPpTail), kPreSlot);
            tma_load_3d(dst + 3 * kPairK, &maps.v, 64 * (int)rank, it.h, key, bar(kPpTail));
          }
          ++tails;
          wait(bar(kPpTail), (uint32_t)((tails - 1) & 1));
          if (stop()) break;
          unsigned char* rows = smem + kPreRing + s * kPairStage + 3 * kPairK + valid * 128;
          for (int x = lane; x < (kPreKeys - valid) * 8; x += 32)
            reinterpret_cast<uint4*>(rows)[x] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_release_cluster(full);
        }
        ++values;
        if (++s == kPairStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    stop();
    // After a timeout: copies still in flight land in memory of this CTA, which stays until
    // the cluster's last barrier; they are few and unconditional, so a bounded pause is enough.
    if (gone && lane == 0) {
      if (tails > 0) mbar_wait_bounded(bar(kPpTail), (uint32_t)((tails - 1) & 1));
      const long long t0 = clock64();
      while (clock64() - t0 < (1LL << 22)) {
      }
    }
  } else if (kPair && warp == 9) {
    // ---- products of the pair, issued by its first CTA ----
    if (rank == 0) {
      const uint32_t id_s = idesc_bf16(2 * kPreRows, kPreKeys, false, false);
      const uint32_t id_o = idesc_bf16(2 * kPreRows, kVDim, false, true);
      const uint64_t d_q = smem_desc(sb + kPreQ, 16, 1024), d_k = smem_desc(sb + kPreRing, 16, 1024);
      const uint64_t d_v = smem_desc(sb + kPreRing + 3 * kPairK, 16, 1024);
      auto wait_pair = [&](uint32_t b, uint32_t parity) {
        wait(b, parity);
        __syncwarp();
        tc_fence_after();
      };
      int q = 0, done0 = 0, done1 = 0;
      int s = 0, s_prev = 0;     // stage of this key tile and of the one before
      uint32_t ph = 0;
      // One place each for the products of every query tile: a copy of them for the last step
      // would run once an item, from cold instruction caches.
      auto scores = [&](int t) {
        const uint64_t a = d_q + (uint64_t)((t * kPreQTile) >> 4), b = d_k + (uint64_t)((s * kPairStage) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss<true>(tmem + 128 * t, a + (uint64_t)((c * kPreRows * 128 + ks * 32) >> 4),
                           b + (uint64_t)((c * kPairK + ks * 32) >> 4), id_s, c + ks > 0);
          mma_commit<true>(bar(kPbS + t));
        }
        __syncwarp();
      };
      auto values = [&](int t, int stage, int& done, bool first) {
        const uint64_t b = d_v + (uint64_t)((stage * kPairStage) >> 4);
        const uint32_t o = tmem + 256 + 128 * t, a = tmem + 128 * t, more = first ? 0u : 1u;
        wait_pair(bar(kPbP + t), (uint32_t)(done & 1));
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < kPreFirst / 16; ++ks)
            mma_ts<true>(o, a + 8 * ks, b + (uint64_t)((ks * 2048) >> 4), id_o, ks > 0 ? 1u : more);
        }
        __syncwarp();
        wait_pair(bar(kPbP2 + t), (uint32_t)(done & 1));
        ++done;
        if (elect_one()) {
#pragma unroll
          for (int ks = kPreFirst / 16; ks < 8; ++ks)
            mma_ts<true>(o, a + 8 * ks, b + (uint64_t)((ks * 2048) >> 4), id_o, 1u);
          mma_commit<true>(bar(kPbPv + t));
        }
        __syncwarp();
      };
      auto done_with = [&](int b) {
        if (elect_one()) mma_commit<true>(bar(b));
        __syncwarp();
      };
      while (take(it)) {
        const int nt = it.nt();
        if (nt == 0) continue;  // (== : told that nt is positive, the compiler builds a loop that is 3% slower)
        wait_pair(bar(kPbQ), (uint32_t)(q & 1));
        ++q;
        for (int i = it.i0; i <= nt; ++i) {
          const bool keys = i < nt;
          if (keys) {
            wait_pair(bar(kPpFullK + s), ph);
            if (i < it.n0) scores(0);
          }
          if (i > it.i0) {
            if (i - 1 < it.n1) values(1, s_prev, done1, i - 1 == it.i0);
            done_with(kPpEmptyV + s_prev);
          }
          if (!keys) break;
          if (i < it.n1) scores(1);
          done_with(kPpEmptyK + s);
          if (i + 1 == nt) done_with(kPbQEmpty);
          wait_pair(bar(kPpFullV + s), ph);
          if (it.lk < (i + 1) * kPreKeys) mbar_try_wait_cluster(bar(kPpFullV + s), ph);  // acquires the cleared rows
          if (i < it.n0) values(0, s, done0, i == it.i0);
          s_prev = s;
          if (++s == kPairStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (done0 > 0) mbar_wait_bounded(bar(kPbPv), (uint32_t)((done0 - 1) & 1));
      if (done1 > 0) mbar_wait_bounded(bar(kPbPv + 1), (uint32_t)((done1 - 1) & 1));
    }
  } else if (warp == 8) {
    // ---- copies.  Key tile g's five slots (two key blocks, pe, two value blocks) start at
    //      slot 5 g % 8: its first key block follows the last one of tile g - 2 (free where the
    //      values of g - 1 could be sent), its other two the values of g - 2, its values the keys
    //      of g - 1 ----
    bool gone = false;
    int keys0 = 0, keys = 0, values = 0, q = 0;  // tiles whose parts, and items whose queries, are on the way
    auto stop = [&]() {
      __syncwarp();
      gone = __any_sync(0xffffffffu, *s_abort != 0);
      return gone;
    };
    while (!gone && take(it)) {
      const int nt = it.nt();
      for (int i = it.i0; i < nt && !gone; ++i, ++g) {
        const int key = it.k0 + i * kPreKeys, s = g & 1;
        auto dst = [&](int c) { return sb + kPreRing + ((5 * g + c) % kPreSlots) * kPreSlot; };
        if (lane == 0) {
          mbar_expect_tx(bar(kPbFullK0 + s), kPreSlot);
          tma_load_3d(dst(0), &maps.k, 0, it.h, key, bar(kPbFullK0 + s));
        }
        ++keys0;
        if (g >= 2) wait(bar(kPbEmptyV + s), (uint32_t)(((g - 2) >> 1) & 1));
        if (stop()) break;
        if (lane == 0) {
          mbar_expect_tx(bar(kPbFullK + s), 2 * kPreSlot);
          tma_load_3d(dst(1), &maps.k, 64, it.h, key, bar(kPbFullK + s));
          tma_load_2d(dst(2), &maps.pe, 0, key, bar(kPbFullK + s));
        }
        ++keys;
        if (i == it.i0) {
          if (q > 0) wait(bar(kPbQEmpty), (uint32_t)((q - 1) & 1));
          if (stop()) break;
          if (lane == 0) {
            mbar_expect_tx(bar(kPbQ), 2 * kPreQTile);
            for (int t = 0; t < 2; ++t)
              for (int b = 0; b < 3; ++b)
                tma_load_3d(sb + kPreQ + t * kPreQTile + b * kPreRows * 128, &maps.q, 64 * b, it.h,
                            (int)(it.q0 + it.r0 + t * kPreRows), bar(kPbQ));
          }
          ++q;
        }
        if (g >= 1) wait(bar(kPbEmptyK + (s ^ 1)), (uint32_t)(((g - 1) >> 1) & 1));
        if (stop()) break;
        if (lane == 0) {
          mbar_expect_tx(bar(kPbFullV + s), 2 * kPreSlot);
          tma_load_3d(dst(3), &maps.v, 0, it.h, key, bar(kPbFullV + s));
          tma_load_3d(dst(4), &maps.v, 64, it.h, key, bar(kPbFullV + s));
        }
        ++values;
      }
    }
    stop();
    // After a timeout: let the copies still in flight land before leaving.
    if (gone && lane == 0) {
      auto drain = [&](int b, int n) {
        for (int i = max(0, n - 2); i < n; ++i) mbar_wait_bounded(bar(b + (i & 1)), (uint32_t)((i >> 1) & 1));
      };
      drain(kPbFullK0, keys0);
      drain(kPbFullK, keys);
      drain(kPbFullV, values);
      if (q > 0) mbar_wait_bounded(bar(kPbQ), (uint32_t)((q - 1) & 1));
    }
  } else if (warp == 9) {
    // ---- products ----
    const uint32_t id_s = idesc_bf16(kPreRows, kPreKeys, false, false);
    const uint32_t id_o = idesc_bf16(kPreRows, kVDim, false, true), id_o64 = idesc_bf16(kPreRows, 64, false, true);
    const uint64_t d_q = smem_desc(sb + kPreQ, 16, 1024), d_k = smem_desc(sb + kPreRing, 16, 1024);
    const uint64_t d_v = smem_desc(sb + kPreRing, kPreSlot, 1024);
    int q = 0, done0 = 0, done1 = 0;  // items; weights used of the two query tiles
    auto slot_of = [&](int tile, int c) { return (5 * tile + c) % kPreSlots; };
    auto full_wait = [&](int b, int tile) {
      wait(bar(b + (tile & 1)), (uint32_t)((tile >> 1) & 1));
      __syncwarp();
      tc_fence_after();
    };
    // S of query tile t against key tile `tile`; `fresh`: the first product to read these keys
    auto scores = [&](int t, int tile, bool fresh) {
      const uint64_t a = d_q + (uint64_t)((t * kPreQTile) >> 4);
      auto part = [&](int c) {
        const uint64_t b = d_k + (uint64_t)((slot_of(tile, c) * kPreSlot) >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss<false>(tmem + 128 * t, a + (uint64_t)((c * kPreRows * 128 + ks * 32) >> 4), b + 2 * ks, id_s, c + ks > 0);
      };
      if (fresh) full_wait(kPbFullK0, tile);
      if (elect_one()) part(0);
      __syncwarp();
      if (fresh) full_wait(kPbFullK, tile);
      if (elect_one()) {
        part(1);
        part(2);
        mma_commit<false>(bar(kPbS + t));
      }
      __syncwarp();
    };
    // O of query tile t += its weights times the values of key tile `tile`
    auto values = [&](int t, int tile, int& done, bool first) {
      wait(bar(kPbP + t), (uint32_t)(done & 1));
      ++done;
      __syncwarp();
      tc_fence_after();
      const int s0 = slot_of(tile, 3), s1 = slot_of(tile, 4);
      const uint32_t o = tmem + 256 + 128 * t, a = tmem + 128 * t, more = first ? 0u : 1u;
      const uint64_t b0 = d_v + (uint64_t)((s0 * kPreSlot) >> 4), b1 = d_v + (uint64_t)((s1 * kPreSlot) >> 4);
      if (elect_one()) {
        if (s1 == s0 + 1) {  // the two 64-column blocks lie one slot apart: one operand of 128 columns
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ts<false>(o, a + 8 * ks, b0 + (uint64_t)((ks * 2048) >> 4), id_o, ks > 0 ? 1u : more);
        } else {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            mma_ts<false>(o, a + 8 * ks, b0 + (uint64_t)((ks * 2048) >> 4), id_o64, ks > 0 ? 1u : more);
            mma_ts<false>(o + 64, a + 8 * ks, b1 + (uint64_t)((ks * 2048) >> 4), id_o64, ks > 0 ? 1u : more);
          }
        }
        mma_commit<false>(bar(kPbPv + t));
      }
      __syncwarp();
    };
    auto done_with = [&](int b) {
      if (elect_one()) mma_commit<false>(bar(b));
      __syncwarp();
    };
    while (take(it)) {
      const int nt = it.nt();
      if (nt == 0) continue;
      wait(bar(kPbQ), (uint32_t)(q & 1));
      ++q;
      __syncwarp();
      for (int i = it.i0; i <= nt; ++i) {
        const int tile = g + i - it.i0;
        const bool keys = i < nt;
        if (keys && i < it.n0) scores(0, tile, true);
        if (i > it.i0) {
          if (i - 1 < it.n1) values(1, tile - 1, done1, i - 1 == it.i0);
          done_with(kPbEmptyV + ((tile - 1) & 1));
        }
        if (!keys) break;
        if (i < it.n1) scores(1, tile, i >= it.n0);
        done_with(kPbEmptyK + (tile & 1));
        if (i + 1 == nt) done_with(kPbQEmpty);
        full_wait(kPbFullV, tile);
        const int valid = it.lk - i * kPreKeys;
        if (valid < kPreKeys) {
          // rows behind the sequence take part with weight 0: they have to be finite
          for (int c = 3; c < 5; ++c) {
            unsigned char* rows = smem + kPreRing + slot_of(tile, c) * kPreSlot + valid * 128;
            for (int x = lane; x < (kPreKeys - valid) * 8; x += 32)
              reinterpret_cast<uint4*>(rows)[x] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (i < it.n0) values(0, tile, done0, i == it.i0);
      }
      g += nt - it.i0;
    }
    // the last products complete before tensor memory is freed
    if (done0 > 0) mbar_wait_bounded(bar(kPbPv), (uint32_t)((done0 - 1) & 1));
    if (done1 > 0) mbar_wait_bounded(bar(kPbPv + 1), (uint32_t)((done1 - 1) & 1));
  } else if (warp == 10) {
    // ---- the items: the next one is found while the others work on theirs (found by each
    //      role for itself, it cost the products some 3000 cycles between two items) ----
    PreWalk<kPair> walk;
    PreShare<kPair> share;
    const int mine = kPair ? blockIdx.x >> 1 : blockIdx.x;
    if constexpr (kSplit) share.start(p, per, sp, mine);
    else walk.start(p, p.B * per);
    bool have = true;
    for (uint32_t n = 0; have; ++n) {
      if constexpr (kSplit) have = share.next(p, per, mine, it);
      else have = walk.next(p, per, it);
      if (!have) it.h = -1;
      if (n > 0 && !wait_long(bar(kPbItemRead), (n - 1) & 1)) break;
      if (lane == 0) {
        int4* to = reinterpret_cast<int4*>(smem + kPreItem);
        to[0] = make_int4(it.q0, it.k0, it.lq, it.lk);
        to[1] = make_int4(it.r0, it.h, it.n0, it.n1);
        if (kSplit) *reinterpret_cast<int2*>(to + 2) = make_int2(it.i0, it.slot);
        mbar_arrive(bar(kPbItem));
      }
      __syncwarp();
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kPreRegsMany));
    // ---- softmax and output: thread = row of tile t ----
    const int t = warp >> 2, q = warp & 3;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    const uint32_t t_s = tmem + lane_base + 128 * t, t_o = tmem + lane_base + 256 + 128 * t;
    const float sl = p.scale_log2;
    const f32x2 sl2 = f2(sl, sl);
    int done = 0;  // scores used
    auto hand_over = [&](int b) {  // the weights stored so far, to the products
      tc_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair) mbar_arrive_cluster(lead(b));
        else mbar_arrive(bar(b));
      }
    };
    while (take(it)) {
      const int n = t == 0 ? it.n0 : it.n1;
      const int row = it.r0 + (kPair ? 2 * t + (int)rank : t) * kPreRows + q * 32 + lane;  // query within the sequence
      const int lim = p.causal ? min(it.lk, row + it.lk - it.lq + 1) : it.lk;
      const int lim_first = p.causal ? min(it.lk, row - lane + it.lk - it.lq + 1) : it.lk;  // the warp's first row's
      float m = -INFINITY, l = 0.f;  // maximum (times scale, log2) and sum
      for (int i = it.i0; i < n; ++i, ++done) {
        wait(bar(kPbS + t), (uint32_t)(done & 1));
        __syncwarp();
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32_nowait(t_s + 32 * c, s + 32 * c);
        tc_ld_wait();
        if ((i + 1) * kPreKeys > lim_first) {
          const int rem = lim - i * kPreKeys;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= rem) s[c] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[c + 2 * e], s[c + 2 * e + 1]);
        mx[0] = max3(mx[0], s[124], s[125]);
        mx[1] = max3(mx[1], s[126], s[127]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
        if (__any_sync(0xffffffffu, top > m + kPreSlack)) {
          float f = 1.0f;
          if (top > m + kPreSlack) {
            f = ex2(m - top);
            m = top;
            l *= f;
          }
          if (i > it.i0) {
            wait(bar(kPbPv + t), (uint32_t)((done - 1) & 1));
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              float o[16];
              tc_ld16(t_o + c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= f;
              tc_st16(t_o + c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : -m;
        const f32x2 base2 = f2(base, base);
        f32x2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          // 32 weights as bf16 pairs (the operand type; the sum is taken before the rounding): on the 8192-token
          // prompt a relative RMS against 64 bits of 0.0020, of which 0.0015 are the output's rounding
          float w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = f2u(fma2(f2(s[c + 2 * e], s[c + 2 * e + 1]), sl2, base2));
            const float a = ex2(x.x), b = ex2(x.y);
            sum[e & 1] = add2(sum[e & 1], f2(a, b));
            w[e] = __uint_as_float(pack_bf16(a, b));
          }
          tc_st16(t_s + c / 2, w);
          if (kPair && c == kPreFirst - 32) hand_over(kPbP + t);
        }
        hand_over((kPair ? kPbP2 : kPbP) + t);
        const float2 z = f2u(add2(sum[0], sum[1]));
        l += z.x + z.y;
      }
      // ---- this row ----
      if (n > it.i0) {
        wait(bar(kPbPv + t), (uint32_t)((done - 1) & 1));
        __syncwarp();
        tc_fence_after();
      }
      const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
      const int64_t at = ((int64_t)it.q0 + row) * p.H + it.h;
      const int64_t part_row = (int64_t)it.slot * (kPair ? 4 : 2) * kPreRows + row - it.r0;
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        float o[64];
        if (n > it.i0) {
          tc_ld32_nowait(t_o + c, o);
          tc_ld32_nowait(t_o + c + 32, o + 32);
          tc_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e] = 0.f;
        }
        if (kSplit && it.slot >= 0) {
          if (row < it.lq) {
            float* dst = sp.part + part_row * kVDim + c;
#pragma unroll
            for (int e = 0; e < 64; e += 8)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + e), "f"(o[e] * inv),
                           "f"(o[e + 1] * inv), "f"(o[e + 2] * inv), "f"(o[e + 3] * inv), "f"(o[e + 4] * inv),
                           "f"(o[e + 5] * inv), "f"(o[e + 6] * inv), "f"(o[e + 7] * inv)
                           : "memory");
          }
        } else if (row < it.lq) {
          // whole 32-byte sectors: a 16-byte store of a row alone would write halves of them.  The
          // wide store needs a 32-byte boundary; an `out` that starts in the middle of one gets halves
          uint16_t* dst = p.out + at * kVDim + c;
          const bool aligned = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;  // (rows are 256 bytes)
#pragma unroll
          for (int e = 0; e < 64; e += 16) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = pack_bf16(o[e + 2 * x] * inv, o[e + 2 * x + 1] * inv);
            if (aligned) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + e), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                           : "memory");
            } else {
              reinterpret_cast<uint4*>(dst + e)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(dst + e)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
      if (kSplit && it.slot >= 0) {
        if (row < it.lq) sp.part_lse[part_row] = lse2;
      } else if (p.lse && row < it.lq) {
        p.lse[at] = lse2 * 0.6931471805599453f;
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // nothing of this pair reaches a CTA that has left
  tc_fence_after();
  if (warp == 9) {
    if constexpr (kPair)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
  }
}

namespace {

// [tokens][H][d] with token / head strides: 64 x 1 x `rows` boxes
bool head_map(CUtensorMap* m, const uint16_t* base, int d, int64_t H, int64_t tokens, int64_t st, int64_t sh, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
  return encode_map_bf16(m, base, 3, dims, strides, box);
}

template <bool kPair, bool kSplit>
bool launch_prefill(const PrefillParams& p, const PrefillSplit& sp, int sms, cudaStream_t s) {
  static std::once_flag once[64];
  static cudaError_t rc[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  std::call_once(once[dev], [&] {
    rc[dev] = cudaFuncSetAttribute(kda_latent_prefill_kernel<kPair, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   kPreSmem);
  });
  if (rc[dev] != cudaSuccess) return false;
  const int rows = kPair ? 2 * kPrefillRows : kPrefillRows;
  const int64_t per = (p.Tq + rows - 1) / rows;
  const int64_t items = (p.items ? p.Tq / rows + p.N : p.B * per) * p.H;
  if (items > INT32_MAX) return false;
  PrefillMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!head_map(&maps.q, p.q, kQkDim, p.H, p.B * p.Tq, p.q_st, p.q_sh, kPreRows)) return false;
  const int64_t keys = p.B * p.Tk;
  if (keys > 0) {  // (without keys no key tile exists and nothing is copied)
    const int box_keys = kPair ? kPreKeys / 2 : kPreKeys;
    const cuuint64_t dims[2] = {kLatPe, (cuuint64_t)keys};
    const cuuint64_t strides[1] = {(cuuint64_t)p.pe_st * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_keys};
    if (!head_map(&maps.k, p.k, kNope, p.H, keys, p.k_st, p.k_sh, box_keys) ||
        !head_map(&maps.v, p.v, kVDim, p.H, keys, p.v_st, p.v_sh, kPreKeys) ||
        !encode_map_bf16(&maps.pe, p.k_pe, 2, dims, strides, box))
      return false;
  }
  const int64_t ctas = kSplit ? sp.shares : std::min<int64_t>(items, kPair ? sms / 2 : sms);
  return launch_overlapped(kda_latent_prefill_kernel<kPair, kSplit>, dim3((unsigned)(kPair ? 2 * ctas : ctas)), kPreThreads,
                         kPreSmem, s, kPair ? 2 : 1, p, per, sp, maps);
}

}  // namespace

// The split form, in a file of its own.
bool launch_prefill_split(const PrefillParams& p, const PrefillSplit& sp, int sms, cudaStream_t s);

}  // namespace kda
