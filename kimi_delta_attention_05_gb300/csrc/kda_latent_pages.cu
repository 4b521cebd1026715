// Pages of the latent cache that several rows of a block table hold: fork,
// release, compact and copy (include/kda_latent.h).
//
// Holders are counted beyond the first (shares[page]: 0 where one row holds the
// page), so pages that kda_latent_plan takes are right as they come.  Counts are
// changed by integer atomics, whose order does not show, and every list that
// comes out is in ascending order of pages, by a scan: results do not depend on
// timing.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "../../include/kda_latent.h"
#include "kda_common.cuh"
#include "kda_kernels.cuh"
#include "kda_latent.cuh"

namespace kda {

namespace cg = cooperative_groups;

constexpr int kRowPieces = kLatRow / 8;         // 16-byte pieces of a cache row
constexpr int kGroupRows = 8;                   // page sizes are multiples of this
constexpr int kCopyThreads = 4 * kRowPieces;    // four rows at a time, twice a group
constexpr int kPageThreads = 512;
constexpr int kPageCluster = 8;                 // CTAs of the kernels that list pages

struct PageCache {
  uint16_t* data;
  int64_t num_pages, page_stride, token_stride;
};

__device__ __forceinline__ int warp_scan_int(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Pages of a length that is not negative.
__device__ __forceinline__ int pages_of(int tokens, int page) { return (int)(((uint32_t)tokens + (uint32_t)page - 1) / (uint32_t)page); }

// Exclusive prefix over the block's warps of a value that each warp's lanes share; `total` gets the sum.  (One warp
// adds up the warps' values: every thread for itself took 3600 cycles of 1024 threads.)
template <int kThreads>
__device__ __forceinline__ int warps_before(int x, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int own = lane < kThreads / 32 ? sums[lane] : 0, upto = warp_scan_int(own, lane);
    __syncwarp();
    if (lane < kThreads / 32) sums[lane] = upto - own;
    if (lane == 31) sums[kThreads / 32] = upto;
  }
  __syncthreads();
  const int before = sums[warp];
  total = sums[kThreads / 32];
  __syncthreads();  // sums are read
  return before;
}

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// ---- copies of pages ----
//
// A CTA takes four groups of eight rows at a time (36.9 KB), a thread eight 16-byte
// pieces of them, all loaded before the first is stored: enough bytes in flight for
// HBM with a few CTAs an SM, and any page size is whole groups.  8000 pages of 16
// tokens, 295 MB read and written: 49.7 us, 5.9 TB/s; 33 pages of 64 in 2.8 us, the
// latency of a launch.
struct CopyPlace {
  const uint16_t* src;  // nullptr: nothing to copy
  uint16_t* dst;
  int rows;             // of the group
};

template <class Place>
__device__ __forceinline__ void copy_groups(int64_t groups, int64_t src_stride, int64_t dst_stride, int64_t cta,
                                            int64_t ctas, Place place) {
  const int row = threadIdx.x / kRowPieces, col = (threadIdx.x % kRowPieces) * 8;
  for (int64_t g0 = cta * 4; g0 < groups; g0 += ctas * 4) {
    CopyPlace at[4];
    uint4 x[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      at[k].src = nullptr;
      if (g0 + k < groups) at[k] = place(g0 + k);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (at[k].src && row + 4 * h < at[k].rows)
          x[k][h] = __ldcs(reinterpret_cast<const uint4*>(at[k].src + (row + 4 * h) * src_stride + col));
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (at[k].src && row + 4 * h < at[k].rows)
          *reinterpret_cast<uint4*>(at[k].dst + (row + 4 * h) * dst_stride + col) = x[k][h];
  }
}

// a / b of non-negative numbers, in 32 bits where they fit
__device__ __forceinline__ int64_t div_pages(int64_t a, int b) {
  return (a >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

struct CopyParams {
  PageCache src, dst;
  const int32_t *src_pages, *dst_pages;
  int64_t n;
  int page;
  int* status;
};

__device__ __forceinline__ CopyPlace page_group(const PageCache& src, const PageCache& dst, int64_t from, int64_t to,
                                                int group, int* status) {
  CopyPlace c = {nullptr, nullptr, kGroupRows};
  if (from < 0 || from >= src.num_pages || to < 0 || to >= dst.num_pages) {
    if (threadIdx.x == 0) atomicExch(status, KDA_ERR_BAD_PAGE);
    return c;
  }
  c.src = src.data + from * src.page_stride + (int64_t)group * kGroupRows * src.token_stride;
  c.dst = dst.data + to * dst.page_stride + (int64_t)group * kGroupRows * dst.token_stride;
  return c;
}

__global__ void __launch_bounds__(kCopyThreads) kda_latent_copy_kernel(const CopyParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int per = p.page / kGroupRows;
  copy_groups(p.n * per, p.src.token_stride, p.dst.token_stride, blockIdx.x, gridDim.x, [&](int64_t g) {
    const int64_t i = div_pages(g, per);
    return page_group(p.src, p.dst, p.src_pages[i], p.dst_pages[i], (int)(g - i * per), p.status);
  });
}

// ---- fork ----
//
// Child f takes the first t_f tokens of its parent: floor(t_f / P) table entries,
// whose counts go up by one, and where t_f is not whole pages the free page
// number sum_{e < f} [t_e mod P > 0] with the last t_f mod P rows.  Every CTA checks
// all forks and counts the pages of those before its own for itself (as the plan
// kernel does: a second launch would cost more), then does its share of one fork.
// Bound by launch and three rounds of latency: 8 children of 1000 tokens in 3.4 us, 256
// of up to 8192 tokens, 17.7 MB of rows and entries, in 6.6.
struct ForkParams {
  const int32_t *parents, *children, *take, *cached;
  int32_t* table;
  int64_t table_stride, max_pages;
  const int32_t* free_pages;
  int64_t num_free;
  int32_t* shares;
  PageCache cache;
  int32_t *seq_lens, *taken;
  int F, B, page, parts;  // parts: CTAs a fork
  int* status;
};

__global__ void __launch_bounds__(kCopyThreads) kda_latent_fork_kernel(const ForkParams p) {
  extern __shared__ uint32_t is_child[];  // a bit a row of the table
  __shared__ int counts[2];               // free pages taken: by the forks before this one, by all
  const int tid = threadIdx.x, mine = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  for (int i = tid; i < (p.B + 31) / 32; i += kCopyThreads) is_child[i] = 0;
  if (tid < 2) counts[tid] = 0;
  __syncthreads();
  int bad = 0, before = 0, all = 0;
  for (int f = tid; f < p.F; f += kCopyThreads) {
    const int from = p.parents[f], to = p.children[f];
    if (from < 0 || from >= p.B || to < 0 || to >= p.B) {
      bad = 1;
      continue;
    }
    if (atomicOr(&is_child[to >> 5], 1u << (to & 31)) >> (to & 31) & 1) bad = 1;  // twice
    if (p.cached[to] != 0) bad = 1;                                                // holds pages, which would be lost
    const int held = p.cached[from], t = p.take ? p.take[f] : held;
    if (held < 0 || t < 0 || t > held || held > p.max_pages * p.page) {
      bad = 1;
      continue;
    }
    const int need = t % p.page > 0;
    all += need;
    if (f < mine) before += need;
  }
  if (before) atomicAdd(&counts[0], before);
  if (all) atomicAdd(&counts[1], all);
  __syncthreads();
  for (int f = tid; f < p.F; f += kCopyThreads) {  // a parent that is a child too
    const int from = p.parents[f];
    if (from >= 0 && from < p.B && (is_child[from >> 5] >> (from & 31) & 1)) bad = 1;
  }
  bad = __syncthreads_or(bad);
  const bool refused = bad || counts[1] > p.num_free;
  if (blockIdx.x == 0) {
    if (tid == 0) {
      if (refused) atomicExch(p.status, bad ? KDA_ERR_BAD_LENGTHS : KDA_ERR_NO_PAGES);
      p.taken[0] = refused ? 0 : counts[1];
    }
    for (int b = tid; b < p.B; b += kCopyThreads)
      if (refused || !(is_child[b >> 5] >> (b & 31) & 1)) p.seq_lens[b] = p.cached[b];
    if (!refused)
      for (int f = tid; f < p.F; f += kCopyThreads) p.seq_lens[p.children[f]] = p.take ? p.take[f] : p.cached[p.parents[f]];
  }
  if (refused || mine >= p.F) return;
  const int from = p.parents[mine], to = p.children[mine];
  const int t = p.take ? p.take[mine] : p.cached[from];
  const int full = t / p.page, rest = t - full * p.page;
  const int32_t* src = p.table + from * p.table_stride;
  int32_t* dst = p.table + to * p.table_stride;
  for (int j = part * kCopyThreads + tid; j < full; j += p.parts * kCopyThreads) {
    const int id = src[j];
    dst[j] = id;
    if (id < 0 || id >= p.cache.num_pages) atomicExch(p.status, KDA_ERR_BAD_PAGE);
    else atomicAdd(p.shares + id, 1);
  }
  if (rest == 0) return;
  const int fresh = p.free_pages[counts[0]], old = src[full];
  if (part == 0 && tid == 0) dst[full] = fresh;
  copy_groups((rest + kGroupRows - 1) / kGroupRows, p.cache.token_stride, p.cache.token_stride, part, p.parts,
              [&](int64_t g) {
                CopyPlace c = page_group(p.cache, p.cache, old, fresh, (int)g, p.status);
                c.rows = min(kGroupRows, rest - (int)g * kGroupRows);
                return c;
              });
}

// ---- release ----
//
// The counts of the dropped pages go down (L2 atomics), then the pages that fell
// below 0 are listed in order.  One cluster of eight CTAs does both: its barrier
// stands between them, a CTA lists an eighth, and its place in the list comes from
// the others' numbers over distributed shared memory: one launch, no workspace.  Eight
// SMs take 2.5 cycles an atomic each, so calls with many entries have a kernel on all
// SMs do the counts first.  16 rows of up to 64 pages 5.4 us; 256 rows of up to 1024,
// 144127 pages, 28 us in one kernel and 17.9 in two; a million pages listed in 31 us.
struct ReleaseParams {
  const int32_t *rows, *keep, *cached, *table;
  int64_t table_stride, max_pages;
  int32_t* shares;
  int64_t num_pages;
  int32_t *seq_lens, *pages, *count;
  int F, B, page;
  int* status;
};

constexpr int kReleaseCached = 2048;  // rows whose entries to drop are kept in shared memory

// What a row drops: entries [first, end) of row b of the table.
struct Dropped {
  int b, first, end;
};

size_t release_smem(int64_t B, int64_t F) {
  return (size_t)(B + 31) / 32 * 4 + (size_t)std::min<int64_t>(F, kReleaseCached) * sizeof(Dropped);
}

// Checks the rows, for every CTA by itself: a bit a released row of the table, and what each drops.
__device__ __forceinline__ bool release_rows(const ReleaseParams& p, uint32_t* is_released, Dropped* rows) {
  for (int i = threadIdx.x; i < (p.B + 31) / 32; i += kPageThreads) is_released[i] = 0;
  __syncthreads();
  int bad = 0;
  for (int f = threadIdx.x; f < p.F; f += kPageThreads) {
    const int b = p.rows[f];
    if (b < 0 || b >= p.B) {
      bad = 1;
      continue;
    }
    if (atomicOr(&is_released[b >> 5], 1u << (b & 31)) >> (b & 31) & 1) bad = 1;  // twice
    const int held = p.cached[b], keep = p.keep ? p.keep[f] : 0;
    if (held < 0 || keep < 0 || keep > held || held > p.max_pages * p.page) bad = 1;
    else if (f < kReleaseCached) rows[f] = {b, pages_of(keep, p.page), pages_of(held, p.page)};
  }
  return !__syncthreads_or(bad);
}

// The counts of all dropped pages down: warps take equal parts of rows, eight loads of 32 entries at a time.
__device__ __forceinline__ void release_counts(const ReleaseParams& p, const Dropped* rows, int cta, int ctas) {
  const int lane = threadIdx.x & 31, warps = ctas * (kPageThreads / 32);
  const int part = (int)min((p.F * p.max_pages / warps / 256 + 1) * 256, (int64_t)1 << 30);
  const int parts = (int)(((uint32_t)p.max_pages + part - 1) / part);  // (parts * F is at most about the warps and F)
  for (int i = cta * (kPageThreads / 32) + (threadIdx.x >> 5); i < parts * p.F; i += warps) {
    const int f = i / parts;
    Dropped d;
    if (f < kReleaseCached) {
      d = rows[f];
    } else {
      d.b = p.rows[f];
      d.first = pages_of(p.keep ? p.keep[f] : 0, p.page);
      d.end = pages_of(p.cached[d.b], p.page);
    }
    const int32_t* ids = p.table + d.b * p.table_stride;
    const uint32_t j0 = (uint32_t)(i - f * parts) * part, end = min((uint32_t)d.end, j0 + part);
    for (uint32_t j = max(j0, (uint32_t)d.first) + lane; j < end; j += 256) {
      int id[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) id[k] = j + 32 * k < end ? ids[j + 32 * k] : INT32_MIN;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (id[k] >= 0 && id[k] < p.num_pages) atomicSub(p.shares + id[k], 1);
        else if (j + 32 * k < end) atomicExch(p.status, KDA_ERR_BAD_PAGE);
      }
    }
  }
}

__global__ void __launch_bounds__(kPageThreads) kda_latent_release_counts_kernel(const ReleaseParams p) {
  extern __shared__ uint32_t release_smem_[];
  Dropped* rows = reinterpret_cast<Dropped*>(release_smem_ + (p.B + 31) / 32);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (release_rows(p, release_smem_, rows)) release_counts(p, rows, blockIdx.x, gridDim.x);
}

// counts: whether this kernel does the counts too
__global__ void __launch_bounds__(kPageThreads) kda_latent_release_kernel(const ReleaseParams p, const int counts) {
  extern __shared__ uint32_t release_smem_[];
  __shared__ int sums[kPageThreads / 32 + 1];
  __shared__ int freed[2][kPageCluster];  // pages that each CTA lists in a round, and in the one before or behind it
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster.block_rank();
  Dropped* rows = reinterpret_cast<Dropped*>(release_smem_ + (p.B + 31) / 32);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const bool good = release_rows(p, release_smem_, rows);
  if (good && counts) release_counts(p, rows, rank, kPageCluster);
  if (rank == kPageCluster - 1) {  // (the last CTA: it has the least to do)
    if (!good && tid == 0) atomicExch(p.status, KDA_ERR_BAD_LENGTHS);
    for (int b = tid; b < p.B; b += kPageThreads)
      if (!good || !(release_smem_[b >> 5] >> (b & 31) & 1)) p.seq_lens[b] = p.cached[b];
    if (good)
      for (int f = tid; f < p.F; f += kPageThreads) p.seq_lens[p.rows[f]] = p.keep ? p.keep[f] : 0;
  }
  cluster.sync();  // (waits for the atomics)
  // Rounds of runs of up to 32 x 32 pages, a run a warp: lane w keeps the bits of its pages 32 w .. 32 w + 31, so that
  // a page is read once and stores are of neighbouring lanes.
  constexpr uint32_t kWarps = kPageThreads / 32;
  const uint32_t pages = (uint32_t)p.num_pages;
  const int words = (int)min(32u, (pages + kPageCluster * kWarps * 32 - 1) / (kPageCluster * kWarps * 32));
  const uint32_t length = 32 * words;
  uint32_t all = 0;
  int round = 0;
  for (uint32_t base = 0; base < pages; base += kPageCluster * kWarps * length, ++round) {
    const uint32_t run = base + (rank * kWarps + warp) * length;
    uint32_t bits = 0;
    if (good && run < pages) {
#pragma unroll 1
      for (int w0 = 0; w0 < words; w0 += 16) {
        int x[16];  // (loaded without a branch, so that all are on their way at once)
#pragma unroll
        for (int w = 0; w < 16; ++w) x[w] = __ldcg(p.shares + min(run + 32 * (w0 + w) + lane, pages - 1));
#pragma unroll
        for (int w = 0; w < 16; ++w) {
          const uint32_t mask = __ballot_sync(0xffffffffu, x[w] < 0 && w0 + w < words && run + 32 * (w0 + w) + lane < pages);
          if (lane == w0 + w) bits = mask;
        }
      }
    }
    int total;
    const int before = warps_before<kPageThreads>(warp_sum(__popc(bits)), sums, total);
    if (tid < kPageCluster) *cluster.map_shared_rank(&freed[round & 1][rank], tid) = total;
    cluster.sync();
    uint32_t at = all + before;
#pragma unroll
    for (int r = 0; r < kPageCluster; ++r) {
      const int c = freed[round & 1][r];
      if (r < rank) at += c;
      all += c;
    }
    uint32_t left = __ballot_sync(0xffffffffu, bits != 0);
    while (left) {
      const int w = __ffs(left) - 1;
      left &= left - 1;
      const uint32_t mask = __shfl_sync(0xffffffffu, bits, w), page = run + 32 * w + lane;
      if (mask >> lane & 1) {
        p.pages[at + __popc(mask & ((1u << lane) - 1))] = (int32_t)page;
        p.shares[page] = 0;
      }
      at += __popc(mask);
    }
  }
  for (uint32_t i = all + rank * kPageThreads + tid; i < pages; i += kPageCluster * kPageThreads) p.pages[i] = -1;
  if (rank == 0 && tid == 0) p.count[0] = (int32_t)all;
}

// ---- compact ----
//
// U pages are held.  Those at U and behind move to the places below U that nobody
// holds; there are as many of the one as of the other, and both go in ascending
// order.  A cluster of eight CTAs keeps a bit a page in distributed shared memory,
// an eighth each: marks, counts and places need its barriers and no other memory.
// A second kernel moves the rows and renames the tables' entries: no page is both
// read and written.  8 requests of up to 512 tokens 8.7 us; 72 MB to move, 31.8 us, 8 of
// them the list's.
struct CompactParams {
  const int32_t *cached, *table;
  int32_t* table_out;
  int64_t table_stride, table_out_stride, max_pages;
  const int32_t* shares;
  int32_t *shares_out, *page_map, *used;
  PageCache cache;
  int words;  // of 32 pages, of a CTA
  int B, page;
  int* status;
};

__global__ void __launch_bounds__(kPageThreads) kda_latent_compact_kernel(const CompactParams p) {
  extern __shared__ uint32_t held_words[];  // [words] a bit a page of this CTA's eighth
  __shared__ int sums[kPageThreads / 32 + 1];
  __shared__ int counts[kPageCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster.block_rank();
  const uint32_t pages = (uint32_t)p.cache.num_pages, eighth = 32 * (uint32_t)p.words;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  for (int w = tid; w < p.words; w += kPageThreads) held_words[w] = 0;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  int bad = 0;
  for (int b = tid; b < p.B; b += kPageThreads) {
    const int len = p.cached[b];
    bad |= len < 0 || len > p.max_pages * p.page;
  }
  bad = __syncthreads_or(bad);
  if (bad) {  // (every CTA of the cluster finds the same)
    for (uint32_t i = rank * kPageThreads + tid; i < pages; i += kPageCluster * kPageThreads) {
      p.page_map[i] = (int32_t)i;
      p.shares_out[i] = p.shares[i];
    }
    if (rank == 0 && tid == 0) {
      atomicExch(p.status, KDA_ERR_BAD_LENGTHS);
      p.used[0] = (int32_t)pages;
    }
    return;
  }
  cluster.sync();
  {  // warps take equal parts of rows
    const int warps = kPageCluster * kPageThreads / 32;
    const int part = (int)min((p.B * p.max_pages / warps / 128 + 1) * 128, (int64_t)1 << 30);
    const int parts = (int)(((uint32_t)p.max_pages + part - 1) / part);  // (parts * B is at most about the warps and B)
    for (int i = rank * (kPageThreads / 32) + warp; i < parts * p.B; i += warps) {
      const int b = i / parts;
      const int32_t* ids = p.table + b * p.table_stride;
      const uint32_t j0 = (uint32_t)(i - b * parts) * part;
      const uint32_t end = min((uint32_t)pages_of(p.cached[b], p.page), j0 + part);
      for (uint32_t j = j0 + lane; j < end; j += 128) {
        int id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) id[k] = j + 32 * k < end ? ids[j + 32 * k] : INT32_MIN;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (id[k] >= 0 && (uint32_t)id[k] < pages) {
            const uint32_t owner = (uint32_t)id[k] / eighth, in = (uint32_t)id[k] - owner * eighth;
            atomicOr(cluster.map_shared_rank(held_words + (in >> 5), (int)owner), 1u << (in & 31));
          } else if (j + 32 * k < end) {
            atomicExch(p.status, KDA_ERR_BAD_PAGE);
          }
        }
      }
    }
  }
  cluster.sync();
  // a warp a run of words; held pages before it, first of this CTA's
  const int run = (p.words + kPageThreads / 32 - 1) / (kPageThreads / 32);
  const int w0 = min(p.words, warp * run), w1 = min(p.words, w0 + run);
  int n = 0, total;
  for (int w = w0 + lane; w < w1; w += 32) n += __popc(held_words[w]);
  uint32_t before = warps_before<kPageThreads>(warp_sum(n), sums, total);
  if (tid < kPageCluster) *cluster.map_shared_rank(counts + rank, tid) = total;
  cluster.sync();
  uint32_t used = 0, below = 0;  // U, and the held pages below place U
#pragma unroll
  for (int r = 0; r < kPageCluster; ++r) {
    if (r < rank) before += counts[r];
    used += counts[r];
  }
  const uint32_t owner = used / eighth;  // the CTA of place U (none where all pages are held and fill their eighths)
  for (uint32_t r = 0; r < owner; ++r) below += counts[r];
  n = 0;
  if (owner < kPageCluster) {
    const uint32_t* words = cluster.map_shared_rank(held_words, (int)owner);
    const uint32_t in = used - owner * eighth;
    for (uint32_t w = tid; 32 * w < in; w += kPageThreads)
      n += __popc(words[w] & (in - 32 * w >= 32 ? 0xffffffffu : (1u << (in - 32 * w)) - 1));
  }
  warps_before<kPageThreads>(warp_sum(n), sums, total);
  below += total;
  // the places, listed in the map's first entries, which get their values at the end
  auto each = [&](auto body) {
    uint32_t at = before;  // held pages before the word
    for (int w = w0; w < w1; ++w) {
      const uint32_t mask = held_words[w], page = rank * eighth + 32 * w + lane;
      if (page < pages) body(page, mask >> lane & 1, at + __popc(mask & ((1u << lane) - 1)));
      at += __popc(mask);
    }
  };
  each([&](uint32_t page, bool held, uint32_t k) {
    if (!held && page < used) p.page_map[page - k] = (int32_t)page;
  });
  if (rank == 0 && tid == 0) p.used[0] = (int32_t)used;
  cluster.sync();
  // (shares_out may be shares: a mover's count is taken and cleared by one thread)
  each([&](uint32_t page, bool held, uint32_t k) {
    if (page < used) {
      if (held) p.shares_out[page] = p.shares[page];
      return;
    }
    int to = -1;
    if (held) {
      to = __ldcg(p.page_map + (k - below));
      p.shares_out[to] = p.shares[page];
    }
    p.page_map[page] = to;
    p.shares_out[page] = 0;
  });
  cluster.sync();
  each([&](uint32_t page, bool held, uint32_t) {
    if (page < used) p.page_map[page] = held ? (int32_t)page : -1;
  });
}

__global__ void __launch_bounds__(kCopyThreads) kda_latent_move_kernel(const CompactParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int64_t used = p.used[0];
  const int per = p.page / kGroupRows;
  const int64_t entries = p.B * p.max_pages;
  // the tables first: they are small, and their entries are renamed while the first rows are on their way
  for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < entries; e += (int64_t)gridDim.x * kCopyThreads) {
    const int b = (int)div_pages(e, (int)p.max_pages), j = (int)(e - b * p.max_pages);
    int id = p.table[b * p.table_stride + j];
    if (p.cached[b] > 0 && j < pages_of(p.cached[b], p.page) && id >= 0 && id < p.cache.num_pages) id = p.page_map[id];
    p.table_out[b * p.table_out_stride + j] = id;
  }
  // (refused: the map is the identity, and no page lies behind U)
  copy_groups((p.cache.num_pages - used) * per, p.cache.token_stride, p.cache.token_stride, blockIdx.x, gridDim.x,
              [&](int64_t g) {
                const int64_t i = div_pages(g, per), to = p.page_map[used + i];
                CopyPlace c = {nullptr, nullptr, kGroupRows};
                return to < 0 ? c : page_group(p.cache, p.cache, used + i, to, (int)(g - i * per), p.status);
              });
}

namespace {

// Entries from which on the counts go to a kernel of their own (16 rows of 1024 entries 7.9 us in one kernel, 256 of 64
// 6.8; 256 of 256 22 in one and 12 in two).
constexpr int64_t kReleaseApart = 32768;

bool al4(const void* p) { return ((uintptr_t)p & 3) == 0; }

PageCache page_cache(const kda_latent_cache& c) {
  return {static_cast<uint16_t*>(c.data), c.num_pages, c.page_stride, c.token_stride};
}

// Table sizes that all calls check alike.
int check_table(int64_t rows, int64_t max_pages, int64_t stride, const void* table) {
  if (rows < 0 || rows > kMaxPlanRequests || max_pages < 0 || max_pages > INT32_MAX || stride < max_pages)
    return KDA_ERR_SHAPE;
  if (rows > 0 && max_pages > 0 && !table) return KDA_ERR_NULL_ARG;
  return al4(table) ? KDA_OK : KDA_ERR_ALIGNMENT;
}

unsigned copy_ctas(int64_t groups) { return (unsigned)std::min<int64_t>(std::max<int64_t>(1, (groups + 3) / 4), 152 * 6); }

int check_compact(const kda_latent_compact_args* a) {
  if (!a) return KDA_ERR_NULL_ARG;
  int rc = check_table(a->B, a->max_pages, a->table_stride, a->block_table);
  if (rc != KDA_OK) return rc;
  rc = check_table(a->B, a->max_pages, a->table_out_stride, a->block_table_out);
  if (rc != KDA_OK) return rc;
  rc = latent_check_cache(&a->cache);
  if (rc != KDA_OK) return rc;
  if (a->cache.num_pages > KDA_LATENT_COMPACT_PAGES) return KDA_ERR_SHAPE;
  if (!a->pages_used || (a->B > 0 && !a->cached_lens) ||
      (a->cache.num_pages > 0 && (!a->shares || !a->shares_out || !a->page_map)))
    return KDA_ERR_NULL_ARG;
  if (!al4(a->cached_lens) || !al4(a->shares) || !al4(a->shares_out) || !al4(a->page_map) || !al4(a->pages_used))
    return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" int kda_latent_copy(const kda_latent_copy_args* a, void* stream) {
  if (!a) return KDA_ERR_NULL_ARG;
  if (a->n < 0 || a->n > INT32_MAX) return KDA_ERR_SHAPE;
  int rc = latent_check_cache(&a->src);
  if (rc == KDA_OK) rc = latent_check_cache(&a->dst);
  if (rc != KDA_OK) return rc;
  if (a->src.page_size != a->dst.page_size) return KDA_ERR_PAGE_SIZE;
  if (a->n > 0 && (!a->src_pages || !a->dst_pages)) return KDA_ERR_NULL_ARG;
  if (!al4(a->src_pages) || !al4(a->dst_pages)) return KDA_ERR_ALIGNMENT;
  if (a->n == 0) return KDA_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = status_slot(s);
  if (!status) return KDA_ERR_LAUNCH;
  const CopyParams p{page_cache(a->src), page_cache(a->dst), a->src_pages, a->dst_pages, a->n, (int)a->src.page_size, status};
  const unsigned ctas = copy_ctas(a->n * (a->src.page_size / kGroupRows));
  return launch_overlapped(kda_latent_copy_kernel, dim3(ctas), kCopyThreads, 0, s, 1, p) ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" int kda_latent_fork(const kda_latent_fork_args* a, void* stream) {
  if (!a) return KDA_ERR_NULL_ARG;
  int rc = check_table(a->B, a->max_pages, a->table_stride, a->block_table);
  if (rc != KDA_OK) return rc;
  if (a->F < 0 || a->F > kMaxPlanRequests || a->num_free < 0 || a->num_free > INT32_MAX) return KDA_ERR_SHAPE;
  rc = latent_check_cache(&a->cache);
  if (rc != KDA_OK) return rc;
  if (!a->pages_taken || (a->B > 0 && (!a->cached_lens || !a->seq_lens)) || (a->F > 0 && (!a->parents || !a->children)) ||
      (a->num_free > 0 && !a->free_pages) || (a->cache.num_pages > 0 && !a->shares))
    return KDA_ERR_NULL_ARG;
  if (!al4(a->parents) || !al4(a->children) || !al4(a->fork_lens) || !al4(a->cached_lens) || !al4(a->free_pages) ||
      !al4(a->shares) || !al4(a->seq_lens) || !al4(a->pages_taken))
    return KDA_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = status_slot(s);
  if (!status) return KDA_ERR_LAUNCH;
  ForkParams p{a->parents, a->children, a->fork_lens, a->cached_lens, a->block_table, a->table_stride, a->max_pages,
               a->free_pages, a->num_free, a->shares, page_cache(a->cache), a->seq_lens, a->pages_taken, (int)a->F,
               (int)a->B, (int)a->cache.page_size, 1, status};
  // CTAs a fork: one for 32 rows of its last page, as long as all are on the GPU at once
  const int64_t forks = std::max<int64_t>(1, a->F);
  p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(152 * 4 / forks, (a->cache.page_size + 31) / 32));
  return launch_overlapped(kda_latent_fork_kernel, dim3((unsigned)(forks * p.parts)), kCopyThreads,
                           (size_t)(a->B + 31) / 32 * 4, s, 1, p)
             ? KDA_OK
             : KDA_ERR_LAUNCH;
}

extern "C" int kda_latent_release(const kda_latent_release_args* a, void* stream) {
  if (!a) return KDA_ERR_NULL_ARG;
  const int rc = check_table(a->B, a->max_pages, a->table_stride, a->block_table);
  if (rc != KDA_OK) return rc;
  if (a->F < 0 || a->F > kMaxPlanRequests || a->num_pages < 0 || a->num_pages > INT32_MAX) return KDA_ERR_SHAPE;
  if (a->page_size <= 0 || a->page_size % 8 || a->page_size > (1 << 24)) return KDA_ERR_PAGE_SIZE;
  if (!a->count || (a->B > 0 && (!a->cached_lens || !a->seq_lens)) || (a->F > 0 && !a->rows) ||
      (a->num_pages > 0 && (!a->shares || !a->pages)))
    return KDA_ERR_NULL_ARG;
  if (!al4(a->rows) || !al4(a->keep_lens) || !al4(a->cached_lens) || !al4(a->shares) || !al4(a->seq_lens) ||
      !al4(a->pages) || !al4(a->count))
    return KDA_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = status_slot(s);
  if (!status) return KDA_ERR_LAUNCH;
  const ReleaseParams p{a->rows, a->keep_lens, a->cached_lens, a->block_table, a->table_stride, a->max_pages, a->shares,
                        a->num_pages, a->seq_lens, a->pages, a->count, (int)a->F, (int)a->B, (int)a->page_size, status};
  const size_t smem = release_smem(a->B, a->F);
  const bool apart = a->F * a->max_pages > kReleaseApart;
  if (apart) {
    const int64_t ctas = std::min<int64_t>((a->F * a->max_pages + 1023) / 1024, 152);
    if (!launch_overlapped(kda_latent_release_counts_kernel, dim3((unsigned)ctas), kPageThreads, smem, s, 1, p))
      return KDA_ERR_LAUNCH;
  }
  return launch_overlapped(kda_latent_release_kernel, dim3(kPageCluster), kPageThreads, smem, s, kPageCluster, p, !apart)
             ? KDA_OK
             : KDA_ERR_LAUNCH;
}

extern "C" int kda_latent_compact(const kda_latent_compact_args* a, void* stream) {
  const int rc = check_compact(a);
  if (rc != KDA_OK) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = status_slot(s);
  if (!status) return KDA_ERR_LAUNCH;
  const int64_t pages = a->cache.num_pages;
  CompactParams p{a->cached_lens, a->block_table, a->block_table_out, a->table_stride, a->table_out_stride, a->max_pages,
                  a->shares, a->shares_out, a->page_map, a->pages_used, page_cache(a->cache),
                  (int)std::max<int64_t>(1, (pages + 32 * kPageCluster - 1) / (32 * kPageCluster)), (int)a->B,
                  (int)a->cache.page_size, status};
  const size_t smem = (size_t)p.words * 4;
  if (smem > 40 * 1024) {
    static std::atomic<int> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_LAUNCH;
    if (!set[dev].load()) {
      if (cudaFuncSetAttribute(kda_latent_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               KDA_LATENT_COMPACT_PAGES / (8 * kPageCluster)) != cudaSuccess)
        return KDA_ERR_LAUNCH;
      set[dev].store(1);
    }
  }
  if (!launch_overlapped(kda_latent_compact_kernel, dim3(kPageCluster), kPageThreads, smem, s, kPageCluster, p))
    return KDA_ERR_LAUNCH;
  // as many CTAs as half of the pages could need, the most that can move
  const int64_t groups = pages / 2 * (a->cache.page_size / kGroupRows);
  const int64_t entries = (a->B * a->max_pages + kCopyThreads - 1) / kCopyThreads;
  const unsigned ctas = std::max(copy_ctas(groups), (unsigned)std::min<int64_t>(entries, 152));
  return launch_overlapped(kda_latent_move_kernel, dim3(ctas), kCopyThreads, 0, s, 1, p) ? KDA_OK : KDA_ERR_LAUNCH;
}
