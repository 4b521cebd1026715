// Parameter blocks and launch entry points of the latent-attention calls
// (include/kda_latent.h).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda_latent.h"

namespace kda {

constexpr int kLat = 512;           // latent values of a cache row
constexpr int kLatPe = 64;          // shared key values
constexpr int kLatRow = kLat + kLatPe;
constexpr int kQkDim = 192;         // expanded query / key channels
constexpr int kNope = 128;          // the heads' own key channels
constexpr int kVDim = 128;          // expanded value channels
constexpr int kMaxPlanRequests = 16384;

struct DecodeParams {
  const uint16_t* q;                // bf16 [B, R * H, 576]
  const uint16_t* cache;
  int64_t num_pages, page_size, page_stride, token_stride;
  const int32_t* table;
  int64_t table_stride, max_pages;
  const int32_t* lens;
  float scale_log2;                 // scale * log2(e)
  uint16_t* out;                    // bf16 [B, R * H, 512]
  float* lse;                       // [B, R * H] or nullptr
  int B, R, H;
  unsigned char* ws;
  int* status;
};

// A block of query rows of a packed sequence.
struct PrefillItem {
  int q0, k0;                       // first query and key of the sequence
  int lq, lk;                       // its lengths
  int r0;                           // first row of the block within it
  int tiles, start;                 // split calls: its key tiles, and the cost of the blocks before it
  int pad;
};
static_assert(sizeof(PrefillItem) == 32, "read as two 16-byte pieces");

struct PrefillParams {
  const uint16_t *q, *k, *k_pe, *v;
  int64_t q_st, q_sh, k_st, k_sh, pe_st, v_st, v_sh;  // element strides: token, head
  float scale_log2;
  uint16_t* out;                    // bf16 [tokens, H, 128]
  float* lse;                       // [tokens, H] or nullptr
  const int64_t *cu_q, *cu_k;       // [N + 1] or nullptr (dense)
  const PrefillItem* items;         // query blocks in the order of their work (packed only)
  int32_t* count;                   // their number, how many were taken by counter, their cost (packed only)
  int64_t B, Tq, Tk, N;
  int H;
  int causal;
  int pairs;                        // CTA pairs and items of 2 kPrefillRows rows
  float* part;                      // partial rows of a split call, or nullptr
  int* status;
};

// Whether `rows` queries of `sequences` sequences go to CTA pairs.
bool prefill_pairs(int64_t rows, int64_t sequences, bool packed);

// Bytes that a split call needs for its partial rows; 0: it is not split.
size_t prefill_split_bytes(const PrefillParams& p);
constexpr int64_t kPrefillSplitKeys = KDA_LATENT_SPLIT_KEYS;  // fewer keys are never split

constexpr int kPreKeys = 128;     // keys of a tile
constexpr int kPreItemCost = 2;   // what an item costs beside its key tiles, in tiles
// Key tiles of the block of 2 `tile_rows` rows from r0 on of a sequence: of its first and its second tile.
__host__ __device__ __forceinline__ void block_tiles(int lq, int lk, int causal, int r0, int tile_rows, int& n0, int& n1) {
  int n[2];
  for (int t = 0; t < 2; ++t) {
    const int first = r0 + t * tile_rows;
    const int last = (lq < first + tile_rows ? lq : first + tile_rows) - 1;
    const int seen = !causal || last + lk - lq + 1 > lk ? lk : last + lk - lq + 1;
    n[t] = first < lq && seen > 0 ? (seen + kPreKeys - 1) / kPreKeys : 0;
  }
  n0 = n[0];
  n1 = n[1];
}

// Query rows of one work item of the expanded form (of single CTAs).
constexpr int kPrefillRows = 256;

// Launches a kernel whose set-up may overlap the end of the kernel before it in
// the stream; it waits (griddepcontrol.wait) before it touches memory.
// cluster: CTAs of a cluster.
template <class... P, class... A>
bool launch_overlapped(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, unsigned cluster,
                       A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess;
}

// The checks of a cache's address, sizes and strides.
int latent_check_cache(const kda_latent_cache* c);

// ---- decoding behind shared prefixes ----
constexpr int kPfxTile = 128;      // cached rows of a tile of the shared pass
constexpr int kPfxRows = 128;      // query rows of an item, a CTA pair's
// A share's cost: 4 a tile, and an item's set-up and output.
constexpr int kPfxTileCost = 4, kPfxItemCost = 6;

struct SharedHead {
  int64_t total, size;             // cost of all items, and of a share
};

// Groups of requests: group g has the requests [cu[g], cu[g + 1]).
struct SharedGroups {
  const int64_t* cu;               // [G + 1]
  const int32_t* prefix;           // [G]
  int G;
};

struct SharedParams {
  DecodeParams d;
  SharedGroups groups;
  int pairs;                       // CTA pairs of the shared pass, a share each; 0: there is none
  // workspace
  SharedHead* head;
  int64_t* line;                   // [G] cost of the items before the group's
  // fp32 rows and their lse (log2): a row's first part at its own place, those that begin
  // within a share behind them
  float *pre_part, *pre_lse;       // [B R H + pairs * kPfxRows]
  float *own_part, *own_lse;       // [B R H + CTAs * N]
  int4* split;                     // [B][blocks of N rows] what is left to join: request or -1, first and last share
                                   // of the own pass, group or -1
  int own_n, own_row_blocks;       // N and the blocks of N rows
};

// Tokens of a group's prefix that are shared: whole tiles, of groups of two and more.
__device__ __forceinline__ int shared_tokens(int64_t first, int64_t end, int64_t prefix, int64_t cap) {
  const int64_t len = prefix < 0 ? 0 : (prefix > cap ? cap : prefix);
  return end - first < 2 ? 0 : (int)(len / kPfxTile * kPfxTile);
}
// Whether all new tokens of a request see the shared ones.
__device__ __forceinline__ bool sees_shared(int len, int64_t cap, int R, int tokens) {
  const int64_t n = len < 0 ? 0 : (len > cap ? cap : len);
  return n - (R - 1) >= tokens;
}
// a / b of numbers that are not negative, in 32 bits where they fit (a 64-bit division takes some 100 instructions)
__device__ __forceinline__ int64_t div_costs(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Cost of an item, and the share that holds tile t of the one that begins at `item` of the line.
__device__ __forceinline__ int64_t prefix_item_cost(int tokens) {
  return kPfxItemCost + (int64_t)(tokens / kPfxTile) * kPfxTileCost;
}
__device__ __forceinline__ int64_t prefix_share(int64_t item, int t, int64_t size) {
  return div_costs(item + kPfxItemCost + (int64_t)t * kPfxTileCost, size);
}
// The parts of a row of a group in the shared pass: how many, and the place of the second.
__device__ __forceinline__ int prefix_parts(int64_t line, int64_t size, int tokens, int row, int64_t all, int64_t& second) {
  const int64_t item = line + row / kPfxRows * prefix_item_cost(tokens);
  const int64_t first = prefix_share(item, 0, size);
  second = all + (first + 1) * kPfxRows + row % kPfxRows;
  return (int)(prefix_share(item, tokens / kPfxTile - 1, size) - first) + 1;
}

size_t shared_workspace_bytes(const DecodeParams& p, int64_t G);
bool launch_latent_shared(const DecodeParams& p, const SharedGroups& groups, cudaStream_t s);
// Its parts: the shared pass; a request's own tokens (sizes first, then the launch).
bool launch_latent_prefix(const SharedParams& p, cudaStream_t s);
struct OwnLayout {
  int n, row_blocks, ctas;
};
OwnLayout own_layout(const DecodeParams& p);
bool launch_latent_own(const SharedParams& p, cudaStream_t s);
int device_sm_count();

size_t decode_workspace_bytes(const DecodeParams& p);
// false: a tensor map could not be made or a launch attribute set (nothing launched)
bool launch_latent_decode(const DecodeParams& p, cudaStream_t s);
bool launch_latent_prefill(const PrefillParams& p, cudaStream_t s);

}  // namespace kda
