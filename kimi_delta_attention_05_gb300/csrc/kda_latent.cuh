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

size_t decode_workspace_bytes(const DecodeParams& p);
// false: a tensor map could not be made or a launch attribute set (nothing launched)
bool launch_latent_decode(const DecodeParams& p, cudaStream_t s);
bool launch_latent_prefill(const PrefillParams& p, cudaStream_t s);

}  // namespace kda
