// Latent attention for serving: host entry points (include/kda_latent.h), the
// kernel that plans block tables and slot maps, and the one that writes new
// rows into the paged cache.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/kda_latent.h"
#include "kda_common.cuh"
#include "kda_kernels.cuh"
#include "kda_latent.cuh"

namespace kda {

// ---- block tables and slot maps ----
//
// With need_b = ceil((c_b + n_b) / P) - ceil(c_b / P), request b takes the
// entries [F_b, F_b + need_b) of free_pages, F the exclusive prefix of need,
// and its new tokens the packed range [O_b, O_b + n_b), O that of n.  Every
// CTA forms both prefixes for itself in shared memory (they are a few
// kilobytes, and a second launch or a wait between CTAs would cost more than
// the scan) and then writes its share of the tokens and pages, finding an
// element's request by bisection of the prefix.  A token's page comes from the
// table where the request held it before and straight from free_pages where it
// is new, so no CTA reads what another writes.  Bound by launch and two rounds of
// latency: 4.0 us for a decoding step of 256 requests, 4.4 us for packed prompts
// that write 1.2 MB of slots and tables.
constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 1024;  // tokens of slot_map per CTA

struct PlanParams {
  const int32_t *cached, *fresh;
  int32_t* table;
  int64_t table_stride;
  const int32_t* free_pages;
  int32_t* seq_lens;
  int64_t* cu;
  int64_t* slots;
  int32_t* taken;
  int B;
  int64_t max_pages, num_free, T;
  int page;
  int* status;
};

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// largest b in [0, n) with off[b] <= x (off ascending, off[0] = 0)
__device__ __forceinline__ int find_request(const int32_t* off, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kda_latent_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  int32_t* tok = plan_smem;            // [B + 1] prefix of new tokens
  int32_t* pag = plan_smem + p.B + 1;  // [B + 1] prefix of pages taken
  __shared__ int64_t sums[2][kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t P = p.page;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  int64_t carry_t = 0, carry_p = 0;
  int bad = 0;
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    int64_t n = 0, need = 0;
    if (b < p.B) {
      const int64_t c = p.cached[b];
      n = p.fresh[b];
      const int64_t pages = (c + n + P - 1) / P;
      if (c < 0 || n < 0 || c + n > INT32_MAX || pages > p.max_pages) {
        bad = 1;
        n = 0;
      } else {
        need = pages - (c + P - 1) / P;
      }
    }
    const int64_t st = warp_scan(n, lane), sp = warp_scan(need, lane);
    if (lane == 31) {
      sums[0][warp] = st;
      sums[1][warp] = sp;
    }
    __syncthreads();
    int64_t before_t = carry_t, before_p = carry_p;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const int64_t a = sums[0][w], g = sums[1][w];
      if (w < warp) {
        before_t += a;
        before_p += g;
      }
      carry_t += a;
      carry_p += g;
    }
    if (b < p.B) {  // (sums beyond 2^31 - 1 are refused below: T and num_free are below it)
      tok[b] = (int32_t)(before_t + st - n);
      pag[b] = (int32_t)(before_p + sp - need);
    }
    __syncthreads();  // sums are read
  }
  bad = __syncthreads_or(bad);
  const bool no_room = carry_t > p.T, no_pages = carry_p > p.num_free;
  const bool refused = bad || no_room || no_pages;
  if (blockIdx.x == 0) {
    if (tid == 0) {
      if (refused && p.status) atomicExch(p.status, bad || no_room ? KDA_ERR_BAD_LENGTHS : KDA_ERR_NO_PAGES);
      p.cu[p.B] = refused ? 0 : carry_t;
      p.taken[0] = refused ? 0 : (int32_t)carry_p;
    }
    for (int b = tid; b < p.B; b += kPlanThreads) {
      p.cu[b] = refused ? 0 : tok[b];
      p.seq_lens[b] = p.cached[b] + (refused ? 0 : p.fresh[b]);
    }
  }
  const int64_t total_t = refused ? 0 : carry_t, total_p = refused ? 0 : carry_p;
  for (int64_t k = (int64_t)blockIdx.x * kPlanThreads + tid; k < total_p; k += (int64_t)gridDim.x * kPlanThreads) {
    const int b = find_request(pag, p.B, (int)k);
    const int64_t held = (p.cached[b] + P - 1) / P;
    p.table[b * p.table_stride + held + (k - pag[b])] = p.free_pages[k];
  }
  const int64_t t1 = min(p.T, ((int64_t)blockIdx.x + 1) * kPlanTokens);
  for (int64_t t = (int64_t)blockIdx.x * kPlanTokens + tid; t < t1; t += kPlanThreads) {
    int64_t slot = -1;
    if (t < total_t) {
      const int b = find_request(tok, p.B, (int)t);
      const int cached = p.cached[b];
      const int pos = cached + (int)(t - tok[b]);
      const int held = (int)(((int64_t)cached + P - 1) / P);
      const int at = pos / p.page;
      const int64_t page = at < held ? p.table[b * p.table_stride + at] : p.free_pages[pag[b] + at - held];
      slot = page * P + (pos - at * p.page);
    }
    p.slots[t] = slot;
  }
}

// ---- rows into the cache ----
//
// A warp one or two tokens at a time: lane l holds a token's latent values 8 l ..
// and 256 + 8 l .. (two 16-byte pieces), so the row is read and written in whole
// 512-byte requests, the mean square is one warp reduction, and a row passes
// through the SM once.  Bound by HBM: 2 x 1152 bytes a token; 131072 tokens in
// 52.4 us, 5.8 TB/s of rows in and out; 256 tokens in 2.3 us, the latency of a launch.
struct AppendParams {
  const uint16_t *c, *pe;
  int64_t c_st, pe_st;
  const int64_t* slots;
  uint16_t* cache;
  int64_t num_pages, page_stride, token_stride;
  int page;
  const float* w;
  float eps;
  int64_t T;
  int* status;
};

template <bool kNorm, int kAppendTokens>
__global__ void __launch_bounds__(256) kda_latent_append_kernel(AppendParams p) {
  __shared__ __align__(16) float w[kLat];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (kNorm) {
    for (int i = threadIdx.x; i < kLat; i += 256) w[i] = p.w[i];
    __syncthreads();
  }
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * 8 * kAppendTokens;
  for (int64_t t0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kAppendTokens; t0 < p.T; t0 += step) {
    int64_t slot[kAppendTokens];
    uint4 x[kAppendTokens][2], pe[kAppendTokens];
#pragma unroll
    for (int k = 0; k < kAppendTokens; ++k) {
      const int64_t t = t0 + k;
      slot[k] = -1;
      if (t >= p.T) continue;
      slot[k] = p.slots[t];
      const uint4* c = reinterpret_cast<const uint4*>(p.c + t * p.c_st);
      x[k][0] = __ldcs(c + lane);
      x[k][1] = __ldcs(c + 32 + lane);
      if (lane < 8) pe[k] = __ldcs(reinterpret_cast<const uint4*>(p.pe + t * p.pe_st) + lane);
    }
#pragma unroll
    for (int k = 0; k < kAppendTokens; ++k) {
      if (slot[k] < 0) continue;  // (the same for the whole warp)
      const int64_t page = (slot[k] >> 31) == 0 ? (int64_t)((uint32_t)slot[k] / (uint32_t)p.page) : slot[k] / p.page;
      if (page >= p.num_pages) {
        if (lane == 0 && p.status) atomicExch(p.status, KDA_ERR_BAD_PAGE);
        continue;
      }
      if (kNorm) {
        float f[16], sq = 0.f;
        const uint32_t r[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = unpack_bf16(r[i]);
          f[2 * i] = v.x;
          f[2 * i + 1] = v.y;
          sq += v.x * v.x + v.y * v.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        const float rs = rsqrtf(sq * (1.0f / kLat) + p.eps);
        uint32_t y[8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float4 v = *reinterpret_cast<const float4*>(w + (h >> 1) * 256 + 8 * lane + (h & 1) * 4);
          y[2 * h] = pack_bf16(f[4 * h] * rs * v.x, f[4 * h + 1] * rs * v.y);
          y[2 * h + 1] = pack_bf16(f[4 * h + 2] * rs * v.z, f[4 * h + 3] * rs * v.w);
        }
        x[k][0] = make_uint4(y[0], y[1], y[2], y[3]);
        x[k][1] = make_uint4(y[4], y[5], y[6], y[7]);
      }
      uint4* dst = reinterpret_cast<uint4*>(p.cache + page * p.page_stride + (slot[k] - page * p.page) * p.token_stride);
      dst[lane] = x[k][0];
      dst[32 + lane] = x[k][1];
      if (lane < 8) dst[64 + lane] = pe[k];
    }
  }
}

namespace {

bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }
bool al(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A token stride of rows of `width` elements: whole 16-byte pieces, rows apart.
bool stride_ok(int64_t st, int64_t width) { return st >= width && st % 8 == 0 && st <= ((int64_t)1 << 38); }

int check_cache(const kda_latent_cache& c) {
  if (!c.data && c.num_pages > 0) return KDA_ERR_NULL_ARG;
  if (c.num_pages < 0 || c.num_pages > INT32_MAX) return KDA_ERR_SHAPE;
  if (c.page_size <= 0 || c.page_size % 8 || c.page_size > (1 << 24)) return KDA_ERR_PAGE_SIZE;
  if (!al16(c.data)) return KDA_ERR_ALIGNMENT;
  if (!stride_ok(c.token_stride, kLatRow) ||
      !stride_ok(c.page_stride, (c.page_size - 1) * c.token_stride + kLatRow))
    return KDA_ERR_STRIDE;
  return KDA_OK;
}

int check_decode(const kda_latent_decode_args* a) {
  if (!a) return KDA_ERR_NULL_ARG;
  if (a->B < 0 || a->R < 0 || a->H < 0 || a->max_pages < 0) return KDA_ERR_SHAPE;
  if (a->B > (1 << 20) || a->R > 4096 || a->H > 4096 || a->R * a->H > (1 << 16)) return KDA_ERR_SHAPE;
  if (a->max_pages > INT32_MAX || a->table_stride < a->max_pages) return KDA_ERR_SHAPE;
  const int rc = check_cache(a->cache);
  if (rc != KDA_OK) return rc;
  if (a->max_pages * a->cache.page_size > INT32_MAX - 127) return KDA_ERR_SHAPE;  // tile ends stay in 32 bits
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return KDA_ERR_SCALE;
  if (a->B * a->R * a->H > 0 && (!a->q || !a->out || !a->seq_lens || (a->max_pages > 0 && !a->block_table)))
    return KDA_ERR_NULL_ARG;
  if (!al16(a->q) || !al16(a->out) || !al(a->lse, 4) || !al(a->block_table, 4) || !al(a->seq_lens, 4))
    return KDA_ERR_ALIGNMENT;
  return KDA_OK;
}

DecodeParams decode_params(const kda_latent_decode_args* a) {
  DecodeParams p;
  p.q = static_cast<const uint16_t*>(a->q);
  p.cache = static_cast<const uint16_t*>(a->cache.data);
  p.num_pages = a->cache.num_pages;
  p.page_size = a->cache.page_size;
  p.page_stride = a->cache.page_stride;
  p.token_stride = a->cache.token_stride;
  p.table = a->block_table;
  p.table_stride = a->table_stride;
  p.max_pages = a->max_pages;
  p.lens = a->seq_lens;
  p.scale_log2 = a->scale * kLog2e;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.B = (int)a->B;
  p.R = (int)a->R;
  p.H = (int)a->H;
  p.ws = nullptr;
  p.status = nullptr;
  return p;
}

// Query blocks of packed sequences: at most one a sequence more than the rows fill.
int64_t prefill_blocks(const kda_latent_prefill_args* a) { return a->Tq / kPrefillRows + a->N; }

int check_prefill(const kda_latent_prefill_args* a) {
  if (!a) return KDA_ERR_NULL_ARG;
  if (a->B < 0 || a->Tq < 0 || a->Tk < 0 || a->H < 0 || a->N < 0 || a->H > 65535) return KDA_ERR_SHAPE;
  if (a->flags & ~KDA_LATENT_CAUSAL) return KDA_ERR_GATE_FLAGS;
  if ((a->cu_seqlens_q == nullptr) != (a->cu_seqlens_k == nullptr)) return KDA_ERR_NULL_ARG;
  if (a->cu_seqlens_q) {
    if (a->B != 1) return KDA_ERR_VARLEN_BATCH;
    if (a->N == 0 && (a->Tq > 0 || a->Tk > 0)) return KDA_ERR_BAD_SEQLENS;  // offsets that cannot end at T
  } else if (a->N != a->B) {
    return KDA_ERR_SHAPE;
  }
  const int64_t most = INT32_MAX / 2;
  if (a->N > (1 << 22) || a->Tq > most || a->Tk > most || (a->B > 0 && (a->Tq > most / a->B || a->Tk > most / a->B)))
    return KDA_ERR_SHAPE;
  // (packed sequences may be empty: their blocks and heads are counted in 32 bits)
  if (a->cu_seqlens_q && prefill_blocks(a) * a->H > INT32_MAX) return KDA_ERR_SHAPE;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return KDA_ERR_SCALE;
  const bool queries = a->B * a->Tq * a->H > 0, keys = a->B * a->Tk * a->H > 0;
  if (queries && (!a->q || !a->out)) return KDA_ERR_NULL_ARG;
  if (queries && keys && (!a->k || !a->k_pe || !a->v)) return KDA_ERR_NULL_ARG;
  if (!al16(a->q) || !al16(a->k) || !al16(a->k_pe) || !al16(a->v) || !al16(a->out) || !al(a->lse, 4) ||
      !al(a->cu_seqlens_q, 8) || !al(a->cu_seqlens_k, 8))
    return KDA_ERR_ALIGNMENT;
  if (queries && (!stride_ok(a->q_stride_t, kQkDim) || !stride_ok(a->q_stride_h, kQkDim))) return KDA_ERR_STRIDE;
  if (queries && keys &&
      (!stride_ok(a->k_stride_t, kNope) || !stride_ok(a->k_stride_h, kNope) || !stride_ok(a->k_pe_stride_t, kLatPe) ||
       !stride_ok(a->v_stride_t, kVDim) || !stride_ok(a->v_stride_h, kVDim)))
    return KDA_ERR_STRIDE;
  return KDA_OK;
}

// The sizes and the form of a call.
PrefillParams prefill_shape(const kda_latent_prefill_args* a) {
  PrefillParams p = {};
  p.cu_q = a->cu_seqlens_q;
  p.cu_k = a->cu_seqlens_k;
  p.B = a->B;
  p.Tq = a->Tq;
  p.Tk = a->Tk;
  p.N = a->N;
  p.H = (int)a->H;
  p.causal = (a->flags & KDA_LATENT_CAUSAL) ? 1 : 0;
  // (shares of a split call are even whatever the order of the items)
  p.pairs = prefill_pairs(a->B * a->Tq, a->N, false) ? 1 : 0;
  if (a->cu_seqlens_q && p.pairs && prefill_split_bytes(p) == 0) p.pairs = prefill_pairs(a->Tq, a->N, true) ? 1 : 0;
  return p;
}

// Packed calls: the counts and the list of blocks; then a split call's partial rows.
size_t prefill_list_bytes(const kda_latent_prefill_args* a) {
  return a->cu_seqlens_q ? 256 + ((size_t)prefill_blocks(a) * sizeof(PrefillItem) + 255) / 256 * 256 : 0;
}
size_t prefill_workspace(const kda_latent_prefill_args* a) {
  return prefill_list_bytes(a) + prefill_split_bytes(prefill_shape(a));
}

}  // namespace

// The query blocks of packed sequences, by a counting sort over classes of equal
// work (a sixteenth of an octave from 32 key tiles on).  Single CTAs take them as
// they come: the sequences with most keys first, the blocks of each together, last
// block first (keys and values are then found in L2: 24 sequences of up to 2048
// tokens, 16 heads, 161 us against 165 with single blocks by their work).  Pairs take
// every grid-th: blocks with most work first, so that all end evenly.  Checks 0 =
// cu[0] <= ... <= cu[N] = T of both offset arrays first: a violation sets the
// status word and leaves no block, so nothing is written.  One block; the order
// within a class is that of the atomics, and no result depends on it.
constexpr int kWorkClasses = 352;
// (a warp scans the classes 32 at a time, all lanes in every round: a shuffle waits for lanes that have left)
static_assert(kWorkClasses % 32 == 0, "the scan over the classes needs whole warps");
// (at most 2^30 keys: 2^24 key tiles in the two query tiles of a block, and as many 64ths of a sequence)
static_assert(32 + (24 - 5) * 16 + 15 < kWorkClasses, "every number of key tiles needs a class");
__device__ __forceinline__ int work_class(int tiles) {
  if (tiles < 32) return kWorkClasses - 1 - tiles;
  const int e = 31 - __clz(tiles);
  return kWorkClasses - 1 - (32 + (e - 5) * 16 + ((tiles >> (e - 4)) & 15));
}

__global__ void __launch_bounds__(1024) kda_latent_blocks_kernel(const int64_t* cu_q, const int64_t* cu_k, int64_t N,
                                                                 int64_t Tq, int64_t Tk, int causal, int rows,
                                                                 int together, int split, PrefillItem* items,
                                                                 int32_t* count, int* status) {
  __shared__ int32_t at[kWorkClasses];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kWorkClasses; i += 1024) at[i] = 0;
  int bad = 0;
  for (int64_t n = tid; n <= N; n += 1024) {
    const int64_t a = cu_q[n], b = cu_k[n];
    bad |= (n == 0 && (a != 0 || b != 0)) || (n == N && (a != Tq || b != Tk)) || a < 0 || a > Tq || b < 0 || b > Tk;
    if (n > 0) bad |= a < cu_q[n - 1] || b < cu_k[n - 1];
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && bad && status) atomicExch(status, KDA_ERR_BAD_SEQLENS);
  // a warp a sequence, a lane a block: first counted, then placed
  for (int pass = 0; pass < 2 && !split; ++pass) {
    for (int64_t n = warp; n < N && !bad; n += 32) {
      PrefillItem it;
      it.q0 = (int)cu_q[n];
      it.lq = (int)(cu_q[n + 1] - cu_q[n]);
      it.k0 = (int)cu_k[n];
      it.lk = (int)(cu_k[n + 1] - cu_k[n]);
      it.tiles = it.start = it.pad = 0;
      if (together) {
        const int blocks = (int)(((int64_t)it.lq + rows - 1) / rows);
        int* place = &at[work_class(it.lk / 64)];
        int first = 0;
        if (lane == 0) first = atomicAdd(place, blocks);
        if (pass == 0) continue;
        first = __shfl_sync(0xffffffffu, first, 0);
        for (int j = lane; j < blocks; j += 32) {
          it.r0 = (blocks - 1 - j) * rows;
          items[first + j] = it;
        }
        continue;
      }
      for (int64_t r = (int64_t)lane * rows; r < it.lq; r += 32 * rows) {
        it.r0 = (int)r;
        int tiles = 0;
        for (int t = 0; t < 2; ++t) {
          const int first = it.r0 + t * (rows / 2), last = min(it.lq, first + rows / 2) - 1;
          if (first < it.lq) tiles += (max(0, causal ? min(it.lk, last + it.lk - it.lq + 1) : it.lk) + 127) / 128;
        }
        const int where = atomicAdd(&at[work_class(tiles)], 1);
        if (pass == 1) items[where] = it;
      }
    }
    __syncthreads();
    if (pass == 0 && warp == 0) {  // counts to first places
      int carry = 0;
      for (int i = lane; i < kWorkClasses; i += 32) {
        const int c = at[i], s = (int)warp_scan(c, lane);
        at[i] = carry + s - c;
        carry += __shfl_sync(0xffffffffu, s, 31);
      }
      if (lane == 0) {
        count[0] = carry;
        count[1] = 0;
      }
    }
    __syncthreads();
  }
  if (split && warp == 0) {
    // split calls: the blocks in order (where the line is cut, and so the sums, must not
    // depend on an atomic's), and the line of their costs
    int n = 0;
    for (int64_t base = 0; base < N && !bad; base += 32) {
      const int64_t seq = base + lane;
      PrefillItem it = {};
      if (seq < N) {
        it.q0 = (int)cu_q[seq];
        it.lq = (int)(cu_q[seq + 1] - cu_q[seq]);
        it.k0 = (int)cu_k[seq];
        it.lk = (int)(cu_k[seq + 1] - cu_k[seq]);
      }
      const int blocks = (int)(((int64_t)it.lq + rows - 1) / rows), upto = (int)warp_scan(blocks, lane);
      for (int j = 0; j < blocks; ++j) {
        it.r0 = j * rows;
        items[n + upto - blocks + j] = it;
      }
      n += __shfl_sync(0xffffffffu, upto, 31);
    }
    __syncwarp();
    if (lane == 0) count[0] = n;
    int carry = 0;
    for (int base = 0; base < n; base += 32) {
      const int e = base + lane;
      int n0 = 0, n1 = 0, cost = 0;
      if (e < n) {
        const PrefillItem it = items[e];
        block_tiles(it.lq, it.lk, causal, it.r0, rows / 2, n0, n1);
        cost = max(n0, n1) + kPreItemCost;
      }
      const int upto = (int)warp_scan(cost, lane);
      if (e < n) {
        items[e].tiles = max(n0, n1);
        items[e].start = carry + upto - cost;
      }
      carry += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) count[2] = carry;
  }
}

}  // namespace kda

using namespace kda;

extern "C" int kda_latent_plan(const kda_latent_plan_args* a, void* stream) {
  if (!a) return KDA_ERR_NULL_ARG;
  if (a->B < 0 || a->B > kMaxPlanRequests || a->max_pages < 0 || a->max_pages > INT32_MAX || a->num_free < 0 ||
      a->num_free > INT32_MAX || a->T < 0 || a->T > INT32_MAX || a->table_stride < a->max_pages)
    return KDA_ERR_SHAPE;
  if (a->page_size <= 0 || a->page_size % 8 || a->page_size > (1 << 24)) return KDA_ERR_PAGE_SIZE;
  if (!a->cu_seqlens || !a->pages_taken || (a->T > 0 && !a->slot_map) || (a->num_free > 0 && !a->free_pages) ||
      (a->B > 0 && (!a->cached_lens || !a->new_lens || !a->seq_lens || (a->max_pages > 0 && !a->block_table))))
    return KDA_ERR_NULL_ARG;
  if (!al(a->cached_lens, 4) || !al(a->new_lens, 4) || !al(a->block_table, 4) || !al(a->free_pages, 4) ||
      !al(a->seq_lens, 4) || !al(a->cu_seqlens, 8) || !al(a->slot_map, 8) || !al(a->pages_taken, 4))
    return KDA_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = status_slot(s);
  if (!status) return KDA_ERR_LAUNCH;
  PlanParams p{a->cached_lens, a->new_lens, a->block_table, a->table_stride, a->free_pages, a->seq_lens,
               a->cu_seqlens, a->slot_map, a->pages_taken, (int)a->B, a->max_pages, a->num_free, a->T,
               (int)a->page_size, status};
  const size_t smem = (size_t)(a->B + 1) * 8;
  if (smem > 40 * 1024) {
    static std::atomic<int> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KDA_ERR_LAUNCH;
    if (!set[dev].load()) {
      if (cudaFuncSetAttribute(kda_latent_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (kMaxPlanRequests + 1) * 8) != cudaSuccess)
        return KDA_ERR_LAUNCH;
      set[dev].store(1);
    }
  }
  const int64_t ctas = std::max<int64_t>(1, (a->T + kPlanTokens - 1) / kPlanTokens);
  return launch_overlapped(kda_latent_plan_kernel, dim3((unsigned)ctas), kPlanThreads, smem, s, 1, p) ? KDA_OK
                                                                                                     : KDA_ERR_LAUNCH;
}

extern "C" int kda_latent_append(const kda_latent_append_args* a, void* stream) {
  if (!a) return KDA_ERR_NULL_ARG;
  if (a->T < 0 || a->T > INT32_MAX) return KDA_ERR_SHAPE;
  const int rc = check_cache(a->cache);
  if (rc != KDA_OK) return rc;
  if (a->T > 0 && (!a->c || !a->k_pe || !a->slot_map)) return KDA_ERR_NULL_ARG;
  if (!al16(a->c) || !al16(a->k_pe) || !al(a->slot_map, 8) || !al(a->norm_weight, 4)) return KDA_ERR_ALIGNMENT;
  if (a->T > 0 && (!stride_ok(a->c_stride, kLat) || !stride_ok(a->k_pe_stride, kLatPe))) return KDA_ERR_STRIDE;
  if (a->T == 0) return KDA_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = status_slot(s);
  if (!status) return KDA_ERR_LAUNCH;
  AppendParams p{static_cast<const uint16_t*>(a->c), static_cast<const uint16_t*>(a->k_pe), a->c_stride,
                 a->k_pe_stride, a->slot_map, static_cast<uint16_t*>(a->cache.data), a->cache.num_pages,
                 a->cache.page_stride, a->cache.token_stride, (int)a->cache.page_size, a->norm_weight, a->eps, a->T,
                 status};
  // Two tokens a warp at a time keep enough bytes in flight (131072 tokens: 65.0 us
  // with one, 52.9 with two, 57.1 with four); few tokens spread over more warps.
  const int per = a->T > 8 * 152 * 4 ? 2 : 1;
  const unsigned ctas = (unsigned)std::min<int64_t>((a->T + 8 * per - 1) / (8 * per), 152 * 6);
  void (*kernel)(AppendParams) =
      a->norm_weight ? (per == 2 ? kda_latent_append_kernel<true, 2> : kda_latent_append_kernel<true, 1>)
                     : (per == 2 ? kda_latent_append_kernel<false, 2> : kda_latent_append_kernel<false, 1>);
  return launch_overlapped(kernel, dim3(ctas), 256, 0, s, 1, p) ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" size_t kda_latent_decode_workspace_bytes(const kda_latent_decode_args* a) {
  if (check_decode(a) != KDA_OK || a->B * a->R * a->H == 0) return 0;
  return decode_workspace_bytes(decode_params(a));
}

extern "C" int kda_latent_decode(const kda_latent_decode_args* a, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const int rc = check_decode(a);
  if (rc != KDA_OK) return rc;
  if (a->B * a->R * a->H == 0) return KDA_OK;
  DecodeParams p = decode_params(a);
  const size_t need = decode_workspace_bytes(p);
  if (need > 0 && (!workspace || !al(workspace, 256) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.ws = static_cast<unsigned char*>(workspace);
  p.status = status_slot(s);
  if (!p.status || !launch_latent_decode(p, s)) return KDA_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

extern "C" size_t kda_latent_prefill_workspace_bytes(const kda_latent_prefill_args* a) {
  return check_prefill(a) == KDA_OK ? prefill_workspace(a) : 0;
}

extern "C" int kda_latent_prefill(const kda_latent_prefill_args* a, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  const int rc = check_prefill(a);
  if (rc != KDA_OK) return rc;
  const size_t need = prefill_workspace(a);
  // (a dense call without one is not split)
  const bool given = a->cu_seqlens_q || workspace;
  if (given && need > 0 && (!workspace || !al(workspace, 256) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (a->N == 0 || a->H == 0 || (!a->cu_seqlens_q && a->Tq == 0)) return KDA_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* status = status_slot(s);
  if (!status) return KDA_ERR_LAUNCH;
  PrefillParams p = prefill_shape(a);
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.k_pe = static_cast<const uint16_t*>(a->k_pe);
  p.v = static_cast<const uint16_t*>(a->v);
  p.q_st = a->q_stride_t;
  p.q_sh = a->q_stride_h;
  p.k_st = a->k_stride_t;
  p.k_sh = a->k_stride_h;
  p.pe_st = a->k_pe_stride_t;
  p.v_st = a->v_stride_t;
  p.v_sh = a->v_stride_h;
  p.scale_log2 = a->scale * kLog2e;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.status = status;
  const size_t list = prefill_list_bytes(a);
  if (workspace && need > list) p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + list);
  if (a->cu_seqlens_q) {
    int32_t* count = static_cast<int32_t*>(workspace);
    PrefillItem* items = reinterpret_cast<PrefillItem*>(static_cast<unsigned char*>(workspace) + 256);
    if (!launch_overlapped(kda_latent_blocks_kernel, dim3(1), 1024, 0, s, 1, a->cu_seqlens_q, a->cu_seqlens_k, a->N, a->Tq,
                           a->Tk, p.causal, p.pairs ? 2 * kPrefillRows : kPrefillRows, !p.pairs,
                           p.part != nullptr, items, count, status))
      return KDA_ERR_LAUNCH;
    p.items = items;
    p.count = count;
  }
  if (a->Tq > 0 && !launch_latent_prefill(p, s)) return KDA_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}
