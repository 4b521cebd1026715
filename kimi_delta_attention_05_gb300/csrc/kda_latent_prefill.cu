// Expanded latent attention: which form a call takes, and the unsplit ones.
#include "kda_latent_prefill.cuh"

namespace kda {

namespace {

// Whether and how a dense call is split: where the unsplit items' busiest CTA has
// more than a ninth more to do than a share and the join (taken as ten key tiles).
// 1024 rows behind 15360 cached, 16 heads: 180 us unsplit, 99 split; 256 behind 32768,
// 8 heads: 442 and 46; two of the first, whose 64 items nearly fill the 76 pairs: 188
// and 195, so those stay whole.  Fewer than kPrefillSplitKeys keys are not looked at,
// which spares short calls the workspace and its query; at the limit a split brings 256
// rows and 8 heads from 59.7 us to 28.5, 512 rows and 32 heads from 61.5 to 46.4.  It
// would still gain below (the same over 3000 keys: 46.5 and 28.7, 48.0 and 39.9); from
// 2048 keys down the rule splits none of these.  Packed sequences, whose lengths are on
// the device, are split where their blocks cannot fill the GPU and they have many keys on
// average (1024 rows behind up to 15360, 16 heads: 229 us unsplit, 103 split).
constexpr int kMostCtas = 512;
PrefillSplit split_of(const PrefillParams& p, int sms) {
  PrefillSplit sp = {};
  const int tile_rows = p.pairs ? 2 * kPreRows : kPreRows;
  const int64_t per = (p.Tq + 2 * tile_rows - 1) / (2 * tile_rows), bh = p.B * p.H, wide = p.pairs ? sms / 2 : sms;
  if (p.cu_q) {
    const int64_t items = (p.Tq / (2 * tile_rows) + p.N) * p.H;
    if (p.Tk >= kPrefillSplitKeys * p.N && items > 0 && items <= wide) sp.shares = (int)wide;
    return sp;
  }
  if (p.Tk < kPrefillSplitKeys || per * bh == 0 || per * bh > 3 * wide || wide > kMostCtas) return sp;
  int64_t total = 0, worst = 0;
  int64_t busy[kMostCtas] = {};
  for (int64_t back = 0, place = 0; back < per; ++back) {
    int n0, n1;
    block_tiles((int)p.Tq, (int)p.Tk, p.causal, (int)(per - 1 - back) * 2 * tile_rows, tile_rows, n0, n1);
    const int64_t cost = std::max(n0, n1) + kPreItemCost;
    total += bh * cost;
    for (int64_t x = 0; x < bh; ++x, ++place) {
      const int64_t at = place % wide, cta = (place / wide) & 1 ? wide - 1 - at : at;
      worst = std::max(worst, busy[cta] += cost);
    }
  }
  const int64_t size = std::max<int64_t>((total + wide - 1) / wide, kSplitLeast);
  if ((size + 10) * 10 > worst * 9) return sp;
  sp.size = size;
  sp.shares = (int)((total + size - 1) / size);
  return sp;
}

int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return sms;
}

size_t part_floats(const PrefillParams& p, const PrefillSplit& sp) {
  return (size_t)2 * sp.shares * (p.pairs ? 2 : 1) * kPrefillRows * kVDim;
}

}  // namespace

// Pairs halve the traffic of keys and values, but their items are twice as long and
// in a fixed order.  Packed: 12 sequences of 1167 rows on average, 32 heads, 216 us in
// single CTAs and 236 in pairs; 8 of 2547, 16 heads, 266 and 251.  Dense, where the
// items of single CTAs have a fixed order too: from 1024 rows on (16 sequences, 32 heads,
// in pairs and in single CTAs: 768 rows 138 us and 112, 1024 168 and 170, 1280 266 and 241,
// 1536 304 and 329, 2048 511 and 543, 3000 1082 and 1190; one of 8 heads 14.9 and 16.3,
// 19.1 and 19.5, 20.1 and 22.9, 24.3 and 26.1, 29.7 and 33.3, 40.8 and 46.8).
bool prefill_pairs(int64_t rows, int64_t sequences, bool packed) { return rows >= (packed ? 2048 : 1024) * sequences; }

size_t prefill_split_bytes(const PrefillParams& p) {
  const PrefillSplit sp = split_of(p, std::max(2, device_sms()));
  return sp.shares ? (part_floats(p, sp) + part_floats(p, sp) / kVDim) * sizeof(float) : 0;
}

bool launch_latent_prefill(const PrefillParams& p, cudaStream_t s) {
  const int sms = device_sms();
  if (sms < 2) return false;
  if (p.part) {
    PrefillSplit sp = split_of(p, sms);
    sp.part = p.part;
    sp.part_lse = p.part + part_floats(p, sp);
    return launch_prefill_split(p, sp, sms, s);
  }
  const PrefillSplit none = {};
  return p.pairs ? launch_prefill<true, false>(p, none, sms, s) : launch_prefill<false, false>(p, none, sms, s);
}

}  // namespace kda
