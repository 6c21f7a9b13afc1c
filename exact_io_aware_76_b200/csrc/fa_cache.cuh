// fa_cache.cuh -- a paged e4m3 K/V cache on sm_100a: quantising new tokens into its pages, and attention over it.
//
// The cache: pages of `page` tokens, codes [num_pages, Hkv, page, D] (e4m3) and one fp32 scale per page and head for
// K and for V (value = code * scale); a table [B, max_pages] of page numbers and a length per sequence. A page of one
// head is contiguous (page * D bytes), so it arrives as one TMA box, and 128 keys of a head are 128 / page boxes.
//
// Few query rows (decoding): attention without converting the cache. K and V stay e4m3 all the way into the tensor core
// (tcgen05 kind::f8f6f4); it is the other operand that is brought to 8 bits, without loss: a 16-bit number has 8 (bf16) or
// 11 (fp16)
// significant bits and an e4m3 number 4, so q = q1 + q2 (+ q3) with q1 = e4m3(q), q2 = e4m3(q - q1) and, for fp16,
// a third part for the 3 bits left is exact as long as the parts stay in range (split_f16x2).
// Each query row is first scaled by a power of two that brings its largest element to [128, 256); elements below
// 2^-9 of the largest lose what falls under the last part's smallest step, an absolute error of at most 2^-17 (bf16) or
// 2^-21 (fp16) of the row's largest element. S = q K^T is the sum of the parts' products in the fp32 accumulator.
// The weights are rounded to fp16 (relative error 2^-11) and split exactly into three parts, in e5m2: a significant bit
// less than e4m3 each, still 11 in all (every residual is signed, which counts for a bit), and a range down to 2^-16 that
// keeps the light weights beside a heavy one (split_weight).
//
// Scales. With ks, vs the scales of key j's page and c = scale * log2 e, the weight that reaches the PV product is
//   w_ij = 2^(s_ij c ks + log2 vs - m_i + 13),   O_i = sum_j w_ij v_j / l_i,   l_i = sum_j w_ij / vs_j,
// with m_i the running maximum of s c ks + log2 vs: the V scale is part of the exponent, so pages of any scales share one
// accumulator, and the largest weights have full precision whatever the scales are. The factor 2^13 uses e5m2's and
// fp16's range upwards (m may lag by up to 2, so w <= 2^15); what a small weight loses is at most 2^-17, so 2^-30 of the
// row's largest weight (split_weight), about 20 in the exponent of e below it.
// Scales lie in [2^-50, 2^50], so l (at most 2^(13+2+50) times the number of keys) stays finite.
//
// Work split. A unit is (sequence, block of query rows, K/V head); its walk is the 128-key tiles its rows see (window
// tiles, and before them the tiles with sinks). All units' tiles are laid end to end, each unit's with a few places
// before them for what a unit costs by itself (kCacheUnitCost), and every CTA takes an equal run of places, whatever the
// lengths are, so neither one long sequence nor many short ones load the SMs unevenly. Units cut by a run's border leave fp32 partial
// sums (O, m, l) in the workspace, and fa_cache_join_kernel adds them in key order, so results repeat bit for bit.
#pragma once
#include "fa_fwd.cuh"

namespace fa {

constexpr int kCacheCtas = 148;      // one CTA per SM; a fixed number, so that the workspace size needs no device
// Beginning and ending a unit takes a CTA about as long as this many tiles. Measured in a loop with 0 / 1 / 3 / 6 / 12 places
// per unit (us; bf16, pages of 64):
//    8 rows, 8 heads of 128, 32 sequences of 100 to 8000 tokens    95 /  88 /  76 /  74 /  76    (heads of 64: 70 / 68 / 61 / 57 / 60)
//    8 rows, 8 heads of 128, 64 sequences of 100 to 1000           61 /  51 /  43 /  42 /  43    (51 / 45 / 37 / 37 / 39)
//   16 rows, 4 heads of 128, 100 to 8000                           73 /  65 /  55 /  54 /  59    (52 / 47 / 42 / 44 / 46)
//   32 rows, 4 heads of 128, 100 to 8000                           82 /  74 /  62 /  61 /  66    (58 / 53 / 52 / 53 / 57)
//  256 rows, 8 heads of 128, 16 sequences of 300 to 8000          212 / 186 / 173 / 156 / 149    (150 / 137 / 131 / 124 / 129)
// 3 is within 7% of the best for up to 32 rows. Units of 256 rows would be 4 to 18% faster with 6 (a number of their own is
// not built).
constexpr int kCacheUnitCost = 3;
constexpr float kCacheLag = 2.0f;    // how far the running maximum may lag (log2)
constexpr float kCacheShift = 13.0f;  // weights carry 2^13 (see above)
// The same for blocks of many rows, whose weights are fp16 (w <= 2^15; what is lost lies below 2^-34 of the largest).
constexpr float kManyLag = 6.0f, kManyShift = 9.0f;

struct CacheParams {
  const void* q;         // [B, Sq, H, D]
  void* out;             // [B, Sq, H, D]
  float* lse;            // [B, H, Sq]
  const float* k_scale;  // [num_pages, Hkv]
  const float* v_scale;
  const int* table;      // [B, max_pages]
  const int* lens;       // [B]
  float* part_o;         // [kCacheCtas, 2, rows per unit, D]
  float* part_ml;        // [kCacheCtas, 2, rows per unit, 2]
  int4* cuts;            // [kCacheCtas] the unit cut at a CTA's first tile: item, K/V head, last CTA (item < 0: none)
  int B, H, Hkv, group, Sq;
  int n_rows, n_mt;      // query rows of a (sequence, K/V head) = Sq * group; units they make
  int page, max_pages, num_pages;
  int win_left, sinks;   // win_left < 0: no window (sinks = 0 then)
  int whole;             // units are not cut (all are short): no join follows
  float scale_log2;
};

// ------------------------------------------------------------------------------------------------------ append
struct AppendParams {
  const void *k, *v;     // new K and V, [B, T, Hkv, D]
  uint8_t *k_pages, *v_pages;  // [num_pages, Hkv, page, D]
  float *k_scale, *v_scale;    // [num_pages, Hkv]
  const int* table;
  const int* lens;       // lengths after the append
  const int* counts;     // new tokens per sequence (null: T)
  int B, T, Hkv, page, max_pages, num_pages;
  int n_touch;           // pages that T tokens can touch
};

__device__ __forceinline__ uint32_t e4m3x2_from_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t e5m2x2_from_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Parts of q beyond the stacked ones: the third part of fp16 where it has no rows of its own.
__host__ __device__ constexpr bool part_is_e5m2(int q, int stack) { return q == 2 && stack < 3; }
template <bool kBF16>
__device__ __forceinline__ void unpack2(uint32_t v, float& a, float& b) {
  if (kBF16) {
    a = __uint_as_float(v << 16);
    b = __uint_as_float(v & 0xffff0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
    a = f.x;
    b = f.y;
  }
}

// The smallest power of two s with amax <= 448 s, exponent within [-50, 50] (448 = 0.875 * 2^9).
__device__ __forceinline__ float append_scale(float amax) {
  int e = 0;
  const float m = frexpf(amax, &e);
  e = amax > 0.f ? e - 9 + (m > 0.875f ? 1 : 0) : -50;
  e = max(-50, min(50, e));
  return __int_as_float((e + 127) << 23);
}

// One CTA per (sequence, page its new tokens touch, head, K or V): it alone writes that page of that head, so a
// larger scale can move the page's earlier codes in place. Power-of-two scales make that move exact (but for codes that
// become subnormal), and cost no precision: e4m3's steps are relative. Bound by bytes for long prompts (read 16 bits,
// write 8), by latency for single tokens. The page's new tokens stay in registers between the two passes over them
// (kPasses 16-byte pieces per thread = page * D / 1024), all loads in flight at once: 8 x 1900 tokens, 8 heads of 128,
// 24 -> 19 us; magnitudes compared as packed patterns: 16 us (12 us at the copy rate; 64 x 2048 tokens: 144 us, 0.86
// of it).
template <int D, bool kBF16, int kPasses>
__global__ void __launch_bounds__(128) fa_cache_append_kernel(const AppendParams p) {
  constexpr int kVecs = D / 8;            // 8-element vectors per token
  constexpr int kRows = 128 / kVecs;      // tokens per pass of the CTA
  __shared__ uint32_t red[4];
  unsigned n_cta = blockIdx.x;
  const int which = static_cast<int>(n_cta & 1u);
  n_cta >>= 1;
  const int h = static_cast<int>(n_cta % p.Hkv);
  n_cta /= p.Hkv;
  const int touch = static_cast<int>(n_cta % p.n_touch);
  const int b = static_cast<int>(n_cta / p.n_touch);
  const int len = p.lens[b];
  const int count = min(max(p.counts ? p.counts[b] : p.T, 0), min(p.T, max(len, 0)));
  const int first = len - count;
  const int n = first / p.page + touch;
  if (count == 0 || n >= p.max_pages || static_cast<long long>(n) * p.page >= len) return;
  const int pid = __ldg(p.table + static_cast<size_t>(b) * p.max_pages + n);  // (used after the tokens are on their way)
  const int lo = max(first, n * p.page), hi = min(len, n * p.page + p.page);  // positions written here
  const int vec = threadIdx.x % kVecs, r0 = threadIdx.x / kVecs;
  const uint16_t* src = static_cast<const uint16_t*>(which ? p.v : p.k) +
                        ((static_cast<size_t>(b) * p.T + (p.T - len + lo)) * p.Hkv + h) * D + vec * 8;
  const size_t stride = static_cast<size_t>(p.Hkv) * D;
  uint4 v[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + i * kRows < hi - lo) v[i] = __ldg(reinterpret_cast<const uint4*>(src + (r0 + i * kRows) * stride));
  }
  if (pid < 0 || pid >= p.num_pages) return;
  uint8_t* codes = (which ? p.v_pages : p.k_pages) + (static_cast<size_t>(pid) * p.Hkv + h) * p.page * D;
  float* sc = (which ? p.v_scale : p.k_scale) + static_cast<size_t>(pid) * p.Hkv + h;
  const int kept = lo - n * p.page;  // earlier tokens of this page
  const float old = kept > 0 ? *sc : 0.f;
  // The largest magnitude, as 16-bit patterns two at a time (patterns of magnitudes order as the magnitudes do). Where
  // the page's new tokens hold an infinity or a NaN the patterns of those are left out in a second round.
  constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
  uint32_t top = 0;
#pragma unroll
  for (int round = 0; round < 2; ++round) {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t a = w[e] & 0x7fff7fffu;
        if (round == 1) a = ((a & 0xffffu) < kInf ? a & 0xffffu : 0u) | ((a >> 16) < kInf ? a & 0xffff0000u : 0u);
        mx = __vmaxu2(mx, a);
      }
    }
    mx = max(mx & 0xffffu, mx >> 16);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (round == 1) __syncthreads();  // the first round's values are read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
    __syncthreads();
    top = max(max(red[0], red[1]), max(red[2], red[3]));
    if (top < kInf) break;
  }
  float amax, unused;
  unpack2<kBF16>(top, amax, unused);
  const float now = fmaxf(append_scale(amax), old);
  if (kept > 0 && now != old) {
    const float f = old / now;
    for (int t = threadIdx.x; t < kept * (D / 4); t += 128) {
      uint32_t* c4 = reinterpret_cast<uint32_t*>(codes) + t;
      const uint32_t c = *c4;
      float x0, x1, x2, x3;
      unpack2<false>(f16x2_from_e4m3x2(c & 0xffffu), x0, x1);
      unpack2<false>(f16x2_from_e4m3x2(c >> 16), x2, x3);
      *c4 = pack4_e4m3(x0 * f, x1 * f, x2 * f, x3 * f);
    }
  }
  if (threadIdx.x == 0) *sc = now;
  // A power of two (always, unless the caller's earlier scale was none) is divided by exactly as a product.
  const bool pow2 = (__float_as_uint(now) & 0x7fffffu) == 0u;
  const float inv = 1.f / now;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * kRows;
    if (r >= hi - lo) break;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      unpack2<kBF16>(w[e], x[2 * e], x[2 * e + 1]);
      x[2 * e] = pow2 ? x[2 * e] * inv : x[2 * e] / now;
      x[2 * e + 1] = pow2 ? x[2 * e + 1] * inv : x[2 * e + 1] / now;
    }
    *reinterpret_cast<uint2*>(codes + static_cast<size_t>(kept + r) * D + vec * 8) =
        make_uint2(pack4_e4m3(x[0], x[1], x[2], x[3]), pack4_e4m3(x[4], x[5], x[6], x[7]));
  }
}

// ------------------------------------------------------------------------------------------------- work split
// One item: a (sequence, block of kRows query rows); n: the tiles of its walk (at least one, so that rows without
// a visible key are visited and written).
struct CacheItem {
  int b, row0, rows;    // query rows [row0, row0 + rows) of the Sq * group rows; row r: query r / group
  int c0;               // aligned key of query 0 = length - Sq
  int c_min, c_max;     // aligned keys of the first and last row
  int key_lo, key_hi;   // keys its rows see: [key_lo, key_hi] and the sinks below key_lo
  int j_lo, n_sink, n;  // first window tile, sink tiles before it, tiles in all
};

template <int kRows>
__device__ __forceinline__ CacheItem cache_item(const CacheParams& p, int x) {
  CacheItem t;
  t.b = x / p.n_mt;
  t.row0 = (x % p.n_mt) * kRows;
  t.rows = min(kRows, p.n_rows - t.row0);
  const int len = max(0, min(__ldg(p.lens + t.b), p.max_pages * p.page));
  t.c0 = len - p.Sq;
  t.c_min = t.c0 + t.row0 / p.group;
  t.c_max = t.c0 + (t.row0 + t.rows - 1) / p.group;
  t.key_hi = t.c_max;
  t.key_lo = p.win_left >= 0 ? max(0, t.c_min - p.win_left) : 0;
  t.j_lo = t.n_sink = 0;
  t.n = 1;
  if (t.key_hi >= 0) {
    t.j_lo = t.key_lo / 128;
    t.n_sink = min((p.sinks + 127) / 128, t.j_lo);
    t.n = t.n_sink + t.key_hi / 128 - t.j_lo + 1;
  }
  return t;
}
__device__ __forceinline__ int cache_key0(const CacheItem& t, int w) {
  return (w < t.n_sink ? w : t.j_lo + w - t.n_sink) * 128;
}
// Whether the tile at key0 holds keys that none of the item's rows sees (what the page holds there may be stale).
__device__ __forceinline__ bool cache_ragged(const CacheParams& p, const CacheItem& t, int key0) {
  return key0 + 127 > t.key_hi || (key0 < t.key_lo && key0 + 127 >= p.sinks);
}

// A position in the row of all tiles: tile w of (item x, K/V head hk). Order: items, then heads, then tiles.
struct CachePos {
  int x, hk, w;
};
template <int kRows>
struct CacheWalk {
  CachePos at;
  CacheItem item;
  __device__ __forceinline__ void start(const CacheParams& p, const CachePos& s) {
    at = s;
    item = cache_item<kRows>(p, at.x);
  }
  // Ahead by `by` tiles (the caller stays within the row of tiles).
  __device__ __forceinline__ void advance(const CacheParams& p, int by) {
    at.w += by;
    while (at.w >= item.n) {
      at.w -= item.n;
      if (++at.hk == p.Hkv) {
        at.hk = 0;
        if (++at.x >= p.B * p.n_mt) return;
        item = cache_item<kRows>(p, at.x);
      }
    }
  }
};

struct CacheRun {
  int count;     // tiles of this CTA
  CachePos first;
};
struct CacheScan {  // shared memory of cache_run
  long long sums[16][2];
  long long begin_tile, end_tile;  // tiles before the run's two ends
  CachePos first;
};

// This CTA's run of tiles, found by every thread together (kThreads of them). Places: a unit of n tiles takes
// kCacheUnitCost + n of them, its tiles the last n; CTA c takes places [c share, (c + 1) share). All items are counted
// first, then those holding the run's two ends are searched. Also notes the unit cut at the run's begin, for the join.
template <int kRows, int kThreads>
__device__ __forceinline__ CacheRun cache_run(const CacheParams& p, CacheScan* sh) {
  const int items = p.B * p.n_mt, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  long long tiles = 0;
  for (int x = tid; x < items; x += kThreads) tiles += cache_item<kRows>(p, x).n;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, s);
  if (lane == 0) sh->sums[warp][0] = tiles;
  if (tid == 0) {
    sh->begin_tile = sh->end_tile = 0;
    p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  __syncthreads();
  long long total_tiles = 0;
  for (int i = 0; i < kWarps; ++i) total_tiles += sh->sums[i][0];
  total_tiles *= p.Hkv;
  const long long total = total_tiles + static_cast<long long>(items) * p.Hkv * kCacheUnitCost;
  const long long share = (total + kCacheCtas - 1) / kCacheCtas;
  const long long begin = share * blockIdx.x, end = begin + share;
  if (begin < total) {  // (uniform)
    if (tid == 0 && end >= total) sh->end_tile = total_tiles;
    long long place = 0, tile = 0;  // of the first item of the chunk
    for (int x0 = 0; x0 < items; x0 += kThreads) {
      const int x = x0 + tid;
      const int n = x < items ? cache_item<kRows>(p, x).n : 0;
      const long long my_tiles = static_cast<long long>(n) * p.Hkv;
      const long long mine = x < items ? my_tiles + static_cast<long long>(p.Hkv) * kCacheUnitCost : 0;
      long long incl = mine, incl_t = my_tiles;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, s), ot = __shfl_up_sync(0xffffffffu, incl_t, s);
        if (lane >= s) {
          incl += o;
          incl_t += ot;
        }
      }
      __syncthreads();  // the sums of the count, or of the chunk before, are read
      if (lane == 31) {
        sh->sums[warp][0] = incl;
        sh->sums[warp][1] = incl_t;
      }
      __syncthreads();
      long long lo = place + incl - mine, lo_t = tile + incl_t - my_tiles;
      for (int i = 0; i < warp; ++i) {
        lo += sh->sums[i][0];
        lo_t += sh->sums[i][1];
      }
      // The first tile at or after place `at` of this thread's item (of a unit that begins there, if units stay
      // whole), and how many tiles come before it.
      auto find = [&](long long at, CachePos* pos) {
        const long long unit = n + kCacheUnitCost, rel = at - lo + (p.whole ? unit - 1 : 0);
        const int hk = static_cast<int>(rel / unit);
        pos->x = hk < p.Hkv ? x : x + 1;
        pos->hk = hk < p.Hkv ? hk : 0;
        pos->w = p.whole ? 0 : max(0, static_cast<int>(rel % unit) - kCacheUnitCost);
        return lo_t + static_cast<long long>(hk) * n + pos->w;
      };
      if (lo <= begin && begin < lo + mine) {
        CachePos first;
        sh->begin_tile = find(begin, &first);
        sh->first = first;
        // A unit that goes on here: its first piece's successor joins it.
        const long long u0 = begin - first.w;  // its first tile's place
        if (first.w > 0 && u0 / share == blockIdx.x - 1)
          p.cuts[blockIdx.x] = make_int4(x, first.hk, static_cast<int>((u0 + n - 1) / share), 0);
      }
      if (lo <= end && end < lo + mine) {
        CachePos last;
        sh->end_tile = find(end, &last);
      }
      for (int i = 0; i < kWarps; ++i) {
        place += sh->sums[i][0];
        tile += sh->sums[i][1];
      }
      if (end < place) break;
    }
  }
  __syncthreads();
  return {static_cast<int>(sh->end_tile - sh->begin_tile), sh->first};
}

// Where a piece of a unit leaves its sums: slot 0 of its CTA if the unit began before, slot 1 if it goes on after.
__device__ __forceinline__ int cache_slot(int cta, int w0) { return cta * 2 + (w0 > 0 ? 0 : 1); }

// Joins the pieces of every cut unit: CTA (c, y) takes rows 8 y .. 8 y + 7 of the unit whose second piece begins run c.
template <int D, bool kBF16, int kRows>
__global__ void __launch_bounds__(2 * D) fa_cache_join_kernel(const CacheParams p) {
  const int4 cut = p.cuts[blockIdx.x];
  if (cut.x < 0) return;
  const CacheItem t = cache_item<kRows>(p, cut.x);
  const int c_first = blockIdx.x - 1, c_last = cut.z;
  const int r = blockIdx.y * 8 + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
  if (r < t.rows) {
    float m = -INFINITY;
    for (int c = c_first; c <= c_last; ++c) {
      const size_t s = static_cast<size_t>(cache_slot(c, c > c_first)) * kRows + r;
      m = fmaxf(m, p.part_ml[s * 2]);
    }
    const float m_use = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c_first; c <= c_last; ++c) {
      const size_t s = static_cast<size_t>(cache_slot(c, c > c_first)) * kRows + r;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + s * 2);
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m_use);
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + s * D + d);
      l = fmaf(ml.y, f, l);
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
      o.z = fmaf(x.z, f, o.z);
      o.w = fmaf(x.w, f, o.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // l = 0: no visible key (a NaN stays one)
    const int row = t.row0 + r, i = row / p.group, h = cut.y * p.group + row % p.group;
    uint16_t* dst = static_cast<uint16_t*>(p.out) + ((static_cast<size_t>(t.b) * p.Sq + i) * p.H + h) * D + d;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack2<kBF16>(o.x * inv, o.y * inv), pack2<kBF16>(o.z * inv, o.w * inv));
    if (d == 0)
      p.lse[(static_cast<size_t>(t.b) * p.H + h) * p.Sq + i] =
          l == 0.f ? -INFINITY : (m + log2f(l) - (kRows == 256 ? kManyShift : kCacheShift)) * kLn2;
  }
}

// --------------------------------------------------------------------------------------------- shared pieces
// The issuing warp's products and commits, predicated on the one lane that issues: the warp's control flow stays uniform,
// so the compiler may keep descriptors and addresses in uniform registers, where these instructions take them from.
__device__ __forceinline__ void umma_ss_f8_if(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_ts_f8_if(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

constexpr uint32_t kE5M2A = 1u << 7;  // instruction descriptor, kind::f8f6f4: A in e5m2 (B in e4m3)

// Few query rows per unit: R = 8, 16 or 32.
template <int D, bool kBF16, int R>
struct CacheSmem {
  // Parts of q and of the weights. The A operand holds every row 128 / R times: the lanes of a warp hold it kStack times,
  // with different parts. Two e4m3 parts of the weights are enough for bf16's 8 bits but drop a weight 2^-20 below the row's
  // largest; three cost, in a loop, 431 -> 439 us (R = 8, 32 x 32768 tokens, 8 heads of 128), 313 -> 323 us (heads of 64)
  // and 123 -> 146 us (R = 16, 32 x 16384 tokens, 4 heads of 128: two products per O instead of one).
  // bf16's two parts of q do not fill four rows: they lie there twice, kQStack rows each time, and the second pair of lanes
  // takes the second half of the keys, which saves half the exchange of partial scores (448 -> 439 us, as above).
  static constexpr int kStack = 32 / R;
  static constexpr int kQParts = kBF16 ? 2 : 3, kPParts = 3;
  static constexpr int kQStack = kStack < kQParts || !kBF16 ? kStack : 2;
  static constexpr int kQPass = (kQParts + kQStack - 1) / kQStack;  // products per S
  static constexpr int kPPass = (kPParts + kStack - 1) / kStack;  // products per O
  static constexpr int kTile = 16384;                // 128 rows of one 128-byte swizzle row (head dim 64: half zeros)
  static constexpr int kStages = kQPass == 1 ? 5 : 4;
  static constexpr int kQOff = 0;                    // [product]
  static constexpr int kKOff = kQOff + kQPass * kTile;
  static constexpr int kVOff = kKOff + kStages * kTile;
  // kJoinCols columns of the warps' O, [8 warps][R rows][kJoinCols + 4] floats
  static constexpr int kJoinCols = 1024 / R < D ? 1024 / R : D;
  static constexpr int kXOff = kVOff + kStages * kTile;
  static constexpr int kXBytes = 8 * R * (kJoinCols + 4) * 4;
  static constexpr int kFacOff = kXOff + kXBytes;    // per stage: k factor, log2 v scale, 1 / v scale of 8 key groups
  static constexpr int kMlOff = kFacOff + kStages * 96;  // row factors [2][32], m and l per lane [2][256]
  static constexpr int kBarOff = kMlOff + (64 + 512) * 4;
  static constexpr int kNumBars = 4 * kStages + 8;
  static constexpr int kScanOff = kBarOff + kNumBars * 8;
  static constexpr int kMiscOff = kScanOff + static_cast<int>(sizeof(CacheScan));
  static constexpr int kAlloc = kMiscOff + 16 + 1024;
  static constexpr int kThreads = 384;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kAlloc <= 232448, "shared memory");
};

// A copying warp (K, V or both): walks the run's tiles, a lane per 16-key group, four tiles per batch. The page numbers
// of the batch after next and the scales of the next batch are loaded while this batch's copies are issued, so that
// neither of the two dependent loads is waited for. Pages that no row sees, and page numbers outside the cache, are copied
// from beyond the tensor's end: the copy engine writes zeros and reads nothing. The factors of a tile's key groups go into a
// ring of kFac places; kFac = kStages: they are published with K.
template <int kRows, int kStages, int kFac, bool kK = true, bool kV = true>
__device__ __forceinline__ void cache_producer(const CacheParams& p, const CacheRun& run, const CUtensorMap& tm_k,
                                               const CUtensorMap& tm_v, uint8_t* smem_k, uint8_t* smem_v, float* fac,
                                               uint64_t* k_full, uint64_t* v_full, uint64_t* kv_empty,
                                               uint64_t* fac_full, volatile int* abort_flag) {
  const int lane = lane_id(), tt = lane >> 3, grp = lane & 7;
  struct Slot {
    int row;  // first row of the page in the [num_pages * Hkv * page, D] view, < 0: none
    int hk, id;
    float ks, vs;
  };
  CacheWalk<kRows> walk;
  int ahead = tt;  // tile index (within the run) of the walk's position
  if (ahead < run.count) {
    walk.start(p, run.first);
    walk.advance(p, tt);
  }
  auto load_id = [&]() {
    Slot s;
    s.id = -1;
    s.hk = 0;
    s.ks = s.vs = 0.f;
    if (ahead < run.count) {
      const CacheItem& t = walk.item;
      const int key = cache_key0(t, walk.at.w) + grp * 16;
      const int n = key / p.page, pk = n * p.page;
      s.hk = walk.at.hk;
      if (n < p.max_pages && pk <= t.key_hi && (pk + p.page > t.key_lo || pk < p.sinks))
        s.id = __ldg(p.table + static_cast<size_t>(t.b) * p.max_pages + n);
      ahead += 4;
      if (ahead < run.count) walk.advance(p, 4);
    }
    return s;
  };
  auto load_scales = [&](Slot& s) {
    s.row = -1;
    if (s.id >= 0 && s.id < p.num_pages) {
      const size_t i = static_cast<size_t>(s.id) * p.Hkv + s.hk;
      s.ks = __ldg(p.k_scale + i);
      s.vs = __ldg(p.v_scale + i);
      s.row = static_cast<int>(i * p.page);
    }
  };
  const int beyond = p.num_pages * p.Hkv * p.page;
  const bool leads = (grp * 16) % p.page == 0;  // this lane's group starts a page
  Slot cur = load_id();
  load_scales(cur);
  Slot nxt = load_id();
  int g = 0;
  bool ok = true;
  for (int t0 = 0; ok && t0 < run.count; t0 += 4) {
    Slot far = load_id();
    load_scales(nxt);
    for (int u = 0; u < 4 && t0 + u < run.count; ++u) {
      g = t0 + u;
      const int s = g % kStages;
      const bool got = g < kStages || mbar_wait(&kv_empty[s], ((g / kStages) - 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      // The copies need the page number only; their bytes count towards a phase that the arrival below opens and ends.
      if (tt == u && leads) {
        const int row = cur.row >= 0 ? cur.row : beyond;
        if (kK) tma_load_2d(smem_k + s * 16384 + grp * 2048, &tm_k, &k_full[s], 0, row);
        if (kV) tma_load_2d(smem_v + s * 16384 + grp * 2048, &tm_v, &v_full[s], 0, row);
      }
      __syncwarp();
      if (kK && tt == u) {
        const bool valid = cur.row >= 0;
        float* f = fac + (g % kFac) * 24 + grp;
        f[0] = valid ? cur.ks : 1.f;
        f[8] = valid ? log2f(cur.vs) : -INFINITY;  // a key without a page has weight 0
        f[16] = valid ? 1.f / cur.vs : 0.f;
      }
      __syncwarp();
      if (lane == 0) {
        if (kFac != kStages) mbar_arrive(&fac_full[g % kFac]);
        if (kK) mbar_arrive_expect_tx(&k_full[s], 16384);
        if (kV) mbar_arrive_expect_tx(&v_full[s], 16384);
      }
    }
    cur = nxt;
    nxt = far;
  }
  if (*abort_flag) {
    // Let the copies already issued land before the CTA exits (bounded; own flag, not the CTA's).
    const int issued = ok ? run.count : g;
    for (int i = max(0, issued - kStages); i < issued; ++i) {
      int drain = 0;
      if (kK) mbar_wait(&k_full[i % kStages], (i / kStages) & 1, &drain);
      drain = 0;
      if (kV) mbar_wait(&v_full[i % kStages], (i / kStages) & 1, &drain);
    }
  }
}

// The cleaning warp: hands every V tile on to the MMA thread, and in a ragged one first sets the V rows that no query
// row sees to 0, because their weights are 0 but a stale byte may be a NaN (0 * NaN). (K needs none of this: masked
// scores are replaced.) Every tile goes through here, ragged or not: a warp that waited for some tiles only could
// be two phases of a stage's barrier ahead or behind and mistake one phase for another.
template <int kRows, int kStages>
__device__ __forceinline__ void cache_cleaner(const CacheParams& p, const CacheRun& run, uint8_t* smem_v,
                                              uint64_t* v_full, uint64_t* v_clean, volatile int* abort_flag) {
  CacheWalk<kRows> walk;
  if (run.count > 0) walk.start(p, run.first);
  const int lane = lane_id();
  for (int g = 0; g < run.count; ++g) {
    const CacheItem& t = walk.item;
    const int key0 = cache_key0(t, walk.at.w), s = g % kStages;
    const bool got = mbar_wait(&v_full[s], (g / kStages) & 1, abort_flag);
    if (!__all_sync(0xffffffffu, got)) return;
    if (cache_ragged(p, t, key0)) {
      for (int i = lane; i < 128 * 8; i += 32) {
        const int key = key0 + i / 8;
        if (key > t.key_hi || (key < t.key_lo && key >= p.sinks))
          *reinterpret_cast<uint4*>(smem_v + s * 16384 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (lane == 0) mbar_arrive(&v_clean[s]);
    if (g + 1 < run.count) walk.advance(p, 1);
  }
}

// 2^k as a float, k in [-126, 127].
__device__ __forceinline__ float pow2i(int k) { return __int_as_float((k + 127) << 23); }

// Row scaling of q: with amax the row's largest magnitude, q * mul has its largest element in [128, 256), and a
// product with it is multiplied by back = 1 / mul. Returns whether the row is finite. One with an infinity or a NaN is
// to be NaN where it sees a key, and 0 (LSE -inf) as any other row where it sees none: its callers compute with a row of
// zeros in its place and turn the row's sum of weights into a NaN at the end, if it has seen a key.
__device__ __forceinline__ bool q_row_scale(uint32_t amax_bits, float& mul, float& back) {
  // (magnitudes of floats order as their bits; bits of 2^128 and above are infinities and NaNs)
  const bool finite = amax_bits < 0x7f800000u;
  if (!finite) amax_bits = 0;
  int e = static_cast<int>(amax_bits >> 23) - 127;
  e = max(e, -100);  // smaller rows keep a fixed factor (0 rows included)
  mul = pow2i(min(7 - e, 127));
  back = pow2i(max(e - 7, -126));
  return finite;
}
constexpr uint32_t kNanBits = 0x7fc00000u;

// Two fp16 numbers -> kParts pairs of 8-bit codes, largest part first. Part q is multiplied by 2^(4 (q % kStack)), so
// that the parts that lie in different rows of an operand (kStack of them) all use the whole e4m3 range; a part behind
// them adds to the first one's row, unscaled, in e5m2, which reaches down to 2^-16.
template <int kParts, int kStack>
__device__ __forceinline__ void split_f16x2(uint32_t h, uint32_t* code) {
  static_assert(kParts <= 3, "a factor for every part");
#pragma unroll
  for (int q = 0; q < kParts; ++q) {
    constexpr uint32_t kUp[3] = {0x3c003c00u, 0x4c004c00u, 0x5c005c00u};    // 1, 2^4, 2^8
    constexpr uint32_t kDown[3] = {0x3c003c00u, 0x2c002c00u, 0x1c001c00u};  // 1, 2^-4, 2^-8
    const uint32_t up = q % kStack ? mul_f16x2(h, kUp[q % kStack]) : h;
    if (part_is_e5m2(q, kStack)) {
      code[q] = e5m2x2_from_f16x2(up);
    } else {
      code[q] = e4m3x2_from_f16x2(up);
      if (q + 1 < kParts) {
        const uint32_t back = f16x2_from_e4m3x2(code[q]);
        h = sub_f16x2(h, q % kStack ? mul_f16x2(back, kDown[q % kStack]) : back);
      }
    }
  }
}

// Eight elements of q (16 bytes) -> kParts x 8 codes.
template <bool kBF16, int kParts, int kStack>
__device__ __forceinline__ void q_split8(const uint4& v, float mul, uint2* part) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4][kParts];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2<kBF16>(w[i], a, b);
    split_f16x2<kParts, kStack>(pack2_f16(a * mul, b * mul), c[i]);  // at most 256, 11 bits: exact down to 2^-24
  }
#pragma unroll
  for (int q = 0; q < kParts; ++q) part[q] = make_uint2(c[0][q] | (c[1][q] << 16), c[2][q] | (c[3][q] << 16));
}
template <bool kBF16>
__device__ __forceinline__ uint32_t q_amax8(const uint4& v, uint32_t amax) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack2<kBF16>(w[i], a, b);
    amax = max(amax, max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
  }
  return amax;
}

// Two weights, rounded to fp16 (at most 2^15) -> three pairs of e5m2 codes, largest part first, part q multiplied by
// 2^(4 (q % kStack)) as in split_f16x2. Exact for kStack = 4, and for weights of 2^-6 and above otherwise; what smaller ones
// lose there is at most 2^-17.
template <int kStack>
__device__ __forceinline__ void split_weight(uint32_t h, uint32_t* code) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    constexpr uint32_t kUp[3] = {0x3c003c00u, 0x4c004c00u, 0x5c005c00u};    // 1, 2^4, 2^8
    constexpr uint32_t kDown[3] = {0x3c003c00u, 0x2c002c00u, 0x1c001c00u};  // 1, 2^-4, 2^-8
    code[q] = e5m2x2_from_f16x2(q % kStack ? mul_f16x2(h, kUp[q % kStack]) : h);
    if (q < 2) {
      const uint32_t back = __byte_perm(code[q], 0u, 0x1404);  // e5m2 is the upper byte of fp16
      h = sub_f16x2(h, q % kStack ? mul_f16x2(back, kDown[q % kStack]) : back);
    }
  }
}
// Four weights -> their parts' codes, packed four to a register (first weight lowest).
template <int kStack>
__device__ __forceinline__ void p_split4(float a, float b, float c, float d, uint32_t* part) {
  uint32_t lo[3], hi[3];
  split_weight<kStack>(pack2_f16(a, b), lo);
  split_weight<kStack>(pack2_f16(c, d), hi);
#pragma unroll
  for (int q = 0; q < 3; ++q) part[q] = lo[q] | (hi[q] << 16);
}

// -------------------------------------------------------------------------------- attention of few query rows
// Decoding: up to R = 8, 16 or 32 rows (the query heads of a K/V head, times a few tokens) against a long cache. The
// bytes of the cache bound it, so everything else is arranged to hide behind the copies. An M = 128 product costs the
// same however few of its rows are used, so the rows are put into the A operand 128 / R times. kStack neighbouring
// copies hold the parts of q (and later of the weights), so that one product does the work of all parts: their partial
// scores are added across lanes, and their rows of O at the end. The warps share out the tile's 128 keys, 32 each: a
// warp's copies have a running maximum, sums and rows of O of their own, and weights of 0 for the other warps' keys. Nothing else is exchanged until the copies are joined, once, at the end of
// the unit. Measured at 32 x 32768 tokens, 64 query heads on 8, bf16 (2.15 GB: 328 us at the copy rate): one product
// per part 505 us; one product with all parts 427; two softmax warpgroups 398; each score computed by one lane 383; two
// warps copying 388, but 526 -> 420 with pages of 16; the issuing warp uniform 371; a third part of the weights, for the
// light ones' sake, 389 for single calls (84% of the copy rate; fp16 406) and 448 in a loop of seconds (73%; fp16 463),
// where the power cap holds the SMs at 1.47 GHz and the same copy takes 331. Heads of 64: 315 and 328 us, half the copy
// rate. What bounds it is the chain issue -> scores -> weights -> issue, 1300 cycles a tile as traced (1360 in fp16, 1150
// for heads of 64; the trace's own stores included).
//
// Warps: 0-3 and 4-7 softmax of the even and the odd tiles of the run, each warpgroup with its own S and O (so its own
// maxima and sums too, joined with the others at the end): two tiles are in work at any time, and a warpgroup's
// latencies have two tiles' time to pass in. 8 and 11 copy K and V (TMA), 9 MMA, 10 cleaner (see cache_cleaner).
// TMEM columns: S of both [0,128) and [128,256), O [256,384) and [384,512); the parts of P overwrite their S, 32 columns
// each. The MMA order is S(g+1), PV(g), S(g+2), ..., so when S(g) has arrived PV(g-2), the last product of that
// warpgroup, is complete: O may be rescaled without a further wait.
template <int D, bool kBF16, int R>
__global__ void __launch_bounds__(384, 1)
    fa_cache_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const CacheParams p) {
  using L = CacheSmem<D, kBF16, R>;
  constexpr int kStages = L::kStages, kStack = L::kStack, kQStack = L::kQStack, kQParts = L::kQParts, kPParts = L::kPParts;
  constexpr int kQPass = L::kQPass, kPPass = L::kPPass;
  constexpr int kCopies = 8 * (32 / R);  // of a row, in both warpgroups
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* k_full = bars;
  uint64_t* v_full = k_full + kStages;
  uint64_t* kv_empty = v_full + kStages;
  uint64_t* v_clean = kv_empty + kStages;
  uint64_t* s_full = v_clean + kStages;   // [2]
  uint64_t* p_full = s_full + 2;          // [2]
  uint64_t* q_ready = s_full + 4;
  uint64_t* joint = s_full + 5;           // the softmax warps among themselves
  uint64_t* unit_done = s_full + 6;       // a unit's products complete
  uint64_t* mma_done = s_full + 7;
  float* fac = reinterpret_cast<float*>(smem + L::kFacOff);
  float* row_back = reinterpret_cast<float*>(smem + L::kMlOff);  // [parity of the unit][32]
  float* q_m = row_back + 64;                                     // [256 lanes]
  float* q_l = q_m + 256;                                         // [256 lanes]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const uint32_t warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&v_clean[s], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(&p_full[0], 128);
    mbar_init(&p_full[1], 128);
    mbar_init(q_ready, 256);
    mbar_init(joint, 256);
    mbar_init(unit_done, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_holder, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  const CacheRun run = cache_run<R, L::kThreads>(p, reinterpret_cast<CacheScan*>(smem + L::kScanOff));
  if (warp >= 8) {
    regs_dec<88>();
    if (run.count == 0) {
    } else if (warp == 8) {
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      cache_producer<R, kStages, kStages, true, false>(p, run, tm_k, tm_v, smem + L::kKOff, smem + L::kVOff, fac, k_full,
                                                       v_full, kv_empty, nullptr, abort_flag);
    } else if (warp == 11) {
      cache_producer<R, kStages, kStages, false, true>(p, run, tm_k, tm_v, smem + L::kKOff, smem + L::kVOff, fac, k_full,
                                                       v_full, kv_empty, nullptr, abort_flag);
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t id_s = idesc_e4m3(128, 128, false, false);  // (| kE5M2A for the third parts)
      constexpr uint32_t id_o = idesc_e4m3(128, 128, false, true) | kE5M2A;
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::kQOff), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::kKOff), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::kVOff), 16384, 1024);
      // This warp paces the kernel (8 products a tile, 72 cycles each, and as long again in waits): its control flow is
      // uniform, stages and phases are counted, not divided out, and the barriers that are mostly complete are tested
      // together and ahead of their use.
      const uint32_t lead = lane == 0 ? 1u : 0u;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int count = __shfl_sync(0xffffffffu, run.count, 0);
      auto all = [&](bool x) { return __all_sync(0xffffffffu, x) != 0; };
      auto issue_s = [&](uint32_t buf, int s) {
        const uint64_t b0 = sdesc_add(k_desc, s * L::kTile);
        const uint32_t d = tm + buf * 128;
#pragma unroll
        for (int q = 0; q < kQPass; ++q)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_ss_f8_if(lead, d, sdesc_add(q_desc, q * L::kTile + kk * 32), sdesc_add(b0, kk * 32),
                          id_s | (part_is_e5m2(q * kQStack, kQStack) ? kE5M2A : 0u), (q > 0 || kk > 0) ? 1u : 0u);
        umma_commit_if(lead, &s_full[buf]);
      };
      CacheWalk<R> walk;
      walk.start(p, run.first);
      bool ok = true;
      int s = 0;          // stage of tile g
      uint32_t ph = 0;    // phase of its barriers
      for (int g = 0, unit = 0; ok && g < count; ++unit) {
        const int left = __shfl_sync(0xffffffffu, min(count - g, walk.item.n - walk.at.w), 0);  // the unit's, in the run
        ok = all(mbar_wait(q_ready, unit & 1, abort_flag) && mbar_wait(&k_full[s], ph, abort_flag));
        if (!ok) break;
        tc_fence_after_sync();
        issue_s(g & 1, s);
        for (int it = 0; it < left; ++it, ++g) {
          const int s1 = s + 1 == kStages ? 0 : s + 1;
          const uint32_t ph1 = s1 == 0 ? ph ^ 1u : ph, buf = g & 1, pp = (g >> 1) & 1;
          const bool more = it + 1 < left;
          const bool v_ok = mbar_try_wait(&v_clean[s], ph), k_ok = !more || mbar_try_wait(&k_full[s1], ph1);
          const bool p_ok = mbar_test_wait(&p_full[buf], pp);
          if (more) {
            // Into the other buffer: the product that read the weights there was issued before.
            if (!all(k_ok || mbar_wait(&k_full[s1], ph1, abort_flag))) { ok = false; break; }
            tc_fence_after_sync();
            issue_s(buf ^ 1u, s1);
          }
          if (!all((p_ok || mbar_wait(&p_full[buf], pp, abort_flag)) && (v_ok || mbar_wait(&v_clean[s], ph, abort_flag)))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t b0 = sdesc_add(v_desc, s * L::kTile);
          const uint32_t d = tm + 256 + buf * 128, a = tm + buf * 128;
#pragma unroll
          for (int q = 0; q < kPPass; ++q)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_ts_f8_if(lead, d, a + q * 32 + kk * 8, sdesc_add(b0, kk * 4096), id_o,
                            (it > 1 || q > 0 || kk > 0) ? 1u : 0u);
          umma_commit_if(lead, &kv_empty[s]);
          s = s1;
          ph = ph1;
        }
        umma_commit_if(lead, unit_done);
        if (ok && g < count) walk.advance(p, left);
      }
      umma_commit_if(lead, mma_done);
      int drain = 0;
      mbar_wait(mma_done, 0, &drain);
    } else if (warp == 10) {
      cache_cleaner<R, kStages>(p, run, smem + L::kVOff, v_full, v_clean, abort_flag);
    }
  } else {
    regs_inc<208>();
    if (run.count > 0) {
      // ---------------------------------------------------------------- softmax (lane = copy, row)
      const int wg = warp / 4, quarter = warp % 4;  // even or odd tiles; keys 32 * quarter .. + 31 of a tile
      const uint32_t lane_base = tmem + ((quarter * 32) << 16);
      const uint32_t s_tmem = lane_base + wg * 128, o_tmem = lane_base + 256 + wg * 128;
      const int r = lane % R, stack = lane / R;  // row; part, and which R of the warp's 32 keys this lane computes
      const float down = pow2i(-4 * stack), down_q = pow2i(-4 * (stack % kQStack));
      int joins = 0;
      auto join = [&]() {  // all threads of these warps, bounded like every wait
        mbar_arrive(joint);
        return mbar_wait(joint, joins++ & 1, abort_flag);
      };
      // q of a unit: from memory to registers (ahead of time), and from there into the A operand, each row to its 128 / R
      // places, when the previous unit's scores are complete.
      constexpr int kVec = D * R > 256 * 8 ? D * R / (256 * 8) : 1;  // 8-element vectors per thread
      constexpr int kThreadsPerRow = D / (8 * kVec);
      const int row_q = threadIdx.x / kThreadsPerRow, piece = threadIdx.x % kThreadsPerRow;
      uint4 v[kVec];
      auto load_q = [&](const CacheItem& t, int hk) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row_q < t.rows) {
          const int row = t.row0 + row_q, qi = row / p.group, h = hk * p.group + row % p.group;
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                            ((static_cast<size_t>(t.b) * p.Sq + qi) * p.H + h) * D) +
                             piece * kVec;
#pragma unroll
          for (int i = 0; i < kVec; ++i) v[i] = src[i];
        }
      };
      // The row factors have two places, by the unit's parity: a warp may place unit u + 1's q while another still has to
      // read unit u's factors (a unit's last scores can be complete before every warp has begun it). The same place is
      // written again with unit u + 2's q, when every warp has passed unit u's joins and so read its factors.
      auto place_q = [&](int unit) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) amax = q_amax8<kBF16>(v[i], amax);
#pragma unroll
        for (int s = 1; s < kThreadsPerRow; s <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, s));
        float mul, back;
        if (!q_row_scale(amax, mul, back)) {
          back = __uint_as_float(kNanBits);
#pragma unroll
          for (int i = 0; i < kVec; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (row_q < R) {
          if (piece == 0) row_back[(unit & 1) * 32 + row_q] = back * p.scale_log2;
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            uint2 part[kQPass * kQStack];
            q_split8<kBF16, kQParts, kQStack>(v[i], mul, part);
#pragma unroll
            for (int q = kQParts; q < kQPass * kQStack; ++q) part[q] = make_uint2(0u, 0u);
            const int e8 = piece * kVec + i;  // 8-byte unit of the row
#pragma unroll
            for (int c = 0; c < 128 / R; ++c) {
              const int m = c * R + row_q;
              uint8_t* dst = smem + L::kQOff + m * 128 + ((e8 >> 1) ^ (m & 7)) * 16 + (e8 & 1) * 8;
#pragma unroll
              for (int q = 0; q < kQPass; ++q)
                *reinterpret_cast<uint2*>(dst + q * L::kTile) = part[q * kQStack + c % kQStack];
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_ready);
      };
      CacheWalk<R> walk;
      walk.start(p, run.first);
      load_q(walk.item, walk.at.hk);
      place_q(0);
      bool ok = join();
      for (int g = 0, unit = 0; ok && g < run.count; ++unit) {
        const CacheItem t = walk.item;
        const int hk = walk.at.hk, w0 = walk.at.w;
        const int left = min(run.count - g, t.n - w0);
        const float factor = row_back[(unit & 1) * 32 + r];
        const bool finite = factor == factor;  // else see q_row_scale
        const float c_row = finite ? factor : 0.f;
        const int row = t.row0 + min(r, t.rows - 1);
        const int aligned = t.c0 + row / p.group;
        const int from = p.win_left >= 0 ? aligned - p.win_left : 0;
        const bool more = g + left < run.count;
        if (more) {  // while the first scores are on their way
          walk.advance(p, left);
          load_q(walk.item, walk.at.hk);
        }
        float m = -INFINITY, l = 0.f;
        const int first = (wg - g) & 1;  // this warpgroup's first tile of the unit
        for (int it = first; it < left; it += 2) {
          const int gi = g + it, s = gi % kStages;
          const int tile0 = cache_key0(t, w0 + it), key0 = tile0 + 32 * quarter + R * stack;
          if (!mbar_wait(&s_full[wg], (gi >> 1) & 1, abort_flag) ||
              !mbar_wait(&k_full[s], (gi / kStages) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after_sync();
          // Scores of this lane's R keys: the parts' partial scores of the R * kQStack keys that contain them lie in
          // kQStack lanes of the row, which exchange halves until each has the sums of its own keys.
          float x[R];
          {
            float v[32];
            tmem_ld_x32(s_tmem + 32 * quarter, reinterpret_cast<uint32_t*>(v));
            if (kQStack < kStack) {
#pragma unroll
              for (int c = 0; c < 16; ++c) v[c] = stack & 2 ? v[16 + c] : v[c];
            }
            if (kQStack > 1) {
#pragma unroll
              for (int c = 0; c < R * kQStack; ++c) v[c] *= down_q;
            }
#pragma unroll
            for (int n = kQStack / 2; n > 0; n /= 2) {
              const bool upper = (stack & n) != 0;
#pragma unroll
              for (int c = 0; c < R * n; ++c) {
                const float keep = upper ? v[R * n + c] : v[c], send = upper ? v[c] : v[R * n + c];
                v[c] = keep + __shfl_xor_sync(0xffffffffu, send, R * n);
              }
            }
#pragma unroll
            for (int c = 0; c < R; ++c) x[c] = v[c];
          }
          // this lane's 16-key groups: one (R <= 16) or two
          const float* f = fac + s * 24 + 2 * quarter + R * stack / 16;
          const float a0 = c_row * f[0], lv0 = f[8], iv0 = f[16];
          const float a1 = R == 32 ? c_row * f[1] : a0, lv1 = R == 32 ? f[9] : lv0, iv1 = R == 32 ? f[17] : iv0;
#pragma unroll
          for (int c = 0; c < R; ++c) x[c] = fmaf(x[c], c < 16 ? a0 : a1, c < 16 ? lv0 : lv1);
          if (tile0 + 127 > t.c_min ||
              (p.win_left >= 0 && tile0 < t.c_max - p.win_left && tile0 + 127 >= p.sinks)) {
#pragma unroll
            for (int c = 0; c < R; ++c)
              if (key0 + c > aligned || (key0 + c < from && key0 + c >= p.sinks)) x[c] = -INFINITY;
          }
          float m_new = m;
#pragma unroll
          for (int c = 0; c < R; c += 2) m_new = fmax3(m_new, x[c], x[c + 1]);
#pragma unroll
          for (int n = 1; n < kStack; n *= 2) m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, R * n));
          if (__any_sync(0xffffffffu, m_new > m + kCacheLag)) {
            const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
            if (it >= 2) {
#pragma unroll
              for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                tmem_ld_x32(o_tmem + c0, reinterpret_cast<uint32_t*>(o));
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] *= alpha;
                tmem_st_x32(o_tmem + c0, reinterpret_cast<uint32_t*>(o));
              }
            }
            l *= alpha;
            m = m_new;
          }
          const float off = kCacheShift - (m == -INFINITY ? 0.f : m);
          float sum0 = 0.f, sum1 = 0.f;
          uint32_t part[kPPass * kStack][R / 4];
#pragma unroll
          for (int c = 0; c < R; c += 4) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2_approx(x[c + e] + off);
            (c < 16 ? sum0 : sum1) += (w[0] + w[1]) + (w[2] + w[3]);
            uint32_t code[kPParts];
            p_split4<kStack>(w[0], w[1], w[2], w[3], code);
#pragma unroll
            for (int q = 0; q < kPPass * kStack; ++q) part[q][c / 4] = q < kPParts ? code[q] : 0u;
          }
          // The row of P in product q holds part q * kStack + stack of the warp's 32 keys: the same lanes exchange parts.
          uint32_t pk[kPPass][8];
#pragma unroll
          for (int q = 0; q < kPPass; ++q) {
            uint32_t row_p[kStack][R / 4];
#pragma unroll
            for (int u = 0; u < R / 4; ++u) {
              if (kStack == 1) {
                row_p[0][u] = part[q][u];
              } else if (kStack == 2) {
                const uint32_t keep = stack ? part[2 * q + 1][u] : part[2 * q][u];
                const uint32_t send = stack ? part[2 * q][u] : part[2 * q + 1][u];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, send, R);
                row_p[0][u] = stack ? got : keep;
                row_p[kStack - 1][u] = stack ? keep : got;
              } else {
                const bool hi = (stack & 2) != 0, lo = (stack & 1) != 0;
                uint32_t half[2][2];  // [part within this lane's pair][keys of the lower, upper two lanes]
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint32_t keep = hi ? part[(2 + k) % (kPPass * kStack)][u] : part[k][u];
                  const uint32_t send = hi ? part[k][u] : part[(2 + k) % (kPPass * kStack)][u];
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, send, 2 * R);
                  half[k][0] = hi ? got : keep;
                  half[k][1] = hi ? keep : got;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint32_t keep = lo ? half[1][k] : half[0][k], send = lo ? half[0][k] : half[1][k];
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, send, R);
                  row_p[(2 * k) % kStack][u] = lo ? got : keep;
                  row_p[(2 * k + 1) % kStack][u] = lo ? keep : got;
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) pk[q][k] = row_p[k * 4 / R][k % (R / 4)];
          }
          l += sum0 * iv0 + sum1 * iv1;
          const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
          for (int q = 0; q < kPPass; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t at = s_tmem + q * 32 + 8 * k;
              if (k == quarter)
                tmem_st_x8(at, pk[q]);
              else
                tmem_st_x8(at, zero);
            }
          tmem_st_wait();
          tc_fence_before_sync();
          mbar_arrive(&p_full[wg]);
        }
        if (!ok) break;
        g += left;
        // ---- the unit's (or piece's) end. The next unit's q first: its scores can run during the join.
        q_m[warp * 32 + lane] = m;
        q_l[warp * 32 + lane] = finite || m == -INFINITY ? l : __uint_as_float(kNanBits);
        const bool whole = left == t.n;
        if (more) {
          // (the last tile's scores may be the other warpgroup's)
          if (!mbar_wait(&s_full[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
          place_q(unit + 1);
        }
        if (!join()) { ok = false; break; }
        float m_all = -INFINITY, l_all = 0.f;
#pragma unroll
        for (int q = 0; q < kCopies; ++q) m_all = fmaxf(m_all, q_m[q * R + r]);
        const float m_use = m_all == -INFINITY ? 0.f : m_all;
#pragma unroll
        for (int q = 0; q < kCopies; ++q)
          l_all += q_l[q * R + r] * ex2_approx(q_m[q * R + r] - m_use);
        float f = ex2_approx(m - m_use) * down;
        if (whole) f *= l_all == 0.f ? 0.f : 1.f / l_all;  // l = 0: no visible key (a NaN stays one)
        const size_t slot0 = static_cast<size_t>(cache_slot(blockIdx.x, w0)) * R;
        if (warp == 0 && static_cast<int>(lane) < t.rows) {
          if (whole) {
            const int h = hk * p.group + row % p.group, qi = row / p.group;
            p.lse[(static_cast<size_t>(t.b) * p.H + h) * p.Sq + qi] =
                l_all == 0.f ? -INFINITY : (m_all + log2f(l_all) - kCacheShift) * kLn2;
          } else {
            *reinterpret_cast<float2*>(p.part_ml + (slot0 + lane) * 2) = make_float2(m_all, l_all);
          }
        }
        if (!mbar_wait(unit_done, unit & 1, abort_flag)) { ok = false; break; }
        tc_fence_after_sync();
        // O: first the copies within a warp (the lanes of a row exchange halves of 32 columns until each has the sums of
        // R), then the warps, through shared memory.
        float* xo = reinterpret_cast<float*>(smem + L::kXOff);
        constexpr int kCols = L::kJoinCols, kStride = kCols + 4;
#pragma unroll 1
        for (int cb = 0; cb < D; cb += kCols) {
          if (cb > 0 && !join()) { ok = false; break; }
#pragma unroll 1
          for (int c0 = 0; c0 < kCols; c0 += 32) {
            float o[32];
            tmem_ld_x32(o_tmem + cb + c0, reinterpret_cast<uint32_t*>(o));
            // (A copy that saw no key of this row has f = 0, and weights 0: its O is 0. A warpgroup without a tile in
            // this unit has no O at all.)
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = first < left ? o[c] * f : 0.f;
#pragma unroll
            for (int n = 16 / R; n > 0; n /= 2) {
              const bool upper = (lane / R & n) != 0;
#pragma unroll
              for (int c = 0; c < R * n; ++c) {
                const float keep = upper ? o[R * n + c] : o[c], send = upper ? o[c] : o[R * n + c];
                o[c] = keep + __shfl_xor_sync(0xffffffffu, send, R * n);
              }
            }
            float* dst = xo + (warp * R + r) * kStride + c0 + (lane / R) * R;
#pragma unroll
            for (int c = 0; c < R; c += 4)
              *reinterpret_cast<float4*>(dst + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
          }
          if (!join()) { ok = false; break; }
          const int ro = threadIdx.x / (kCols / 4), col = threadIdx.x % (kCols / 4) * 4;
          if (ro < t.rows) {
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const float4 x = *reinterpret_cast<const float4*>(xo + (w * R + ro) * kStride + col);
              sum.x += x.x;
              sum.y += x.y;
              sum.z += x.z;
              sum.w += x.w;
            }
            if (whole) {
              const int rr = t.row0 + ro, qi = rr / p.group, h = hk * p.group + rr % p.group;
              uint16_t* dst =
                  static_cast<uint16_t*>(p.out) + ((static_cast<size_t>(t.b) * p.Sq + qi) * p.H + h) * D + cb + col;
              *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<kBF16>(sum.x, sum.y), pack2<kBF16>(sum.z, sum.w));
            } else {
              *reinterpret_cast<float4*>(p.part_o + (slot0 + ro) * D + cb + col) = sum;
            }
          }
        }
        if (!ok) break;
        tc_fence_before_sync();
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// ------------------------------------------------------------------------------- attention of many query rows
// Chunks of prompts: units of 256 rows (two 128-row Q tiles, each with its own softmax warpgroup, thread = row), as in
// the forward of fa_fwd.cuh: while one warpgroup runs the softmax of its tile the tensor core works on the other. With
// this many rows splitting every weight into 8-bit parts would cost more than converting V once: two converting warps
// turn each arrived tile of V into an fp16 tile (exact), the weights are fp16 in one rounding, and PV is a 16-bit
// product. K stays e4m3: q's parts are made once per unit, and the parts' products take as long as one 16-bit product
// (bf16). (Weights in parts: 788 us for 4096 tokens of a prompt of 8192, 32 heads on 8, bf16; K and V converted: 644 to
// 738 us; this: 511 us, where the forward on 16-bit K and V of that length takes 399 us. Traced, a pair of tiles takes
// 4480 cycles: the issue of its 32 products 2800, a softmax 2300 beside them.) V rows that no query sees are written as 0.
//
// Warps: 0-3 and 4-7 softmax of Q tiles 0 and 1, 8 TMA, 9 MMA, 10-11 conversion. TMEM columns: S0 [0,128), S1 [128,256),
// O0 [256,256+D), O1 [384,384+D); P_t overwrites the first 64 columns of S_t.
template <int D, bool kBF16>
struct CacheManySmem {
  static constexpr int kRows = 256, kStages = 2, kFac = 4;
  static constexpr int kQParts = kBF16 ? 2 : 3;
  static constexpr int kRaw = 16384;                  // 128 rows of e4m3, 128-byte swizzle rows (a part of q, K or V)
  static constexpr int kTile = 128 * D * 2;           // fp16 V: D / 64 chunks of 128-byte swizzle rows
  static constexpr int kQOff = 0;                     // [part][Q tile]
  static constexpr int kVOff = kQOff + kQParts * 2 * kRaw;
  static constexpr int kKRawOff = kVOff + kTile;      // [kStages]
  static constexpr int kVRawOff = kKRawOff + kStages * kRaw;
  static constexpr int kFacOff = kVRawOff + kStages * kRaw;
  static constexpr int kBarOff = kFacOff + kFac * 96;
  static constexpr int kNumBars = 3 * kStages + 2 + kFac + 11;
  static constexpr int kScanOff = kBarOff + kNumBars * 8;
  static constexpr int kMiscOff = kScanOff + static_cast<int>(sizeof(CacheScan));
  static constexpr int kAlloc = kMiscOff + 16 + 1024;
  static constexpr int kThreads = 384;
  static constexpr uint32_t kRegsSoftmax = 208, kRegsOther = 88;  // 2 * 128 * 208 + 128 * 88 = 384 * 168
  static constexpr uint32_t kTmemCols = 512;
  static constexpr bool kSplitP = D == 64;  // P handed over in two halves (as in fa_fwd.cuh)
  static_assert(kAlloc <= 232448, "shared memory");
};

template <int D, bool kBF16>
__global__ void __launch_bounds__(384, 1)
    fa_cache_many_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const CacheParams p) {
  using L = CacheManySmem<D, kBF16>;
  constexpr int kStages = L::kStages, kRows = L::kRows, kQParts = L::kQParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* k_raw = bars;                  // [kStages] K and V tiles arrived
  uint64_t* v_raw = k_raw + kStages;       // [kStages]
  uint64_t* raw_empty = v_raw + kStages;   // [kStages] K's products done, V converted
  uint64_t* v_full = raw_empty + kStages;  // fp16 V written
  uint64_t* v_empty = v_full + 1;          // its products done
  uint64_t* fac_full = v_empty + 1;        // [kFac]
  uint64_t* s_full = fac_full + L::kFac;   // [2]
  uint64_t* p_half = s_full + 2;           // [2] weights of keys 0..63 published (kSplitP)
  uint64_t* p_full = s_full + 4;           // [2]
  uint64_t* o_full = s_full + 6;           // [2]
  uint64_t* q_ready = s_full + 8;          // [2]
  uint64_t* mma_done = s_full + 10;
  float* fac = reinterpret_cast<float*>(smem + L::kFacOff);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const uint32_t warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_raw[s], 1);
      mbar_init(&v_raw[s], 1);
      mbar_init(&raw_empty[s], 65);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_half[t], 128);
      mbar_init(&p_full[t], 128);
      mbar_init(&o_full[t], 1);
      mbar_init(&q_ready[t], 128);
    }
    mbar_init(v_full, 64);
    mbar_init(v_empty, 1);
    for (int s = 0; s < L::kFac; ++s) mbar_init(&fac_full[s], 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_holder, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  const CacheRun run = cache_run<kRows, L::kThreads>(p, reinterpret_cast<CacheScan*>(smem + L::kScanOff));
  if (warp >= 8) {
    regs_dec<L::kRegsOther>();
    if (run.count == 0) {
    } else if (warp == 8) {
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      cache_producer<kRows, kStages, L::kFac>(p, run, tm_k, tm_v, smem + L::kKRawOff, smem + L::kVRawOff, fac, k_raw,
                                              v_raw, raw_empty, fac_full, abort_flag);
    } else if (warp == 9 && lane == 0) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t id_s = idesc_e4m3(128, 128, false, false);
      constexpr uint32_t id_o = idesc_f16(false, 128, D, false, true);
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem + L::kQOff), 16, 1024);
      const uint64_t k_desc = sdesc_sw128(smem_u32(smem + L::kKRawOff), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(smem + L::kVOff), 16384, 1024);
      auto issue_s = [&](int t, int g, bool last) {
        const uint64_t a0 = sdesc_add(q_desc, t * L::kRaw), b0 = sdesc_add(k_desc, (g % kStages) * L::kRaw);
#pragma unroll
        for (int q = 0; q < kQParts; ++q)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_ss_f8(tmem + t * 128, sdesc_add(a0, q * 2 * L::kRaw + kk * 32), sdesc_add(b0, kk * 32),
                       id_s | (part_is_e5m2(q, 1) ? kE5M2A : 0u), (q > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&s_full[t]);
        if (last) umma_commit(&raw_empty[g % kStages]);
      };
      auto issue_o = [&](int t, bool acc, int half) {
#pragma unroll
        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
          umma_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, sdesc_add(v_desc, kk * 2048), id_o,
                  (acc || kk > 0) ? 1u : 0u);
      };
      CacheWalk<kRows> walk;
      walk.start(p, run.first);
      int steps[2] = {0, 0}, units[2] = {0, 0};  // tiles and units each Q tile has taken part in
      bool ok = true;
      for (int g = 0; ok && g < run.count;) {
        const int left = min(run.count - g, walk.item.n - walk.at.w);  // tiles of this unit in the run
        const int nq = walk.item.rows > 128 ? 2 : 1;                   // Q tiles with rows
        ok = mbar_wait(&k_raw[g % kStages], (g / kStages) & 1, abort_flag);
        for (int t = 0; ok && t < nq; ++t) {
          ok = mbar_wait(&q_ready[t], units[t]++ & 1, abort_flag);
          if (!ok) break;
          tc_fence_after_sync();
          issue_s(t, g, t == nq - 1);
        }
        for (int it = 0; ok && it < left; ++it, ++g) {
          if (!mbar_wait(v_full, g & 1, abort_flag)) { ok = false; break; }
          bool next_k = false;
          for (int t = 0; t < nq; ++t) {
            const int u = steps[t]++;
            if (!mbar_wait(L::kSplitP ? &p_half[t] : &p_full[t], u & 1, abort_flag)) { ok = false; break; }
            tc_fence_after_sync();
            issue_o(t, it > 0, 0);
            if (L::kSplitP) {
              if (!mbar_wait(&p_full[t], u & 1, abort_flag)) { ok = false; break; }
              tc_fence_after_sync();
            }
            issue_o(t, true, 1);
            umma_commit(&o_full[t]);
            if (t == nq - 1) umma_commit(v_empty);
            if (it + 1 < left) {
              if (!next_k) {
                if (!mbar_wait(&k_raw[(g + 1) % kStages], ((g + 1) / kStages) & 1, abort_flag)) { ok = false; break; }
                tc_fence_after_sync();
                next_k = true;
              }
              issue_s(t, g + 1, t == nq - 1);
            }
          }
        }
        if (ok && g < run.count) walk.advance(p, left);
      }
      umma_commit(mma_done);
      int drain = 0;
      mbar_wait(mma_done, 0, &drain);
    } else if (warp >= 10) {
      // ---------------------------------------------------------------- conversion
      // A thread takes 16-byte pieces (16 codes) of one column of the tile; eight neighbouring threads take eight rows, so
      // that neither the reads nor the writes of the swizzled rows meet in a bank.
      constexpr int kPerRow = D / 16;
      const int t = threadIdx.x - 320, col = (t >> 3) % kPerRow, row0 = (t & 7) + 8 * ((t >> 3) / kPerRow);
      constexpr int kStep = 64 / kPerRow;  // tokens between a thread's pieces
      CacheWalk<kRows> walk;
      walk.start(p, run.first);
      auto convert = [&](const uint8_t* raw, uint8_t* tile, auto keep) {
        const int x = t & 7, unit = (col % 4) * 2;  // (row & 7 is the same for all of a thread's rows)
        raw += row0 * 128 + ((col ^ x) * 16);
        uint8_t* dst0 = tile + (col / 4) * 16384 + row0 * 128 + ((unit ^ x) * 16);
        uint8_t* dst1 = tile + (col / 4) * 16384 + row0 * 128 + (((unit + 1) ^ x) * 16);
#pragma unroll 8
        for (int i = 0; i < 128 / kStep; ++i) {
          uint4 v = *reinterpret_cast<const uint4*>(raw + i * kStep * 128);
          if (!keep(row0 + i * kStep)) v = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[2 * e] = f16x2_from_e4m3x2(w[e] & 0xffffu);
            h[2 * e + 1] = f16x2_from_e4m3x2(w[e] >> 16);
          }
          *reinterpret_cast<uint4*>(dst0 + i * kStep * 128) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst1 + i * kStep * 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
      };
      for (int g = 0; g < run.count; ++g) {
        const int s = g % kStages;
        const CacheItem& c = walk.item;
        const int key0 = cache_key0(c, walk.at.w);
        const bool got = mbar_wait(&v_raw[s], (g / kStages) & 1, abort_flag) &&
                         (g == 0 || mbar_wait(v_empty, (g - 1) & 1, abort_flag));
        if (!__all_sync(0xffffffffu, got)) break;
        // Rows that no query sees are 0: their weights are, but a stale byte may be a NaN.
        if (cache_ragged(p, c, key0))
          convert(smem + L::kVRawOff + s * L::kRaw, smem + L::kVOff, [&](int row) {
            return key0 + row <= c.key_hi && (key0 + row >= c.key_lo || key0 + row < p.sinks);
          });
        else
          convert(smem + L::kVRawOff + s * L::kRaw, smem + L::kVOff, [](int) { return true; });
        mbar_arrive(v_full);
        mbar_arrive(&raw_empty[s]);
        if (g + 1 < run.count) walk.advance(p, 1);
      }
    }
  } else {
    regs_inc<L::kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax warpgroups (thread = row)
    const int t = warp / 4;
    const uint32_t quarter = warp % 4;
    const int r_tile = quarter * 32 + lane;  // row within the Q tile = TMEM lane
    const uint32_t lane_base = tmem + ((quarter * 32) << 16);
    const uint32_t s_tmem = lane_base + t * 128, o_tmem = lane_base + 256 + t * 128;
    CacheWalk<kRows> walk;
    if (run.count > 0) walk.start(p, run.first);
    bool ok = true;
    int step = 0;  // tiles this Q tile has taken part in
    for (int g = 0; ok && g < run.count;) {
      const CacheItem& item = walk.item;
      const int hk = walk.at.hk, w0 = walk.at.w;
      const int left = min(run.count - g, item.n - w0);
      if (item.rows <= t * 128) {  // no rows in this Q tile
        g += left;
        if (g < run.count) walk.advance(p, left);
        continue;
      }
      const int r = t * 128 + r_tile;
      const bool valid = r < item.rows;
      const int row = item.row0 + min(r, item.rows - 1), qi = row / p.group, h = hk * p.group + row % p.group;
      // ---- q: this thread's row into the A operand (its previous unit's products are complete: the warpgroup has
      // seen their results)
      float c_row;
      bool finite;
      {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) + ((static_cast<size_t>(item.b) * p.Sq + qi) * p.H + h) * D);
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) amax = q_amax8<kBF16>(src[i], amax);
        float mul, back;
        finite = q_row_scale(amax, mul, back);
        c_row = back * fabsf(p.scale_log2);  // the scale's sign goes to q, so that larger scores mean larger weights
        mul = copysignf(mul, p.scale_log2);
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          uint2 part[kQParts];
          q_split8<kBF16, kQParts, 1>(finite ? src[i] : make_uint4(0u, 0u, 0u, 0u), mul, part);
          uint8_t* dst = smem + L::kQOff + t * L::kRaw + r_tile * 128 + ((i >> 1) ^ (r_tile & 7)) * 16 + (i & 1) * 8;
#pragma unroll
          for (int q = 0; q < kQParts; ++q) *reinterpret_cast<uint2*>(dst + q * 2 * L::kRaw) = part[q];
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_ready[t]);
      }
      // The factor of a group's scores. Never 0, because a masked score is -inf: a row of zeros (back = 2^-107) over a page of
      // zeros (scale 2^-50) would underflow. Scores are below 2^25, so at the smallest normal number they count as 0.
      auto factor = [&](float ks) { return fmaxf(c_row * ks, 1.17549435e-38f); };
      const int aligned = item.c0 + qi;
      const int from = p.win_left >= 0 ? aligned - p.win_left : 0;
      float m = -INFINITY, l = 0.f;
      for (int it = 0; it < left; ++it, ++g, ++step) {
        if (!mbar_wait(&s_full[t], step & 1, abort_flag) ||
            !mbar_wait(&fac_full[g % L::kFac], (g / L::kFac) & 1, abort_flag)) { ok = false; break; }
        if (it > 0 && !mbar_wait(&o_full[t], (step - 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after_sync();
        float x[128];
        tmem_ld_x128(s_tmem, reinterpret_cast<uint32_t*>(x));
        const float* f = fac + (g % L::kFac) * 24;  // ks, log2 vs, 1 / vs of the tile's eight key groups
        const int key0 = cache_key0(item, w0 + it);
        if (key0 + 127 > item.c_min || (p.win_left >= 0 && key0 < item.c_max - p.win_left && key0 + 127 >= p.sinks)) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (key0 + c > aligned || (key0 + c < from && key0 + c >= p.sinks)) x[c] = -INFINITY;
        }
        // The exponent of a weight is s a + log2 vs (a = c ks > 0 of its 16-key group), so a group's largest is that of
        // its largest s.
        float m_new = m;
#pragma unroll
        for (int gr = 0; gr < 8; ++gr) {
          float g0 = x[16 * gr], g1 = x[16 * gr + 1];
#pragma unroll
          for (int c = 2; c < 14; c += 4) {
            g0 = fmax3(g0, x[16 * gr + c], x[16 * gr + c + 1]);
            g1 = fmax3(g1, x[16 * gr + c + 2], x[16 * gr + c + 3]);
          }
          g0 = fmax3(g0, g1, fmaxf(x[16 * gr + 14], x[16 * gr + 15]));
          m_new = fmaxf(m_new, fmaf(g0, factor(f[gr]), f[8 + gr]));
        }
        if (__any_sync(0xffffffffu, m_new > m + kManyLag)) {
          const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
          if (it > 0) {
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              float o[32];
              tmem_ld_x32(o_tmem + c0, reinterpret_cast<uint32_t*>(o));
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] *= alpha;
              tmem_st_x32(o_tmem + c0, reinterpret_cast<uint32_t*>(o));
            }
            tmem_st_wait();
          }
          l *= alpha;
          m = m_new;
        }
        const float off = kManyShift - (m == -INFINITY ? 0.f : m);
        float lsum = 0.f;
        uint32_t pk[64];
#pragma unroll
        for (int gr = 0; gr < 8; ++gr) {
          const float a = factor(f[gr]), b = f[8 + gr] + off;
          const uint64_t a2 = f2_pack(a, a), b2 = f2_pack(b, b);
          uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
          for (int c = 16 * gr; c < 16 * gr + 16; c += 4) {
            float w0_, w1_, w2_, w3_;
            f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), a2, b2), w0_, w1_);
            f2_unpack(f2_fma(f2_pack(x[c + 2], x[c + 3]), a2, b2), w2_, w3_);
            w0_ = ex2_approx(w0_);
            w1_ = ex2_approx(w1_);
            w2_ = ex2_approx(w2_);
            w3_ = ex2_approx(w3_);
            sum2 = f2_add(sum2, f2_add(f2_pack(w0_, w1_), f2_pack(w2_, w3_)));
            pk[c / 2] = pack2_f16(w0_, w1_);
            pk[c / 2 + 1] = pack2_f16(w2_, w3_);
          }
          float s0, s1;
          f2_unpack(sum2, s0, s1);
          lsum = fmaf(s0 + s1, f[16 + gr], lsum);
          if (L::kSplitP && gr == 3) {
            tmem_st_x32(s_tmem, pk);
            tmem_st_wait();
            tc_fence_before_sync();
            mbar_arrive(&p_half[t]);
          }
        }
        if (L::kSplitP)
          tmem_st_x32(s_tmem + 32, pk + 32);
        else
          tmem_st_x64(s_tmem, pk);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&p_full[t]);
        l += lsum;
      }
      if (!ok) break;
      // ---- the unit's (or piece's) end
      if (!mbar_wait(&o_full[t], (step - 1) & 1, abort_flag)) { ok = false; break; }
      tc_fence_after_sync();
      const bool whole = left == item.n;
      if (!finite && m != -INFINITY) l = __uint_as_float(kNanBits);  // (see q_row_scale)
      const float inv = l == 0.f ? 0.f : whole ? 1.f / l : 1.f;
      const size_t slot = static_cast<size_t>(cache_slot(blockIdx.x, w0)) * kRows + r;
      uint16_t* orow = static_cast<uint16_t*>(p.out) + ((static_cast<size_t>(item.b) * p.Sq + qi) * p.H + h) * D;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        tmem_ld_x32(o_tmem + c0, reinterpret_cast<uint32_t*>(o));
        if (valid && whole) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) w[c / 2] = pack2<kBF16>(o[c] * inv, o[c + 1] * inv);
          uint4* dst = reinterpret_cast<uint4*>(orow + c0);
#pragma unroll
          for (int v = 0; v < 4; ++v) dst[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        } else if (valid) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + slot * D + c0);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v] = make_float4(o[4 * v] * inv, o[4 * v + 1] * inv, o[4 * v + 2] * inv, o[4 * v + 3] * inv);
        }
      }
      if (valid) {
        if (whole)
          p.lse[(static_cast<size_t>(item.b) * p.H + h) * p.Sq + qi] =
              l == 0.f ? -INFINITY : (m + log2f(l) - kManyShift) * kLn2;
        else
          *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(m, l);
      }
      tc_fence_before_sync();
      if (g < run.count) walk.advance(p, left);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

}  // namespace fa
