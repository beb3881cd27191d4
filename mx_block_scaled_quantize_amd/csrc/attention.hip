// Attention of new tokens over a paged MXFP8 key/value cache on gfx950: decoding
// steps and chunks of prompts in one call.
//
//   o = sum_j exp(c q.k_j - lse) v_j,   lse = ln sum_j exp(c q.k_j),   j in (p - window, p]
//
// All query heads that share a kv head, of all new tokens of a request, are rows
// of one problem (row = token * group + head within the group), so a key or value
// is read and decoded once for all of them.  One pass over the keys keeps, per
// row, a reference exponent m, the sum l of exp2(t - m) and the unnormalised
// output, t = c log2(e) q.k.
//
// The matrix unit takes S^T = K Q^T and O^T = V^T P^T in 16 x 16 x 32 steps:
//   - S^T leaves lane (q = lane % 16, g = lane / 16) with rows 4g .. 4g + 3 of a
//     16-key tile.  Row 4g + j of tile t of a 32-key step is made key 8g + 4t + j, so
//     the two tiles leave the lane with keys 8g .. 8g + 7, which is what it feeds as
//     P^T: the weights never leave their lane.
//   - K: a lane feeds 8 channels of one key; the order of the channels is free as
//     long as Q has the same, so it takes 16 contiguous bytes per 64 channels.
//   - V: a lane of row r holds dim / 16 contiguous channels of each of its 8 keys.
//     The scaled converter decodes two channels of one key at once with that
//     key's block scale; byte permutes then pair the keys, as the contraction wants.
// The scaled converters (V_CVT_SCALEF32_PK_{BF16,F16}_FP8) read only the exponent
// field of their scale operand (measured: sign and fraction bits change nothing,
// field 0 is 2^-127 and field 255 gives NaN, as E8M0 wants), so a scale byte needs
// one shift to be an operand.

#include "mx_device.hpp"
#include "mx_launch.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace mxk {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f_t __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h_t __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

constexpr float kLowest = -3.402823466e38f;
// The reference exponent of a row moves only when a score exceeds it by 2^kSlack.
constexpr float kSlack = 8.0f;
// F16 weights are kept 2^7 above the usual [0, 1], so that weights down to 2^-31 of the largest
// are not lost below F16's smallest subnormal; with the slack they stay under 2^15.
template <int DT> constexpr float kLift = DT == IN_F16 ? 7.0f : 0.0f;

// Requests of up to so many rows (tokens x group) are taken by workgroups whose waves split the keys.
constexpr int kFewRows = 32;

// Grid: x = kv head, y = place in the list of work, z = split.  The kv head runs
// fastest: neighbouring workgroups go to different XCDs, so with 8 kv heads each
// XCD's L2 serves one head's pages.
//
// A decoding call on short contexts is bound by latency: dependent loads, and code
// that no workgroup has run yet, which has to come from L2 first.  So
// what a workgroup runs once is kept short: no integer division (reciprocals come
// from the host), the page numbers are read beside the lengths and not after them.
struct AttnArgs {
  const void* q;
  int64_t q_ts, q_hs;
  const uint8_t *kc, *ks, *vc, *vs;
  int64_t pages;
  const int32_t* table;
  int64_t table_stride, table_cols;
  const int32_t* cu;
  const int32_t* lens;
  void* out;
  float* lse;
  float* part;                  // [tokens * heads][slots][dim] unnormalised outputs
  float* part_ml;               // [tokens * heads][slots][2] reference exponent and sum; a negative
                                // sum in slot 0: the row is done
  int64_t tokens, max_q, max_kv;
  int requests, heads, kv_heads, group, page;
  int window;                   // 0: none
  int slots;                    // partial results a row has room for
  // how requests of few and of many rows split their keys: how often, and the keys of a split (a multiple of 64)
  int few_splits, few_chunk, tile_splits, tile_chunk;
  float inv_group;              // 1 / group
  double inv_page16;            // 16 / page
  float c;                      // scale * log2(e)
  int tile_units;               // most row tiles that requests of many rows can have
};

template <int DT>
__device__ __forceinline__ v4f mfma16(u32x4_t a, u32x4_t b, v4f acc) {
  if constexpr (DT == IN_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), acc, 0, 0, 0);
}

// Two E4M3 codes (half `HI` of w) times 2^(exponent field of s - 127), in the type of q.
template <int DT, bool HI>
__device__ __forceinline__ uint32_t decode2(uint32_t w, uint32_t s) {
  if constexpr (DT == IN_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, __uint_as_float(s), HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, __uint_as_float(s), HI));
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const v2f v = {a, b};
  if constexpr (DT == IN_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf_t));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2h_t));
}

// The same, rounded towards 0.
template <int DT>
__device__ __forceinline__ uint32_t chop2(float a, float b) {
  if constexpr (DT == IN_BF16) return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
}

typedef uint16_t v2u_t __attribute__((ext_vector_type(2)));
// The larger, the smaller halves (of numbers that are not negative, which compare as their bits do).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u_t, a), __builtin_bit_cast(v2u_t, b)));
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(v2u_t, a), __builtin_bit_cast(v2u_t, b)));
}

// Differences of halves, 0 where they would be negative.
__device__ __forceinline__ uint32_t less2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(v2u_t, a), __builtin_bit_cast(v2u_t, b)));
}

// Half `HI` of a packed pair.
template <int DT, bool HI>
__device__ __forceinline__ float unpack(uint32_t w) {
  if constexpr (DT == IN_BF16) return __uint_as_float(HI ? w & 0xFFFF0000u : w << 16);
  else return float(__builtin_bit_cast(v2h_t, w)[HI ? 1 : 0]);
}

// A weight of 0 times a value that is infinite or NaN would be NaN for rows that do not see it.  Such
// elements are taken out of the product of weights and values; products of marks (1 in their places) with
// 1 for every key that a row sees count them for the rows that do, once with +inf and NaN marked and once
// with -inf and NaN, so that a NaN adds both infinities.
template <int DT> constexpr uint32_t kOneBits = DT == IN_BF16 ? 0x3F80u : 0x3C00u;

// Takes the elements that are infinite or NaN out of a decoded fragment and marks them.
template <int DT>
__device__ __forceinline__ void take_marks(u32x4_t& x, u32x4_t& plus, u32x4_t& minus) {
  // added to a half without its sign: its top bit is set from infinity on
  constexpr uint32_t kUp = (0x8000u - (DT == IN_BF16 ? 0x7F80u : 0x7C00u)) * 0x00010001u;
  auto halves = [](uint32_t top) { return (top << 1) - (top >> 15); };       // all bits of the halves whose top bit is set
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t size = x[j] & 0x7FFF7FFFu, sign = x[j] & 0x80008000u;
    const uint32_t odd = (size + kUp) & 0x80008000u, nan = (size + (kUp - 0x00010001u)) & odd;
    plus[j] = halves(odd & (~sign | nan)) & (kOneBits<DT> * 0x00010001u);
    minus[j] = halves(odd & (sign | nan)) & (kOneBits<DT> * 0x00010001u);
    x[j] &= ~halves(odd);
  }
}

// 0 for a count of 0, else infinity.
__device__ __forceinline__ float infinity_of(float count) { return count * 0x1p127f * 0x1p127f; }

// How a value row of D channels is dealt to the 16 lanes of a row of the matrix
// unit: kA contiguous channels each of the first 16 kA, then kB each of the rest,
// powers of two, so that a lane's run lies in one block of 32.
template <int D> struct Deal {
  static constexpr int kA = D >= 256 ? 16 : D >= 128 ? 8 : 4;
  static constexpr int kB = D / 16 - kA;
  static constexpr int kWordsA = kA / 4, kWordsB = kB ? 1 : 0, kWords = kWordsA + kWordsB;
  static constexpr int kScales = kB ? 2 : 1;
};

// The least power of two beyond the type of q, as a scale code, and the least scale code with which an element
// of 2^8 (E4M3's largest is 448) gets there.
template <int DT> constexpr uint32_t kBeyond = DT == IN_F16 ? 127 + 16 : 127 + 128;
template <int DT> constexpr uint32_t kWideScale = kBeyond<DT> - 8;

// The least magnitude of an E4M3 code that is NaN or, with a scale code, beyond the type of q: without compares,
// whose masks would not fit the scalar registers where many keys are looked at.
template <int DT>
__device__ __forceinline__ uint32_t least_odd_code(uint32_t scale) {
  const int e = int(kBeyond<DT> - scale);        // exponent from which an element is
  const int normal = min((e + 7) * 8, 0x7F), subnormal = 8 >> min(max(-6 - e, 0), 3);
  return uint32_t(max(normal, subnormal)) & (((scale + 1) >> 8) - 1);     // 0 for the scale NaN
}

__device__ __forceinline__ uint32_t any_nan_code(uint32_t w) {   // nonzero if a byte is an E4M3 NaN
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// The request that holds unit `want` of a list in which request i has count(new tokens of i) units;
// `want` becomes the unit's place within it.  -1: the list is shorter.  A launch then has no workgroups
// without work between those with some, which the dispatcher would deal to the same few shader engines
// where requests of one kind recur at a stride.
template <class F>
__device__ __forceinline__ int find_request(const AttnArgs& g, int& want, F count) {
  const int lane = threadIdx.x & 63;
  for (int r0 = 0; r0 < g.requests; r0 += 64) {
    int n = 0;
    if (r0 + lane < g.requests) {
      const int t0 = min(max(g.cu[r0 + lane], 0), int(g.tokens));
      n = count(min(max(g.cu[r0 + lane + 1], t0), int(g.tokens)) - t0);
    }
    int sum = n;                                 // of this and the lanes before
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(sum, off, 64);
      if (lane >= off) sum += x;
    }
    const uint64_t at = __ballot(sum > want);
    if (at) {
      const int i = __builtin_ctzll(at);
      want -= __builtin_amdgcn_readlane(sum - n, i);
      return r0 + i;
    }
    want -= __builtin_amdgcn_readlane(sum, 63);
  }
  return -1;
}

// Page table column of a key: floor(x / d) as (x + 1/2) / d in FP64 (x < 2^27).
__device__ __forceinline__ int page_column(const AttnArgs& g, int key) {
  return int((double(key >> 4) + 0.5) * g.inv_page16);
}

// Entry of a column of a request's row of the page table; -1 past its end.
__device__ __forceinline__ int page_entry(const AttnArgs& g, const int32_t* __restrict__ table, int col) {
  return col < g.table_cols ? table[col] : -1;
}

// Row group (16 rows of one page and head) of keys key .. key + 15 in page `entry`, column col: -1
// where no row sees them (not read), -2 where the page number is out of range.
__device__ __forceinline__ int row_group(const AttnArgs& g, int hk, int key, int col, int entry, int lo, int hi) {
  if (key >= hi || key + 16 <= lo) return -1;
  if (entry < 0 || entry >= g.pages) return -2;
  return (entry * g.kv_heads + hk) * (g.page >> 4) + ((key - col * g.page) >> 4);
}

// NaN for all rows of one kv head of a request that exceeds what the caller announced.
template <int DT, int D>
__device__ __forceinline__ void refuse_request(const AttnArgs& g, int64_t t0, int64_t rows, int hk) {
  const float nan = __uint_as_float(0x7FC00000u);
  for (int64_t i = threadIdx.x; i < rows; i += blockDim.x) {
    const int64_t row = (t0 + i / g.group) * g.heads + hk * g.group + i % g.group;
    for (int d = 0; d < D; ++d) static_cast<uint16_t*>(g.out)[row * D + d] = DT == IN_BF16 ? 0x7FC0u : 0x7E00u;
    if (g.lse) g.lse[row] = nan;
    if (g.slots > 1) g.part_ml[row * g.slots * 2 + 1] = -1.0f;
  }
}

// A split without keys adds nothing to rows [row0, row1).
__device__ __forceinline__ void empty_split(const AttnArgs& g, int64_t t0, int64_t row0, int64_t row1, int hk, int split) {
  for (int64_t i = row0 + threadIdx.x; i < row1; i += blockDim.x) {
    const int64_t row = (t0 + i / g.group) * g.heads + hk * g.group + i % g.group;
    g.part_ml[(row * g.slots + split) * 2] = kLowest;
    g.part_ml[(row * g.slots + split) * 2 + 1] = 0.0f;
  }
}

// Log-sum-exp of reference exponent m and sum l.
__device__ __forceinline__ float log_sum(float m, float l) {
  const float inf = __builtin_inff();
  return l == 0.0f ? -inf : m == inf ? inf : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// A row's statistics: the final ones of an unsplit request, or those of a split; the last
// split also clears the slots that this kind of request does not use.
template <int DT>
__device__ __forceinline__ void put_stats(const AttnArgs& g, int64_t row, int split, int splits, float m, float l) {
  float* ml = g.part_ml + (row * g.slots + split) * 2;
  if (splits > 1) {
    ml[0] = m;
    ml[1] = l;
    for (int i = splits; split == splits - 1 && i < g.slots; ++i) {
      ml[2 * (i - split)] = kLowest;
      ml[2 * (i - split) + 1] = 0.0f;
    }
    return;
  }
  if (g.lse) g.lse[row] = log_sum(m, l);
  if (g.slots > 1) ml[1] = -1.0f;
}

// ---------------------------------------------------------------------------
// Few rows a request: the waves of a workgroup split the keys
// ---------------------------------------------------------------------------
// How the scale bytes of a step come: with 2 or 4 blocks to a row, whole words are
// loaded and a rotation brings the byte a lane needs under the exponent field;
// otherwise byte by byte.
template <int D> struct ScaleLoad {
  static constexpr bool kWordsK = D == 64 || D == 128 || D == 256, kWordsV = D == 64 || D == 128;
  static constexpr int kK = D == 256 ? 2 : kWordsK ? 1 : (D + 63) / 64;   // registers for a key
  static constexpr int kV = kWordsV ? D / 16 : 8 * Deal<D>::kScales;      // for a lane's 8 keys' values
};

// LDS of join_waves: the waves' outputs, rows 4 floats apart beyond D so that the 16
// rows of a tile meet different banks, and their statistics.
template <int D, int NQ, int NW> struct FewLds {
  float o[NW][NQ * 16][D + 4];
  float m[NW][NQ * 16], l[NW][NQ * 16];
};

// One request, kv head and split of up to 16 NQ rows.  Wave w takes the 32-key steps
// w, w + NW, ... of the split: no wave waits for another before the end.  Bound by
// memory: a step of 128 channels is 8.4 KB and some 340 vector instructions, and the vector
// units are busy 26% of the time, the matrix units 9% (64 requests of 8192 keys).  The next step's
// bytes are loaded while this one is computed where the registers allow it (1 request of 1021
// keys: 9.6 us, without 11.6; long contexts differ by 1%).  Measured with 32 query and 8 kv heads of
// 128 channels: 64 requests of 1650 to 8192 keys 136 us (4.9 TB/s), 4 of 118000 to 131072 keys 185 us
// (5.7 TB/s), 16 of 5 new tokens over 8192 keys 60 us.  192 and 256 channels: 64 requests of up to
// 8192 keys 204 and 260 us.
template <int DT, int D, int NQ, int NW>
__device__ __forceinline__ void few_rows(const AttnArgs& g, int req, int split, FewLds<D, NQ, NW>& lds) {
  using L = Deal<D>;
  using SL = ScaleLoad<D>;
  using T = uint16_t;
  constexpr int kFrags = D / 32;                 // K steps of S^T
  constexpr int kTiles = D / 16;                 // 16-channel tiles of O^T
  constexpr int kRows = NQ * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, quarter = lane >> 4;

  const int hk = blockIdx.x, G = g.group;
  const int32_t* table = g.table + req * g.table_stride;
  // without a window the split's first key does not depend on the length: its pages come meanwhile
  int key = split * g.few_chunk + lane * 16, col = page_column(g, key);
  int entry = page_entry(g, table, col);
  const int t0 = min(max(g.cu[req], 0), int(g.tokens)), t1 = min(max(g.cu[req + 1], t0), int(g.tokens));
  const int m = t1 - t0, kv = max(g.lens[req], 0);
  if (__builtin_expect(m > g.max_q || kv > g.max_kv, 0)) {   // not what the grid was sized for
    if (split == 0) refuse_request<DT, D>(g, t0, int64_t(m) * G, hk);
    return;
  }
  const int rows = m * G;
  if (rows == 0) return;
  // keys that some row sees
  const int hi_all = kv;
  const int lo = g.window ? max(kv - m - g.window + 1, 0) : 0;
  const int64_t start64 = int64_t(lo & ~31) + int64_t(split) * g.few_chunk;
  if (__builtin_expect(split > 0 && start64 >= hi_all, 0)) {
    empty_split(g, t0, 0, rows, hk, split);
    if (split == g.few_splits - 1)
      for (int i = g.few_splits; i < g.slots; ++i) empty_split(g, t0, 0, rows, hk, i);
    return;
  }
  const int start = int(start64), hi = int(min(int64_t(hi_all), start64 + g.few_chunk));

  // this lane's rows: where q is, and the keys (first, last] a row sees
  int last[NQ], first[NQ], orow[NQ];
  u32x4_t qf[NQ][kFrags];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int row = n * 16 + r;
    const int rr = min(row, rows - 1);
    const int i = int((float(rr) + 0.5f) * g.inv_group), head = hk * G + (rr - i * G);   // rr < 32: exact
    orow[n] = (t0 + i) * g.heads + head;
    last[n] = row < rows ? kv - m + i : -1;
    first[n] = g.window ? max(kv - m + i - g.window + 1, 0) : 0;
    const T* q = static_cast<const T*>(g.q) + int64_t(t0 + i) * g.q_ts + head * g.q_hs;
#pragma unroll
    for (int s = 0; s < kFrags; ++s) {
      const int d = s / 2 * 64 + (s / 2 * 2 + 1 < kFrags ? 16 * quarter + 8 * (s & 1) : 8 * quarter);
      qf[n][s] = *reinterpret_cast<const u32x4_t*>(q + d);
    }
  }
  // keys in [all_from, all_to) are seen by every row
  const int all_from = g.window ? max(kv - g.window, 0) : 0, all_to = min(hi, kv - m + 1);

  v4f o[NQ][kTiles];
  float mref[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    mref[n] = kLowest;
    l[n] = 0.0f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) o[n][t] = v4f{0, 0, 0, 0};
  }

  // ---- one 32-key step as it lies in memory
  struct Raw {
    uint32_t k[2][kFrags * 2], ks[2][SL::kK];
    uint32_t v[8][L::kWords], vs[SL::kV];
  };
  // row group of keys 16 i .. 16 i + 15 of the current window of 1024 keys, held by lane i
  int window = 0;
  if (g.window) {
    key = start + lane * 16;
    col = page_column(g, key);
    entry = page_entry(g, table, col);
  }
  int groups = row_group(g, hk, key, col, entry, lo, hi);
  const int blk_a = (L::kA * r) / 32, blk_b = (16 * L::kA + L::kB * r) / 32;   // blocks of the lane's runs
  auto load = [&](Raw& raw, int step) {
    if (__builtin_expect(step >> 5 != window, 0)) {
      window = step >> 5;
      key = start + 1024 * window + lane * 16;
      col = page_column(g, key);
      groups = row_group(g, hk, key, col, page_entry(g, table, col), lo, hi);
    }
    const int ga = __builtin_amdgcn_readlane(groups, 2 * (step & 31)), gb = __builtin_amdgcn_readlane(groups, 2 * (step & 31) + 1);
    if (__builtin_expect((ga & gb) >= 0, 1)) {   // a group that is not read borrows the other's addresses
      const int64_t a16 = int64_t(ga < 0 ? gb : ga) * 16, b16 = int64_t(gb < 0 ? ga : gb) * 16;
      const int64_t krow = ((r & 8) ? b16 : a16) + 8 * ((r >> 2) & 1) + (r & 3);
      const int64_t vrow = ((quarter & 2) ? b16 : a16) + 8 * (quarter & 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint8_t* k = g.kc + krow * D + 4 * t * D;
        const uint8_t* s = g.ks + krow * (D / 32) + 4 * t * (D / 32);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
          const uint4 w = *reinterpret_cast<const uint4*>(k + 64 * u + 16 * quarter);
          raw.k[t][4 * u] = w.x; raw.k[t][4 * u + 1] = w.y; raw.k[t][4 * u + 2] = w.z; raw.k[t][4 * u + 3] = w.w;
          if constexpr (!SL::kWordsK) raw.ks[t][u] = s[2 * u + (quarter >> 1)];
        }
        if constexpr (D == 64) raw.ks[t][0] = *reinterpret_cast<const uint16_t*>(s);
        if constexpr (D == 128) raw.ks[t][0] = *reinterpret_cast<const uint32_t*>(s);
        if constexpr (D == 256) {
          const uint2 w = *reinterpret_cast<const uint2*>(s);
          raw.ks[t][0] = w.x; raw.ks[t][1] = w.y;
        }
        if constexpr (D % 64) {
          const uint2 w = *reinterpret_cast<const uint2*>(k + D / 64 * 64 + 8 * quarter);
          raw.k[t][kFrags * 2 - 2] = w.x; raw.k[t][kFrags * 2 - 1] = w.y;
          raw.ks[t][SL::kK - 1] = s[D / 32 - 1];
        }
      }
      const uint8_t* v = g.vc + vrow * D;
      const uint8_t* s = g.vs + vrow * (D / 32);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t* a = v + j * D + L::kA * r;
        if constexpr (L::kA == 4) {
          raw.v[j][0] = *reinterpret_cast<const uint32_t*>(a);
        } else if constexpr (L::kA == 8) {
          const uint2 w = *reinterpret_cast<const uint2*>(a);
          raw.v[j][0] = w.x; raw.v[j][1] = w.y;
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(a);
          raw.v[j][0] = w.x; raw.v[j][1] = w.y; raw.v[j][2] = w.z; raw.v[j][3] = w.w;
        }
        if constexpr (L::kB) {
          const uint8_t* e = v + j * D + 16 * L::kA + L::kB * r;
          if constexpr (L::kB == 4) raw.v[j][L::kWordsA] = *reinterpret_cast<const uint32_t*>(e);
          else raw.v[j][L::kWordsA] = *reinterpret_cast<const uint16_t*>(e);
        }
        if constexpr (!SL::kWordsV) {
          raw.vs[j] = s[j * (D / 32) + blk_a];
          if constexpr (L::kB) raw.vs[8 + j] = s[j * (D / 32) + blk_b];
        }
      }
      if constexpr (SL::kWordsV) {
#pragma unroll
        for (int w = 0; w < SL::kV / 4; ++w) {
          const uint4 x = reinterpret_cast<const uint4*>(s)[w];
          raw.vs[4 * w] = x.x; raw.vs[4 * w + 1] = x.y; raw.vs[4 * w + 2] = x.z; raw.vs[4 * w + 3] = x.w;
        }
      }
    }
    if (__builtin_expect((ga | gb) < 0, 0)) {    // keys of a bad page are NaN, and so is what sees them; its values count as 0
      const int grp = (r & 8) ? gb : ga;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int u = 0; u < kFrags * 2; ++u) raw.k[t][u] = grp >= 0 ? raw.k[t][u] : 0x7F7F7F7Fu;
#pragma unroll
        for (int u = 0; u < SL::kK; ++u) raw.ks[t][u] = grp >= 0 ? raw.ks[t][u] : 0x7F7F7F7Fu;
      }
      const bool none = ((quarter & 2) ? gb : ga) < 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int w = 0; w < L::kWords; ++w) raw.v[j][w] = none ? 0u : raw.v[j][w];
#pragma unroll
      for (int w = 0; w < SL::kV; ++w) raw.vs[w] = none ? 0x7F7F7F7Fu : raw.vs[w];
    }
  };
  // scale operand of fragments 2 u, 2 u + 1 of tile t's keys; of key j's values, first or second run
  auto k_scale = [&](const Raw& raw, int t, int u) -> uint32_t {
    if constexpr (SL::kWordsK) {
      const uint32_t w = raw.ks[t][u / 2];
      return __builtin_amdgcn_alignbit(w, w, 16 * (u & 1) + 8 * (quarter >> 1) + 9);
    } else {
      return raw.ks[t][u] << 23;
    }
  };
  auto v_scale = [&](const Raw& raw, int j, int run) -> uint32_t {
    if constexpr (D == 64) return __builtin_amdgcn_alignbit(raw.vs[j / 2], raw.vs[j / 2], 16 * (j & 1) + 8 * blk_a + 9);
    else if constexpr (D == 128) return __builtin_amdgcn_alignbit(raw.vs[j], raw.vs[j], 8 * blk_a + 9);
    else return raw.vs[8 * run + j] << 23;
  };

  auto compute = [&](Raw& raw, int key0) {
    // ---- S^T
    v4f s[NQ][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      u32x4_t kf[kFrags];
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        const uint32_t sc = k_scale(raw, t, f / 2);
        kf[f] = u32x4_t{decode2<DT, false>(raw.k[t][2 * f], sc), decode2<DT, true>(raw.k[t][2 * f], sc),
                        decode2<DT, false>(raw.k[t][2 * f + 1], sc), decode2<DT, true>(raw.k[t][2 * f + 1], sc)};
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        s[n][t] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int f = 0; f < kFrags; ++f) s[n][t] = mfma16<DT>(kf[f], qf[n][f], s[n][t]);
      }
    }
    uint32_t vsc[8][L::kScales];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int w = 0; w < L::kScales; ++w) vsc[j][w] = v_scale(raw, j, w);
    // decodes channels of word w of the lane's run, all 8 keys, into two fragments; code(j, w, run) and
    // scale(j, run) are key j's word and scale operand
    auto fragments = [&](int w, auto hi_half, auto code, auto scale, u32x4_t& a, u32x4_t& c) {
      constexpr bool HI = decltype(hi_half)::value;
      const int run = L::kScales > 1 && w >= L::kWordsA ? 1 : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = decode2<DT, HI>(code(2 * j, w, run), scale(2 * j, run));
        const uint32_t y = decode2<DT, HI>(code(2 * j + 1, w, run), scale(2 * j + 1, run));
        a[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        c[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
      }
    };
    auto for_tiles = [&](auto code, auto scale, auto f) {   // f(tile, fragment)
#pragma unroll
      for (int w = 0; w < L::kWords; ++w) {
        u32x4_t a, c;
        fragments(w, std::false_type{}, code, scale, a, c);
        f(4 * w, a); f(4 * w + 1, c);
        if (4 * w + 2 < kTiles) {
          fragments(w, std::true_type{}, code, scale, a, c);
          f(4 * w + 2, a); f(4 * w + 3, c);
        }
      }
    };
    // ---- masks: only a step that some row does not see whole needs them
    const bool edge = key0 + 32 > all_to || key0 < all_from;
    if (edge) {
      // key 8 quarter + j of the step is seen by row n iff unsigned(j - from) < many
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const uint32_t from = uint32_t(first[n] - key0 - 8 * quarter);
        const uint32_t many = uint32_t(max(min(last[n], hi - 1) - first[n] + 1, 0));
#pragma unroll
        for (int j = 0; j < 8; ++j) s[n][j >> 2][j & 3] = uint32_t(j) - from < many ? s[n][j >> 2][j & 3] : -__builtin_inff();
      }
      // values that no row sees may be anything; the weight 0 must not meet an infinity or a NaN there
      const uint32_t from = uint32_t(lo - key0 - 8 * quarter), many = uint32_t(max(hi - lo, 0));
      uint32_t nans = 0, widest = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool keep = uint32_t(j) - from < many;
#pragma unroll
        for (int w = 0; w < L::kWords; ++w) {
          raw.v[j][w] = keep ? raw.v[j][w] : 0u;
          nans |= any_nan_code(raw.v[j][w]);
        }
#pragma unroll
        for (int w = 0; w < L::kScales; ++w) {
          vsc[j][w] = keep ? vsc[j][w] : 127u << 23;
          widest = umax(widest, vsc[j][w] & 0x7F800000u);
        }
      }
      // values that are infinite or NaN go to the rows that see them; what is left of the step has none
      if (__builtin_expect(__ballot(nans != 0 || widest >= kWideScale<DT> << 23) != 0, 0)) {
        // all bits of the bytes of a word that are infinite or NaN; of those that are NaN
        auto bytes = [](uint32_t top) { return (top << 1) - (top >> 7); };      // top bits to whole bytes
        auto odd = [&](int j, int w, int run) {
          asm volatile("" : "+v"(raw.v[j][w]), "+v"(vsc[j][run]));     // computed anew at every use: kept, it would take registers
          return ((raw.v[j][w] & 0x7F7F7F7Fu) + (0x80u - least_odd_code<DT>((vsc[j][run] >> 23) & 255u)) * 0x01010101u) & 0x80808080u;
        };
        auto nan = [&](int j, int w, int run) {
          return any_nan_code(raw.v[j][w]) | ((((vsc[j][run] >> 23) & 255u) + 1) >> 8) * 0x80808080u;
        };
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const uint32_t from = uint32_t(first[n] - key0 - 8 * quarter);
          const uint32_t many = uint32_t(max(min(last[n], hi - 1) - first[n] + 1, 0));
          u32x4_t see;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            see[j] = (uint32_t(2 * j) - from < many ? kOneBits<DT> : 0u) | (uint32_t(2 * j + 1) - from < many ? kOneBits<DT> << 16 : 0u);
#pragma unroll
          for (int minus = 0; minus < 2; ++minus) {
            const uint32_t sign = minus ? 0u : 0x80808080u;
            const float big = minus ? -0x1p127f : 0x1p127f;
            for_tiles([&](int j, int w, int run) {       // marks are E4M3 ones at scale 1
                        return bytes(odd(j, w, run) & ((raw.v[j][w] ^ sign) | nan(j, w, run))) & 0x38383838u;
                      }, [&](int, int) { return 127u << 23; }, [&](int t, u32x4_t a) {
                        const v4f hits = mfma16<DT>(a, see, v4f{0, 0, 0, 0});
#pragma unroll
                        for (int v = 0; v < 4; ++v) o[n][t][v] += hits[v] * big * 0x1p127f;
                        __builtin_amdgcn_sched_barrier(0);   // one tile at a time: this path shall cost no registers
                      });
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int w = 0; w < L::kWords; ++w) raw.v[j][w] &= ~bytes(odd(j, w, L::kScales > 1 && w >= L::kWordsA ? 1 : 0));
#pragma unroll
          for (int w = 0; w < L::kScales; ++w) vsc[j][w] = (vsc[j][w] & 0x7F800000u) == 0x7F800000u ? 127u << 23 : vsc[j][w];
        }
      }
    }
    // ---- reference exponents
    bool grow = false;
    float top[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      top[n] = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                     fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3]))) * g.c;
      grow |= top[n] > mref[n] + (kLift<DT> + kSlack);
    }
    if (__ballot(grow)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float x = top[n];
        x = fmaxf(x, __shfl_xor(x, 16, 64));
        x = fmaxf(x, __shfl_xor(x, 32, 64));
        const float next = fmaxf(mref[n], x - kLift<DT>);
        // before the first score there is nothing to rescale but infinities, which 0 would make NaN
        const float a = mref[n] == next || mref[n] == kLowest ? 1.0f : __builtin_amdgcn_exp2f(mref[n] - next);
        mref[n] = next;
        l[n] *= a;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[n][t] *= a;
      }
    }
    // ---- weights, in two terms of the type of q: one alone is off by up to 2^-9 (BF16), which outputs of
    // the same type would show (error against 64 bits 0.0023, with both 0.0017, the outputs' own rounding).
    // The second product costs 1% where memory bounds (64 requests of 8192 keys: 135.0 us without, 136.5 with).
    // The first term is chopped and the second kept above 0 where the first is (at 2^-16 of it for BF16, from the
    // bits of its exponent; at 2^-24 for F16), so that an infinite value that every row sees makes infinities
    // and no NaN: 0 times infinity.  A step that some row does not see whole has none left, and weights of 0
    // have to stay 0 in any.
    const uint32_t least = DT == IN_BF16 ? (edge ? 0xFFFFFFFFu : 0x08000800u) : edge ? 0u : 0x00010001u;
    u32x4_t p[NQ], rest[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][j >> 2][j & 3], g.c, -mref[n]));
      l[n] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[n][j] = chop2<DT>(e[2 * j], e[2 * j + 1]);
        const uint32_t lost = pack2<DT>(e[2 * j] - unpack<DT, false>(p[n][j]), e[2 * j + 1] - unpack<DT, true>(p[n][j]));
        rest[n][j] = max2(lost, DT == IN_BF16 ? less2(p[n][j], least) : min2(p[n][j], least));
      }
    }
    // ---- O^T
    for_tiles([&](int j, int w, int) { return raw.v[j][w]; }, [&](int j, int run) { return vsc[j][run]; }, [&](int t, u32x4_t a) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) o[n][t] = mfma16<DT>(a, rest[n], mfma16<DT>(a, p[n], o[n][t]));
    });
  };

  const int steps = (hi - start + 31) / 32;
  if (wave < steps) {
    constexpr bool kAhead = D * NQ <= 128;       // two steps' bytes fit the registers
    Raw raw;
    if constexpr (kAhead) load(raw, wave);
    for (int step = wave; step < steps; step += NW) {
      if constexpr (kAhead) {
        Raw next;                                // not from raw: that would wait for raw's loads
        if (step + NW < steps) load(next, step + NW);
        compute(raw, start + 32 * step);
        raw = next;
      } else {
        load(raw, step);
        compute(raw, start + 32 * step);
      }
    }
  }

  // ---- join the waves: every wave brings its outputs to the common reference exponent
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
    if (quarter == 0) { lds.m[wave][n * 16 + r] = mref[n]; lds.l[wave][n * 16 + r] = l[n]; }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    // quarter i reads waves i, i + 4, ...
    float mw[NW / 4], lw[NW / 4], top = kLowest, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < NW / 4; ++k) {
      mw[k] = lds.m[quarter + 4 * k][n * 16 + r];
      lw[k] = lds.l[quarter + 4 * k][n * 16 + r];
      top = fmaxf(top, mw[k]);
    }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
#pragma unroll
    for (int k = 0; k < NW / 4; ++k)
      sum += lw[k] == 0.0f ? 0.0f : mw[k] == top ? lw[k] : lw[k] * __builtin_amdgcn_exp2f(mw[k] - top);
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    float a = mref[n] == top ? 1.0f : __builtin_amdgcn_exp2f(mref[n] - top);
    if (g.few_splits == 1) a = sum == 0.0f ? 0.0f : a * __builtin_amdgcn_rcpf(sum);
    if (wave == 0 && quarter == 0 && n * 16 + r < rows) put_stats<DT>(g, orow[n], split, g.few_splits, top, sum);
    // the lane holds channels kA (4 quarter + v) + t of the first run, likewise of the second
    float* dst = lds.o[wave][n * 16 + r];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
#pragma unroll
      for (int t = 0; t < L::kA; t += 4)
        *reinterpret_cast<v4f*>(dst + L::kA * (4 * quarter + v) + t) =
            v4f{o[n][t][v], o[n][t + 1][v], o[n][t + 2][v], o[n][t + 3][v]} * a;
      if constexpr (L::kB == 4)
        *reinterpret_cast<v4f*>(dst + 16 * L::kA + 4 * (4 * quarter + v)) =
            v4f{o[n][L::kA][v], o[n][L::kA + 1][v], o[n][L::kA + 2][v], o[n][L::kA + 3][v]} * a;
      if constexpr (L::kB == 2)
        *reinterpret_cast<v2f*>(dst + 16 * L::kA + 2 * (4 * quarter + v)) = v2f{o[n][L::kA][v], o[n][L::kA + 1][v]} * a;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += 64 * NW) {
    const int row = i / (D / 4), d = i % (D / 4) * 4;
    v4f x = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < NW; ++w) x += *reinterpret_cast<const v4f*>(&lds.o[w][row][d]);
    const int at = int((float(row) + 0.5f) * g.inv_group);
    const int64_t to = int64_t(t0 + at) * g.heads + hk * G + (row - at * G);
    if (g.few_splits == 1)
      *reinterpret_cast<u32x2_t*>(static_cast<T*>(g.out) + to * D + d) = u32x2_t{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])};
    else
      *reinterpret_cast<v4f*>(g.part + (to * g.slots + split) * D + d) = x;
  }
}

template <int DT, int D, int NQ, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2))) void attention_few_kernel(const AttnArgs g) {
  __shared__ FewLds<D, NQ, NW> lds;
  few_rows<DT, D, NQ, NW>(g, blockIdx.y, blockIdx.z, lds);
}

// ---------------------------------------------------------------------------
// Many rows a request: keys and values decoded once per workgroup
// ---------------------------------------------------------------------------
// How a value row of D channels is dealt to the 32 rows of a 32 x 32 tile.
template <int D> struct Deal32 {
  static constexpr int kA = D >= 256 ? 8 : D >= 128 ? 4 : 2;
  static constexpr int kB = D / 32 - kA;         // 0, 1 or 2
};

template <int DT>
__device__ __forceinline__ v16f_t mfma32(u32x4_t a, u32x4_t b, v16f_t acc) {
  if constexpr (DT == IN_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), acc, 0, 0, 0);
}

// A workgroup of NW waves takes 32 NW rows; a wave takes 32 of them and all keys.
// Of every tile of 64 keys, the waves decode the four groups of 16 (of eight waves,
// four the keys and four the values) and write them to LDS as whole operand
// fragments (64 lanes x 16 bytes), so that every product afterwards is one
// contiguous 16-byte LDS read per lane and a matrix instruction.  Two tiles are kept:
// the next one's codes are in flight or being decoded while this one is computed, one
// barrier a tile.
//   - S^T = K Q^T and O^T = V^T P^T in 32 x 32 x 16 steps.  S^T leaves lane (q =
//     lane % 32, h = lane / 32) with rows 8 i + 4 h + (0 .. 3); a key whose place in its 16
//     has bits b3 b2 b1 b0 is put into row b2 b3 b1 b0, so that the lane's 8 rows of a
//     16-key step are keys 8 h .. 8 h + 7, the ones it feeds as P^T.
//   - fragments are 1040 bytes apart: lanes that write 8 fragments of one key then
//     meet 8 different groups of banks.
// Bound by vector work beside the matrix unit: a tile of 256 rows x 64 keys x 128 channels
// has 2048 clocks of matrix instructions and about as many of vector instructions on every
// SIMD, which overlap little: each kind is busy 46 to 48% of 4200 clocks.  Measured: 2048 tokens
// over 32768 keys (32 and 8 heads of 128 channels) in 964 to 1031 us on different cards, 1.03 to
// 1.10 PFLOP/s; each wave reading the pages by itself took 2783 us.  With 256 channels one wave a
// SIMD has nothing to overlap with: matrix unit 21%, vector unit 34% (600 tokens over 8192 keys, 294 to 301 us).
template <int D, int NW> struct TileLds {
  static constexpr int kFrag = 1040;
  union {
    struct {
      alignas(16) uint8_t k[2][D / 8 * kFrag], v[2][D / 8 * kFrag];
      int odd_tile[2][4];
    };
    float out[NW][32][D + 4];
  };
};

template <int DT, int D, int NW>
__device__ __forceinline__ void tile_rows(const AttnArgs& g, int req, int rt, int split, TileLds<D, NW>& lds) {
  using L = Deal32<D>;
  using T = uint16_t;
  constexpr int kSteps = D / 16;                 // K steps of S^T
  constexpr int kTiles = D / 32;                 // 32-channel tiles of O^T
  constexpr int kFrag = TileLds<D, NW>::kFrag;
  constexpr int kRows = 32 * NW;
  constexpr int kAheadK = 4;                     // fragments of keys read ahead
  constexpr int kKLoads = (D + 63) / 64;         // 16-byte loads of a lane for 16 keys
  auto& odd_tile = lds.odd_tile;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave & 3;                     // row group of a tile that this wave decodes
  const bool decodes_k = NW == 4 || wave < 4, decodes_v = NW == 4 || wave >= 4;
  const int r = lane & 31, h = lane >> 5;

  const int hk = blockIdx.x, G = g.group;
  const int64_t t0 = min(max(int64_t(g.cu[req]), int64_t(0)), g.tokens);
  const int64_t t1 = min(max(int64_t(g.cu[req + 1]), t0), g.tokens);
  const int m = int(t1 - t0), kv = max(g.lens[req], 0);
  const int rows = int(min(int64_t(m) * G, int64_t(0x7FFFFFFF))), row0 = rt * kRows;
  if (m > g.max_q || kv > g.max_kv) {            // not what the grid was sized for
    if (rt == 0 && split == 0) refuse_request<DT, D>(g, t0, rows, hk);
    return;
  }
  const int i0 = row0 / G, i1 = (min(row0 + kRows, rows) - 1) / G;
  const int hi_all = max(kv - m + i1 + 1, 0);
  const int lo = g.window ? max(kv - m + i0 - g.window + 1, 0) : 0;
  const int64_t start64 = int64_t(lo & ~31) + int64_t(split) * g.tile_chunk;
  if (split > 0 && start64 >= hi_all) {
    empty_split(g, t0, row0, min(row0 + kRows, rows), hk, split);
    if (split == g.tile_splits - 1)
      for (int i = g.tile_splits; i < g.slots; ++i) empty_split(g, t0, row0, min(row0 + kRows, rows), hk, i);
    return;
  }
  const int start = int(start64), hi = int(min(int64_t(hi_all), start64 + g.tile_chunk));
  // keys in [all_from, all_to) are seen by every row of the workgroup
  const int all_from = g.window ? max(kv - m + i1 - g.window + 1, 0) : 0, all_to = min(hi, kv - m + i0 + 1);

  int last, first;
  int orow;
  u32x4_t qf[kSteps];
  int wlast_min, wfirst_max;
  {
    const int row = row0 + wave * 32 + r;
    const bool real = row < rows;
    const int rr = real ? row : rows - 1;
    const int i = rr / G, head = hk * G + (rr - i * G);
    orow = real ? int(t0 + i) * g.heads + head : -1;
    last = real ? kv - m + i : -1;
    first = g.window ? max(kv - m + i - g.window + 1, 0) : 0;
    wlast_min = real ? last : 0x7FFFFFFF;
    wfirst_max = real ? first : 0;
    const T* q = static_cast<const T*>(g.q) + (t0 + i) * g.q_ts + head * g.q_hs + 8 * h;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) qf[s] = *reinterpret_cast<const u32x4_t*>(q + 16 * s);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    wlast_min = min(wlast_min, __shfl_xor(wlast_min, off, 64));
    wfirst_max = max(wfirst_max, __shfl_xor(wfirst_max, off, 64));
  }
  wlast_min = __builtin_amdgcn_readfirstlane(wlast_min);
  wfirst_max = __builtin_amdgcn_readfirstlane(wfirst_max);

  v16f_t o[kTiles];
  float mref = kLowest, l = 0.0f;
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int v = 0; v < 16; ++v) o[t][v] = 0.0f;

  // ---- this wave's 16 keys or values of a tile
  constexpr int kWordsV = L::kA == 8 ? 2 : 1, kRuns = L::kB ? 2 : 1;
  uint32_t raw[4 * kKLoads], sc[kKLoads];                // keys
  uint32_t rawv[8 * (kWordsV + kRuns - 1)], scv[8 * kRuns];
  auto rv = [&](int j, int w) -> uint32_t& { return rawv[8 * w + j]; };          // word w of key j; w == kWordsV: second run
  auto rvs = [&](int j, int run) -> uint32_t& { return scv[8 * run + j]; };
  int pending = -1;                              // row group of what is loaded; negative: nothing to read
  int groups = -1;
  const int32_t* table = g.table + req * g.table_stride;
  auto load = [&](int tile0) {
    if (((tile0 - start) & 1023) == 0) {
      const int key = tile0 + lane * 16, col = page_column(g, key);
      groups = row_group(g, hk, key, col, page_entry(g, table, col), lo, hi);
    }
    pending = __builtin_amdgcn_readlane(groups, ((tile0 - start) & 1023) / 16 + part);
    // What is loaded must reach its registers with no copy behind it, which would wait for the load: no other
    // path writes them here, and a group that is not to be read loads group 0 (decode() puts it right)
    if (g.pages > 0) {
      const int grp = max(pending, 0);
      const uint8_t* k = g.kc + int64_t(grp) * 16 * D;
      const uint8_t* ks = g.ks + int64_t(grp) * 16 * (D / 32);
      if (decodes_k) {
#pragma unroll
        for (int u = 0; u < kKLoads; ++u) {
          const int c = lane + 64 * u;           // 16-byte chunk of the 16 rows
          if (D % 64 == 0 || c < D) {
            const uint4 w = *reinterpret_cast<const uint4*>(k + 16 * c);
            raw[4 * u] = w.x; raw[4 * u + 1] = w.y; raw[4 * u + 2] = w.z; raw[4 * u + 3] = w.w;
            sc[u] = ks[c / 2];                   // two chunks to a block of 32
          }
        }
      }
      if (decodes_v) {
      const uint8_t* v = g.vc + int64_t(grp) * 16 * D + 8 * h * D;
      const uint8_t* vs = g.vs + int64_t(grp) * 16 * (D / 32) + 8 * h * (D / 32);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t* a = v + j * D + L::kA * r;
        if constexpr (L::kA == 8) {
          const uint2 w = *reinterpret_cast<const uint2*>(a);
          rv(j, 0) = w.x; rv(j, 1) = w.y;
        } else if constexpr (L::kA == 4) {
          rv(j, 0) = *reinterpret_cast<const uint32_t*>(a);
        } else {
          rv(j, 0) = *reinterpret_cast<const uint16_t*>(a);
        }
        rvs(j, 0) = vs[j * (D / 32) + (L::kA * r) / 32];
        if constexpr (L::kB) {
          const uint8_t* e = v + j * D + 32 * L::kA + L::kB * r;
          if constexpr (L::kB == 2) rv(j, kWordsV) = *reinterpret_cast<const uint16_t*>(e);
          else rv(j, kWordsV) = *e;
          rvs(j, 1) = vs[j * (D / 32) + (32 * L::kA + L::kB * r) / 32];
        }
      }
      }
    }
  };
  auto decode = [&](int tile0, int buf) {
    uint8_t* base = lds.k[buf];
    if (__builtin_expect(pending < 0, 0)) {      // keys of a bad page are NaN, and so is what sees them
#pragma unroll
      for (int u = 0; u < 4 * kKLoads; ++u) raw[u] = 0x7F7F7F7Fu;
#pragma unroll
      for (int u = 0; u < kKLoads; ++u) sc[u] = 127;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int w = 0; w < kWordsV + kRuns - 1; ++w) rv(j, w) = 0;
#pragma unroll
        for (int w = 0; w < kRuns; ++w) rvs(j, w) = 127;
      }
    }
    if (decodes_k)
#pragma unroll
    for (int u = 0; u < kKLoads; ++u) {
      const int c = lane + 64 * u;
      const int key = c / kSteps, s = c % kSteps;
      const int row = ((key >> 2) & 1) * 8 + (key >> 3) * 4 + (key & 3) + 16 * (part & 1);
      const uint32_t scale = sc[u] << 23;
      uint8_t* dst = base + ((part >> 1) * kSteps + s) * kFrag + row * 16;
      if (D % 64 == 0 || c < D) {
        *reinterpret_cast<u32x4_t*>(dst) = u32x4_t{decode2<DT, false>(raw[4 * u + 0], scale), decode2<DT, true>(raw[4 * u + 0], scale),
                                                   decode2<DT, false>(raw[4 * u + 1], scale), decode2<DT, true>(raw[4 * u + 1], scale)};
        *reinterpret_cast<u32x4_t*>(dst + 512) = u32x4_t{decode2<DT, false>(raw[4 * u + 2], scale), decode2<DT, true>(raw[4 * u + 2], scale),
                                                         decode2<DT, false>(raw[4 * u + 3], scale), decode2<DT, true>(raw[4 * u + 3], scale)};
      }
    }
    if (!decodes_v) return;
    // values that no row sees may be anything; the weight 0 must not meet an infinity or a NaN there
    const int key0 = tile0 + 16 * part;
    uint32_t odd = 0;
    if (tile0 < all_from || tile0 + 64 > all_to) {
      const uint32_t from = uint32_t(lo - key0 - 8 * h), many = uint32_t(max(hi - lo, 0));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool keep = uint32_t(j) - from < many;
#pragma unroll
        for (int w = 0; w < kWordsV + kRuns - 1; ++w) {
          rv(j, w) = keep ? rv(j, w) : 0u;
          odd |= any_nan_code(rv(j, w));
        }
#pragma unroll
        for (int w = 0; w < kRuns; ++w) {
          rvs(j, w) = keep ? rvs(j, w) : 127u;
          odd |= rvs(j, w) >= kWideScale<DT> ? 1u : 0u;
        }
      }
    }
    const bool any = __ballot(odd != 0) != 0;
    if (lane == 0) odd_tile[buf][part] = any;
    uint8_t* vb = lds.v[buf] + part * kFrag + lane * 16;        // fragment (tile, step) at 4 tile + step
    auto pair = [&](int w, int run, auto hi_half, int tile, bool both) {
      constexpr bool HI = decltype(hi_half)::value;
      u32x4_t a, c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = decode2<DT, HI>(rv(2 * j, w), rvs(2 * j, run) << 23);
        const uint32_t y = decode2<DT, HI>(rv(2 * j + 1, w), rvs(2 * j + 1, run) << 23);
        a[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        c[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
      }
      *reinterpret_cast<u32x4_t*>(vb + 4 * tile * kFrag) = a;
      if (both) *reinterpret_cast<u32x4_t*>(vb + 4 * (tile + 1) * kFrag) = c;
    };
#pragma unroll
    for (int w = 0; w < kWordsV; ++w) {
      pair(w, 0, std::false_type{}, 4 * w, true);
      if constexpr (L::kA >= 4) pair(w, 0, std::true_type{}, 4 * w + 2, true);
    }
    if constexpr (L::kB) pair(kWordsV, 1, std::false_type{}, L::kA, L::kB == 2);
  };

  // A tile with infinite or NaN values that some rows of the workgroup see and others do not: the outputs of
  // those that do get them, and the tile is left without them.
  auto take_odd = [&](int tile0, int buf) {
    const uint32_t from = uint32_t(first - tile0 - 8 * h), many = uint32_t(max(min(last, hi - 1) - first + 1, 0));
#pragma nounroll
    for (int u = 0; u < 4; ++u) {
      u32x4_t see;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        see[j] = (uint32_t(16 * u + 2 * j) - from < many ? kOneBits<DT> : 0u) |
                 (uint32_t(16 * u + 2 * j + 1) - from < many ? kOneBits<DT> << 16 : 0u);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        u32x4_t x = *reinterpret_cast<const u32x4_t*>(lds.v[buf] + (4 * t + u) * kFrag + lane * 16);
        u32x4_t plus, minus;
        take_marks<DT>(x, plus, minus);
        v16f_t zero;
#pragma unroll
        for (int v = 0; v < 16; ++v) zero[v] = 0.0f;
        const v16f_t up = mfma32<DT>(plus, see, zero);
#pragma unroll
        for (int v = 0; v < 16; ++v) o[t][v] += infinity_of(up[v]);
        __builtin_amdgcn_sched_barrier(0);       // one product at a time: this path shall cost no registers
        const v16f_t down = mfma32<DT>(minus, see, zero);
#pragma unroll
        for (int v = 0; v < 16; ++v) o[t][v] -= infinity_of(down[v]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __syncthreads();
    for (int f = wave; f < 4 * kTiles; f += NW) {
      u32x4_t* at = reinterpret_cast<u32x4_t*>(lds.v[buf] + f * kFrag + lane * 16);
      u32x4_t x = *at, plus, minus;
      take_marks<DT>(x, plus, minus);
      *at = x;
    }
    __syncthreads();
  };

  u32x4_t p[4];                                  // weights of the tile last scored
  auto score = [&](int tile0, int buf) {
    const uint8_t* base = lds.k[buf] + lane * 16;
    // ---- S^T
    // kAheadK fragments are read ahead of the matrix unit; the two 32-key tiles take turns, so that no
    // product waits for the one before
    v16f_t s[2];
#pragma unroll
    for (int v = 0; v < 16; ++v) s[0][v] = s[1][v] = 0.0f;
    auto fragment = [&](int i) {
      return *reinterpret_cast<const u32x4_t*>(base + ((i & 1) * kSteps + (i >> 1)) * kFrag);
    };
    u32x4_t kf[kAheadK];
#pragma unroll
    for (int i = 0; i < kAheadK; ++i) kf[i] = fragment(i);
#pragma unroll
    for (int i = 0; i < 2 * kSteps; ++i) {
      s[i & 1] = mfma32<DT>(kf[i % kAheadK], qf[i >> 1], s[i & 1]);
      if (i + kAheadK < 2 * kSteps) kf[i % kAheadK] = fragment(i + kAheadK);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, kAheadK, 0);
#pragma unroll
    for (int i = 0; i < 2 * kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      if (i + kAheadK < 2 * kSteps) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    // ---- masks: value 8 i + j of s[kt] is key 32 kt + 16 i + 8 h + j of the tile
    const uint32_t from = uint32_t(first - tile0 - 8 * h), many = uint32_t(max(min(last, hi - 1) - first + 1, 0));
    const bool edge = tile0 + 63 > wlast_min || tile0 < wfirst_max || tile0 + 64 > hi;
    if (edge) {
#pragma unroll
      for (int v = 0; v < 32; ++v)
        s[v >> 4][v & 15] = uint32_t(16 * (v >> 3) + (v & 7)) - from < many ? s[v >> 4][v & 15] : -__builtin_inff();
    }
    // ---- reference exponent
    float top = s[0][0];
#pragma unroll
    for (int v = 1; v < 32; ++v) top = fmaxf(top, s[v >> 4][v & 15]);
    top *= g.c;
    if (__ballot(top > mref + (kLift<DT> + kSlack))) {
      const float next = fmaxf(mref, fmaxf(top, __shfl_xor(top, 32, 64)) - kLift<DT>);
      const float a = mref == next || mref == kLowest ? 1.0f : __builtin_amdgcn_exp2f(mref - next);
      mref = next;
      l *= a;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o[t] *= a;
    }
    // ---- weights, rounded to the type of q: off by up to 2^-9 (BF16), so that the error against 64 bits is
    // 0.0023 where the outputs' own rounding is 0.0017.  Both ways to 0.0017 cost the matrix unit's time here
    // (2048 tokens over 32768 keys, 974 us): a second term as for few rows 1377 us, F16 weights and values where
    // the scales allow 1026 us.  The sum of the weights is that of the unrounded ones, which the log-sum-exp
    // needs; roundings to even leave it unbiased.
    // Of the two waves of a SIMD, the one that has come this far goes first until its values
    // are added: it mixes matrix and vector instructions, the other has only matrix ones (2048 tokens over
    // 32768: 983 us without, 975 with; workgroups of four waves lose 1% by it)
    if constexpr (NW == 8) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u >> 1][8 * (u & 1) + j], g.c, -mref));
      l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      p[u] = u32x4_t{pack2<DT>(e[0], e[1]), pack2<DT>(e[2], e[3]), pack2<DT>(e[4], e[5]), pack2<DT>(e[6], e[7])};
    }
  };
  auto add_values = [&](int buf) {              // O^T
    const uint8_t* base = lds.v[buf] + lane * 16;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        o[t] = mfma32<DT>(*reinterpret_cast<const u32x4_t*>(base + (4 * t + u) * kFrag), p[u], o[t]);
  };

  if (start < hi) {
    load(start);
    decode(start, 0);
    if (start + 64 < hi) load(start + 64);
    __syncthreads();
    int buf = 0;
    for (int tile0 = start; tile0 < hi; tile0 += 64) {
      if (odd_tile[buf][0] | odd_tile[buf][1] | odd_tile[buf][2] | odd_tile[buf][3]) take_odd(tile0, buf);
      if (tile0 + 64 < hi) {
        decode(tile0 + 64, buf ^ 1);
        if (tile0 + 128 < hi) load(tile0 + 128);
      }
      score(tile0, buf);
      add_values(buf);
      if constexpr (NW == 8) __builtin_amdgcn_s_setprio(0);
      __syncthreads();
      buf ^= 1;
    }
  }

  // ---- outputs.  The lane holds channels kA c + t of the first run (c = 8 (v / 4) + 4 h + v % 4), likewise
  // of the second, of one row; through LDS, whole rows are stored at a time.
  l += __shfl_xor(l, 32, 64);
  const bool direct = g.tile_splits == 1;
  const float scale = direct ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
  if (h == 0 && orow >= 0) put_stats<DT>(g, orow, split, g.tile_splits, mref, l);
  __syncthreads();                               // the tiles are done with
  auto put = [&](int base, int tile0, auto kWidth) {
    constexpr int W = decltype(kWidth)::value;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      float* dst = &lds.out[wave][r][base + W * (8 * (v >> 2) + 4 * h + (v & 3))];
      if constexpr (W >= 4) {
#pragma unroll
        for (int t = 0; t < W; t += 4)
          *reinterpret_cast<v4f*>(dst + t) = v4f{o[tile0 + t][v], o[tile0 + t + 1][v], o[tile0 + t + 2][v],
                                                 o[tile0 + t + 3][v]} * scale;
      } else {
#pragma unroll
        for (int t = 0; t < W; ++t) dst[t] = o[tile0 + t][v] * scale;
      }
    }
  };
  put(0, 0, std::integral_constant<int, L::kA>{});
  if constexpr (L::kB) put(32 * L::kA, L::kA, std::integral_constant<int, L::kB>{});
  wave_lds_fence();
#pragma unroll 4
  for (int i = lane; i < 32 * (D / 4); i += 64) {
    const int row = i / (D / 4), d = i % (D / 4) * 4;
    const int64_t to = __shfl(orow, row, 64);
    if (to < 0) continue;
    const v4f x = *reinterpret_cast<const v4f*>(&lds.out[wave][row][d]);
    if (direct)
      *reinterpret_cast<u32x2_t*>(static_cast<T*>(g.out) + to * D + d) = u32x2_t{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])};
    else
      *reinterpret_cast<v4f*>(g.part + (to * g.slots + split) * D + d) = x;
  }
}

// Requests of many rows, and in the same launch, behind them, the others of the call: y counts row
// tiles times splits, then requests of few rows times splits.
template <int DT, int D, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(D > 128 ? 1 : 2, D > 128 ? 1 : 2))) void attention_tile_kernel(const AttnArgs g) {
  __shared__ union { TileLds<D, NW> tile; FewLds<D, 2, NW> few; } lds;
  const int G = g.group;
  int unit = blockIdx.z * gridDim.y + blockIdx.y;
  if (unit < g.tile_units * g.tile_splits) {
    const int split = unit % g.tile_splits;
    unit /= g.tile_splits;
    const int req = find_request(g, unit, [&](int m) {
      const int64_t rows = int64_t(m) * G;
      return rows > kFewRows ? int((rows + 32 * NW - 1) / (32 * NW)) : 0;
    });
    if (req >= 0) tile_rows<DT, D, NW>(g, req, unit, split, lds.tile);
  } else {
    unit -= g.tile_units * g.tile_splits;
    const int split = unit % g.few_splits;
    unit /= g.few_splits;
    const int req = find_request(g, unit, [&](int m) { return m > 0 && int64_t(m) * G <= kFewRows ? 1 : 0; });
    if (req >= 0) few_rows<DT, D, 2, NW>(g, req, split, lds.few);
  }
}

// Joins the splits of one row: o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// WPR waves per row take every WPR-th split; a lane takes channels 2 lane, 2 lane + 1 of
// each 128.  Outputs of splits without keys were never written and are not read.  Bound by
// latency where rows are few (3.5 us), by memory where they are many.
template <int DT, int D, int WPR>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttnArgs g, int64_t requests) {
  constexpr int kPer = (D + 127) / 128;
  __shared__ v2f part[4][kPer][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = wave % WPR;
  const int64_t row = int64_t(blockIdx.x) * (4 / WPR) + wave / WPR;
  const int64_t token = row / g.heads;
  const bool mine = row < g.tokens * g.heads && token >= g.cu[0] && token < g.cu[requests] &&
                    !(g.part_ml[row * g.slots * 2 + 1] < 0.0f);
  if (WPR == 1 && !mine) return;
  v2f acc[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) acc[u] = v2f{0, 0};
  float top = kLowest, sum = 0.0f;
  if (mine) {
    const float* ml = g.part_ml + row * g.slots * 2;
    for (int i = lane; i < g.slots; i += 64)
      if (ml[2 * i + 1] != 0.0f) top = fmaxf(top, ml[2 * i]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    for (int i0 = 0; i0 < g.slots; i0 += 64) {
      // lane i holds the weight of split i0 + i
      float w = 0.0f, li = 0.0f;
      bool held = false;
      if (i0 + lane < g.slots) {
        li = ml[2 * (i0 + lane) + 1];
        const float mi = ml[2 * (i0 + lane)];
        held = li != 0.0f;
        w = li == 0.0f ? 0.0f : mi == top ? 1.0f : __builtin_amdgcn_exp2f(mi - top);
        li = li == 0.0f ? 0.0f : w * li;
      }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) li += __shfl_xor(li, off, 64);
      sum += li;
      const float* o = g.part + (row * g.slots + i0) * D;
      uint64_t left = __ballot(held);            // a weight that has vanished still brings a NaN of its slot
      for (int i = 0; i < sub; ++i) left &= left - 1;
      while (left) {
        // up to four slots, loads first
        float wi[4];
        float2 x[4][kPer];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = left ? __builtin_ctzll(left) : 0;
          wi[k] = left ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), i)) : 0.0f;
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int d = u * 128 + 2 * lane;
            x[k][u] = make_float2(0.0f, 0.0f);
            if (left && d < D) x[k][u] = *reinterpret_cast<const float2*>(o + i * D + d);
          }
#pragma unroll
          for (int j = 0; j < WPR; ++j) left &= left - 1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            acc[u][0] += wi[k] * x[k][u].x;
            acc[u][1] += wi[k] * x[k][u].y;
          }
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) part[wave][u][lane] = acc[u];
    __syncthreads();
    if (sub != 0 || !mine) return;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
#pragma unroll
      for (int w = 1; w < WPR; ++w) acc[u] += part[wave + w][u][lane];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int d = u * 128 + 2 * lane;
    if (d < D)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(g.out) + row * D + d) = pack2<DT>(acc[u][0] * inv, acc[u][1] * inv);
  }
  if (g.lse && lane == 0) g.lse[row] = log_sum(top, sum);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct Plan {
  int nq, waves;                // 16-row tiles and waves of attention_few_kernel
  bool tiles;                   // some request may have more than kFewRows rows
  int tile_waves;               // of attention_tile_kernel: 32 rows each
  int64_t tile_units;           // most row tiles that requests of many rows can have
  int64_t few_splits, few_chunk, tile_splits, tile_chunk, slots;
  int64_t window;               // 0: none, or none that a request of max_kv tokens would notice
  int64_t bytes;                // workspace
};

constexpr int64_t cut(int64_t keys, int64_t splits, int64_t least) {   // keys of a split
  return (std::max((keys + splits - 1) / splits, least) + 127) / 128 * 128;
}

mx_status_t plan_attention(int64_t tokens, int heads, int kv_heads, int dim, int64_t requests, int64_t max_q,
                           int64_t max_kv, int64_t window, Plan& p) {
  const int64_t lim = int64_t(1) << 30;
  if (tokens < 0 || requests < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || heads > 65536) return MX_ERR_SHAPE;
  if (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256) return MX_ERR_SHAPE;
  if (max_q < 0 || max_kv < 0 || window < 0) return MX_ERR_ARG;
  if (tokens > lim || requests > 65535 || max_kv > lim || max_q > lim || tokens * heads > 0x7FFFFFFF) return MX_ERR_SHAPE;
  const int64_t cus = device_cus();
  if (cus <= 0) return MX_ERR_LAUNCH;
  // from here on below 2^30, so that sums with it do not overflow
  p.window = window >= max_kv ? 0 : window;
  const int64_t group = heads / kv_heads, reqs = std::max<int64_t>(requests, 1), base = reqs * kv_heads;
  max_q = std::min(max_q, tokens);
  const int64_t rows = std::max<int64_t>(max_q * group, 1);
  p.tiles = rows > kFewRows;
  p.nq = rows <= 16 ? 1 : 2;
  // keys that the rows of one workgroup can see
  auto seen = [&](int64_t n) {
    const int64_t keys = p.window > 0 ? std::min(max_kv, p.window + n / group + 33) : max_kv;
    return std::max<int64_t>((keys + 63) / 64 * 64, 64);
  };
  // Requests of few rows: workgroups of eight waves, one for every CU (measured against two and
  // more: 191 to 193 us for 4 requests of 131072 keys against 195 to 215; uneven lengths of 64
  // requests even out by themselves, 136 us), none with less than 512 keys, two steps a wave.  Calls
  // that would leave most of the CUs idle even at 256 keys take workgroups of four waves with 256
  // keys: code that is new to an instruction cache is fetched by fewer waves at a time (1 request
  // of 1021 keys: 9.6 us, with eight waves 11.3 to 12.4).
  int64_t keys = seen(kFewRows);
  p.waves = !p.tiles && base * ((keys + 255) / 256) <= cus / 4 ? 4 : 8;
  // Beside requests of many rows, of which there are (tokens - requests) / (max_q - 1) if all others have
  // one token: at most 8 splits, since every row of the call has room for as many partial results.
  int64_t many = 0, few_wgs = base, most = keys;
  if (p.tiles) {
    many = std::max<int64_t>(1, std::min(reqs, (tokens - reqs + max_q - 2) / std::max<int64_t>(max_q - 1, 1)));
    few_wgs = (reqs - many) * kv_heads;
    most = few_wgs ? 8 : 1;
  }
  p.few_chunk = p.waves == 4 ? 256 : cut(keys, std::min(most, (cus + few_wgs - 1) / std::max<int64_t>(few_wgs, 1)), 512);
  p.few_splits = (keys + p.few_chunk - 1) / p.few_chunk;
  // Requests of many rows.  Workgroups of eight waves (one fits a CU) where they fill the CUs: a tile of
  // keys is decoded for twice the rows (2048 tokens over 32768: 4% less time).  Fewer
  // are spread better by workgroups of four waves, of which two fit a CU up to 128 channels (300 tokens
  // alone: 14.8 us, with eight waves 17.9).
  // Then the number of splits with the least estimate of rounds over the CUs plus partial results: a tile of
  // 64 keys takes 1.5 us (3 to 4 us with 192 or 256 channels, where one wave a SIMD has nothing to
  // overlap with), a workgroup's beginning and end 7 us, a partial result of 256 rows of 128 channels 0.05 us
  // of the memory's time, a join 5 us.
  p.tile_units = 0;
  p.tile_splits = 1;
  p.tile_chunk = 64;
  p.tile_waves = 4;
  if (p.tiles) {
    if (dim <= 128 && many * ((rows + 255) / 256) * kv_heads >= cus) p.tile_waves = 8;
    const int64_t tile_rows = 32 * p.tile_waves, room = p.tile_waves == 4 && dim <= 128 ? 2 * cus : cus;
    p.tile_units = tokens * group / tile_rows + std::min(reqs, tokens * group / (kFewRows + 1));
    keys = seen(tile_rows);
    const int64_t wgs = many * ((rows + tile_rows - 1) / tile_rows) * kv_heads;
    const double tile = dim > 128 ? dim / 64.0 : 1.5 * dim / 128.0, part = 0.05 * double(tile_rows) / 256.0 * dim / 128.0;
    double least = 0.0;
    for (int64_t n = 1; n <= 16; ++n) {
      const int64_t chunk = cut(keys, n, 256);
      if (n > 1 && (keys + chunk - 1) / chunk < n) break;
      const double cost = double((wgs * n + room - 1) / room) * (double((chunk + 63) / 64) * tile + 7.0) +
                          (n > 1 ? double(wgs * n) * part + 5.0 : 0.0);
      if (n == 1 || cost < least) {
        least = cost;
        p.tile_splits = n;
        p.tile_chunk = chunk;
      }
    }
  }
  p.slots = std::max(p.few_splits, p.tile_splits);
  p.bytes = p.slots > 1 ? tokens * heads * p.slots * (dim + 2) * 4 : 0;
  if (p.few_splits > 65535 || p.tile_units * p.tile_splits + reqs * p.few_splits > (1 << 24)) return MX_ERR_SHAPE;
  return MX_OK;
}

template <int DT, int D>
void launch_attention(const Plan& p, AttnArgs g, int64_t requests, hipStream_t stream) {
  const dim3 grid(unsigned(g.kv_heads), unsigned(requests), unsigned(p.few_splits));
  if (p.tiles) {
    const unsigned units = unsigned(p.tile_units * p.tile_splits + requests * p.few_splits), y = std::min(units, 32768u);
    const dim3 work(unsigned(g.kv_heads), y, (units + y - 1) / y);
    if constexpr (D <= 128) {
      if (p.tile_waves == 8) attention_tile_kernel<DT, D, 8><<<work, 512, 0, stream>>>(g);
    }
    if (p.tile_waves == 4) attention_tile_kernel<DT, D, 4><<<work, 256, 0, stream>>>(g);
  } else if (p.nq == 1) {
    if (p.waves == 4) attention_few_kernel<DT, D, 1, 4><<<grid, 256, 0, stream>>>(g);
    else attention_few_kernel<DT, D, 1, 8><<<grid, 512, 0, stream>>>(g);
  } else {
    constexpr int NW = D > 128 ? 4 : 8;
    attention_few_kernel<DT, D, 2, NW><<<grid, 64 * NW, 0, stream>>>(g);
  }
  const int64_t rows = g.tokens * g.heads;
  if (p.slots >= 8 && !p.tiles) attention_join_kernel<DT, D, 4><<<unsigned(rows), 256, 0, stream>>>(g, requests);
  else if (p.slots > 1) attention_join_kernel<DT, D, 1><<<unsigned((rows + 3) / 4), 256, 0, stream>>>(g, requests);
}

}  // namespace mxk

using namespace mxk;

extern "C" mx_status_t mx_paged_attention_workspace(int64_t tokens, int heads, int kv_heads, int dim, int64_t requests,
                                                    int64_t max_q, int64_t max_kv, int64_t window, int64_t* bytes) {
  if (!bytes) return MX_ERR_NULL;
  Plan p;
  const mx_status_t st = plan_attention(tokens, heads, kv_heads, dim, requests, max_q, max_kv, window, p);
  if (st == MX_OK) *bytes = p.bytes;
  return st;
}

extern "C" mx_status_t mx_paged_attention(const void* q, mx_dtype_t dtype, int64_t tokens, int heads,
                                          int64_t q_token_stride, int64_t q_head_stride, const mx_kv_cache_t* cache,
                                          const int32_t* page_table, int64_t table_stride, int64_t table_cols,
                                          const int32_t* cu, const int32_t* lens, int64_t requests, int64_t max_q,
                                          int64_t max_kv, int64_t window, float scale, void* out, float* lse,
                                          void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (!cache) return MX_ERR_NULL;
  if (dtype != MX_BF16 && dtype != MX_F16) return MX_ERR_UNSUPPORTED;
  mx_status_t st = check_kv_cache(*cache);
  if (st != MX_OK) return st;
  if (tokens < 0 || requests < 0 || heads < 1 || heads > 65536 || heads % cache->kv_heads) return MX_ERR_SHAPE;
  if (table_cols < 0 || table_stride < 0) return MX_ERR_SHAPE;
  if (max_q < 0 || max_kv < 0 || window < 0 || !(scale > 0.0f) || !std::isfinite(scale)) return MX_ERR_ARG;
  if (tokens == 0 || requests == 0) return MX_OK;
  if (!q || !cu || !lens || !out || (table_cols > 0 && !page_table)) return MX_ERR_NULL;
  if (cache->pages > 0 && (!cache->k || !cache->k_scales || !cache->v || !cache->v_scales)) return MX_ERR_NULL;
  if (misaligned(q) || misaligned(out) || misaligned(cache->k) || misaligned(cache->v) ||
      misaligned(cache->k_scales) || misaligned(cache->v_scales) || misaligned(workspace) ||
      (q_token_stride | q_head_stride) % 8)
    return MX_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(lens) |
       reinterpret_cast<uintptr_t>(lse)) & 3u)
    return MX_ERR_ALIGN;
  Plan p;
  st = plan_attention(tokens, heads, cache->kv_heads, cache->dim, requests, max_q, max_kv, window, p);
  if (st != MX_OK) return st;
  if (p.bytes > 0 && !workspace) return MX_ERR_NULL;
  if (workspace_bytes < p.bytes) return MX_ERR_SHAPE;
  AttnArgs g = {};
  g.q = q; g.q_ts = q_token_stride; g.q_hs = q_head_stride;
  g.kc = cache->k; g.ks = cache->k_scales; g.vc = cache->v; g.vs = cache->v_scales;
  g.pages = cache->pages;
  g.table = page_table; g.table_stride = table_stride; g.table_cols = table_cols;
  g.cu = cu; g.lens = lens; g.out = out; g.lse = lse;
  g.part = static_cast<float*>(workspace);
  g.part_ml = g.part ? g.part + tokens * heads * p.slots * cache->dim : nullptr;
  g.tokens = tokens; g.max_q = max_q; g.max_kv = max_kv;
  g.heads = heads; g.kv_heads = cache->kv_heads; g.group = heads / cache->kv_heads; g.page = cache->page;
  g.window = int(p.window);
  g.requests = int(requests); g.tile_units = int(p.tile_units); g.slots = int(p.slots);
  g.few_splits = int(p.few_splits); g.few_chunk = int(p.few_chunk);
  g.tile_splits = int(p.tile_splits); g.tile_chunk = int(p.tile_chunk);
  g.inv_group = 1.0f / float(g.group);
  g.inv_page16 = 16.0 / g.page;
  g.c = scale * 1.44269504088896340736f;
  auto run = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    switch (cache->dim) {
      case 64: launch_attention<DT, 64>(p, g, requests, stream); break;
      case 96: launch_attention<DT, 96>(p, g, requests, stream); break;
      case 128: launch_attention<DT, 128>(p, g, requests, stream); break;
      case 192: launch_attention<DT, 192>(p, g, requests, stream); break;
      default: launch_attention<DT, 256>(p, g, requests, stream); break;
    }
  };
  if (dtype == MX_BF16) run(std::integral_constant<int, IN_BF16>{});
  else run(std::integral_constant<int, IN_F16>{});
  return hipGetLastError() == hipSuccess ? MX_OK : MX_ERR_LAUNCH;
}
