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

// Requests of up to so many rows (tokens x group) go to attention_kernel, whose waves split the keys.
constexpr int kFewRows = 32;

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
  float* part;                  // [tokens * heads][splits][dim] unnormalised outputs
  float* part_ml;               // [tokens * heads][splits][2] reference exponent and sum
  int64_t tokens, max_q, max_kv;
  int heads, kv_heads, group, page;
  int window;                   // 0: none
  int row_tiles, splits, chunk; // keys of a split, a multiple of 32
  float c;                      // scale * log2(e)
  bool few_only;                // requests of more than kFewRows rows are left to attention_tile_kernel
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

// How a value row of D channels is dealt to the 16 lanes of a row of the matrix
// unit: kA contiguous channels each of the first 16 kA, then kB each of the rest,
// powers of two, so that a lane's run lies in one block of 32.
template <int D> struct Deal {
  static constexpr int kA = D >= 256 ? 16 : D >= 128 ? 8 : 4;
  static constexpr int kB = D / 16 - kA;
  static constexpr int kWordsA = kA / 4, kWordsB = kB ? 1 : 0, kWords = kWordsA + kWordsB;
  static constexpr int kScales = kB ? 2 : 1;
};

__device__ __forceinline__ uint32_t any_nan_code(uint32_t w) {   // nonzero if a byte is an E4M3 NaN
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Row group (16 rows of one page and head) of keys key .. key + 15: -1 where no row sees them (not
// read), -2 where the page number or its place is out of range.
__device__ __forceinline__ int row_group(const AttnArgs& g, const int32_t* __restrict__ table, int hk, int key, int lo,
                                         int hi) {
  if (key >= hi || key + 16 <= lo) return -1;
  const int col = key / g.page;
  if (col >= g.table_cols) return -2;
  const int32_t p = table[col];
  if (p < 0 || p >= g.pages) return -2;
  return int((int64_t(p) * g.kv_heads + hk) * (g.page / 16) + (key - col * g.page) / 16);
}

// NaN for all rows of one kv head of a request that exceeds what the caller announced.
template <int DT, int D>
__device__ __forceinline__ void refuse_request(const AttnArgs& g, int64_t t0, int64_t rows, int hk, int rt, int split) {
  if (rt != 0) return;
  const float nan = __uint_as_float(0x7FC00000u);
  for (int64_t i = threadIdx.x; i < rows; i += blockDim.x) {
    const int64_t row = (t0 + i / g.group) * g.heads + hk * g.group + i % g.group;
    if (g.splits > 1) {
      g.part_ml[(row * g.splits + split) * 2] = split ? kLowest : 0.0f;
      g.part_ml[(row * g.splits + split) * 2 + 1] = split ? 0.0f : nan;
    } else {
      for (int d = 0; d < D; ++d) static_cast<uint16_t*>(g.out)[row * D + d] = DT == IN_BF16 ? 0x7FC0u : 0x7E00u;
      if (g.lse) g.lse[row] = nan;
    }
  }
}

// A split without keys adds nothing to rows [row0, row1).
__device__ __forceinline__ void empty_split(const AttnArgs& g, int64_t t0, int64_t row0, int64_t row1, int hk, int split) {
  for (int64_t i = row0 + threadIdx.x; i < row1; i += blockDim.x) {
    const int64_t row = (t0 + i / g.group) * g.heads + hk * g.group + i % g.group;
    g.part_ml[(row * g.splits + split) * 2] = kLowest;
    g.part_ml[(row * g.splits + split) * 2 + 1] = 0.0f;
  }
}

// Log-sum-exp of reference exponent m and sum l.
__device__ __forceinline__ float log_sum(float m, float l) {
  const float inf = __builtin_inff();
  return l == 0.0f ? -inf : m == inf ? inf : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

template <int DT>
__device__ __forceinline__ void put_stats(const AttnArgs& g, int64_t row, int split, float m, float l) {
  if (g.splits > 1) {
    g.part_ml[(row * g.splits + split) * 2] = m;
    g.part_ml[(row * g.splits + split) * 2 + 1] = l;
  } else if (g.lse) {
    g.lse[row] = log_sum(m, l);
  }
}

template <int DT, int D, int NQ, int NW>
__global__ __launch_bounds__(64 * NW) void attention_kernel(const AttnArgs g) {
  using L = Deal<D>;
  constexpr int kFrags = D / 32;                 // K steps of S^T
  constexpr int kTiles = D / 16;                 // 16-channel tiles of O^T
  constexpr int kKS = (D + 63) / 64;             // scale bytes of a key a lane needs
  constexpr int kRows = NQ * 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, quarter = lane >> 4;

  // the kv head runs fastest over the grid: neighbouring workgroups go to different
  // XCDs, so with 8 kv heads each XCD's L2 serves one head's pages
  int64_t b = blockIdx.x;
  const int hk = int(b % g.kv_heads); b /= g.kv_heads;
  const int split = int(b % g.splits); b /= g.splits;
  const int rt = int(b % g.row_tiles);
  const int64_t req = b / g.row_tiles;
  const int G = g.group;

  const int64_t t0 = min(max(int64_t(g.cu[req]), int64_t(0)), g.tokens);
  const int64_t t1 = min(max(int64_t(g.cu[req + 1]), t0), g.tokens);
  const int m = int(t1 - t0), kv = max(g.lens[req], 0);
  const int64_t rows = int64_t(m) * G, row0 = int64_t(rt) * kRows;
  using T = uint16_t;
  if (g.few_only && rows > kFewRows) return;     // attention_tile_kernel's
  if (m > g.max_q || kv > g.max_kv) {            // not what the grid was sized for
    refuse_request<DT, D>(g, t0, rows, hk, rt, split);
    return;
  }
  if (row0 >= rows) return;
  // keys that some row of this tile sees
  const int i0 = int(row0 / G), i1 = int((min(row0 + kRows, rows) - 1) / G);
  const int hi_all = max(kv - m + i1 + 1, 0);
  const int lo = g.window ? max(kv - m + i0 - g.window + 1, 0) : 0;
  const int64_t start64 = int64_t(lo & ~31) + int64_t(split) * g.chunk;
  if (split > 0 && start64 >= hi_all) {
    empty_split(g, t0, row0, min(row0 + kRows, rows), hk, split);
    return;
  }
  const int start = int(start64), hi = int(min(int64_t(hi_all), start64 + g.chunk));

  // this lane's rows: where q is, and the keys (first, last] a row sees
  int last[NQ], first[NQ];
  int64_t orow[NQ];
  u32x4_t qf[NQ][kFrags];
  int wlast_min = 0x7FFFFFFF, wfirst_max = 0;    // what every row of the wave sees
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t row = row0 + n * 16 + r;
    const bool real = row < rows;
    const int64_t rr = real ? row : rows - 1;
    const int i = int(rr / G);
    const int64_t head = int64_t(hk) * G + (rr - int64_t(i) * G);
    orow[n] = real ? (t0 + i) * g.heads + head : -1;
    last[n] = real ? kv - m + i : -1;
    first[n] = g.window ? max(kv - m + i - g.window + 1, 0) : 0;
    if (real) { wlast_min = min(wlast_min, last[n]); wfirst_max = max(wfirst_max, first[n]); }
    const T* q = static_cast<const T*>(g.q) + (t0 + i) * g.q_ts + head * g.q_hs;
#pragma unroll
    for (int s = 0; s < kFrags; ++s) {
      const int d = s / 2 * 64 + (s / 2 * 2 + 1 < kFrags ? 16 * quarter + 8 * (s & 1) : 8 * quarter);
      qf[n][s] = *reinterpret_cast<const u32x4_t*>(q + d);
    }
  }
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) {
    wlast_min = min(wlast_min, __shfl_xor(wlast_min, off, 64));
    wfirst_max = max(wfirst_max, __shfl_xor(wfirst_max, off, 64));
  }

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
    uint32_t k[2][kFrags * 2], ks[2][kKS];
    uint32_t v[8][L::kWords], vs[8][L::kScales];
  } raw;
  // row group of keys 16 i .. 16 i + 15 of the current window of 1024 keys, held by lane i
  int groups = -1;
  const int32_t* table = g.table + req * g.table_stride;
  auto load = [&](int step) {      // step: 32-key step within the window
    const int ga = __builtin_amdgcn_readlane(groups, 2 * step), gb = __builtin_amdgcn_readlane(groups, 2 * step + 1);
    if ((ga & gb) >= 0) {          // a group that is not read borrows the other's addresses
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
          raw.ks[t][u] = s[2 * u + (quarter >> 1)];
        }
        if constexpr (D % 64) {
          const uint2 w = *reinterpret_cast<const uint2*>(k + D / 64 * 64 + 8 * quarter);
          raw.k[t][kFrags * 2 - 2] = w.x; raw.k[t][kFrags * 2 - 1] = w.y;
          raw.ks[t][kKS - 1] = s[D / 32 - 1];
        }
      }
      const uint8_t* v = g.vc + vrow * D + L::kA * r;
      const uint8_t* s = g.vs + vrow * (D / 32) + (L::kA * r) / 32;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (L::kA == 4) {
          raw.v[j][0] = *reinterpret_cast<const uint32_t*>(v + j * D);
        } else if constexpr (L::kA == 8) {
          const uint2 w = *reinterpret_cast<const uint2*>(v + j * D);
          raw.v[j][0] = w.x; raw.v[j][1] = w.y;
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(v + j * D);
          raw.v[j][0] = w.x; raw.v[j][1] = w.y; raw.v[j][2] = w.z; raw.v[j][3] = w.w;
        }
        raw.vs[j][0] = s[j * (D / 32)];
        if constexpr (L::kB) {
          const uint8_t* e = g.vc + (vrow + j) * D + 16 * L::kA + L::kB * r;
          if constexpr (L::kB == 4) raw.v[j][L::kWordsA] = *reinterpret_cast<const uint32_t*>(e);
          else raw.v[j][L::kWordsA] = *reinterpret_cast<const uint16_t*>(e);
          raw.vs[j][1] = g.vs[(vrow + j) * (D / 32) + (16 * L::kA + L::kB * r) / 32];
        }
      }
    }
    if ((ga | gb) < 0) {           // keys of a bad page are NaN, and so is what sees them; values are masked below
      const int grp = (r & 8) ? gb : ga;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int u = 0; u < kFrags * 2; ++u) raw.k[t][u] = grp >= 0 ? raw.k[t][u] : 0x7F7F7F7Fu;
#pragma unroll
        for (int u = 0; u < kKS; ++u) raw.ks[t][u] = grp >= 0 ? raw.ks[t][u] : 127u;
      }
      const bool none = ((quarter & 2) ? gb : ga) < 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int w = 0; w < L::kWords; ++w) raw.v[j][w] = none ? 0u : raw.v[j][w];
#pragma unroll
        for (int w = 0; w < L::kScales; ++w) raw.vs[j][w] = none ? 127u : raw.vs[j][w];
      }
    }
  };

  auto compute = [&](int key0) {
    // ---- S^T
    v4f s[NQ][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      u32x4_t kf[kFrags];
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        const uint32_t sc = raw.ks[t][f / 2] << 23;
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
    // ---- masks: only a step that some row does not see whole needs them
    const bool edge = key0 + 31 > wlast_min || key0 < wfirst_max || key0 + 32 > hi;
    if (edge) {
      // key 8 quarter + j of the step is seen by row n iff unsigned(j - from) < many
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const uint32_t from = uint32_t(first[n] - key0 - 8 * quarter);
        const uint32_t many = uint32_t(max(min(last[n], hi - 1) - first[n] + 1, 0));
#pragma unroll
        for (int j = 0; j < 8; ++j) s[n][j >> 2][j & 3] = uint32_t(j) - from < many ? s[n][j >> 2][j & 3] : -__builtin_inff();
      }
      // values that no row sees may be anything; the weight 0 must not meet a NaN there
      const uint32_t from = uint32_t(lo - key0 - 8 * quarter), many = uint32_t(max(hi - lo, 0));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool keep = uint32_t(j) - from < many;
#pragma unroll
        for (int w = 0; w < L::kWords; ++w) raw.v[j][w] = keep ? raw.v[j][w] : 0u;
#pragma unroll
        for (int w = 0; w < L::kScales; ++w) raw.vs[j][w] = keep ? raw.vs[j][w] : 127u;
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
        const float a = mref[n] == next ? 1.0f : __builtin_amdgcn_exp2f(mref[n] - next);
        mref[n] = next;
        l[n] *= a;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[n][t] *= a;
      }
    }
    // ---- weights
    u32x4_t p[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][j >> 2][j & 3], g.c, -mref[n]));
      l[n] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      p[n] = u32x4_t{pack2<DT>(e[0], e[1]), pack2<DT>(e[2], e[3]), pack2<DT>(e[4], e[5]), pack2<DT>(e[6], e[7])};
    }
    // channels 2 c, 2 c + 1 of the lane's run, all 8 keys
    auto fragments = [&](int w, auto hi_half, u32x4_t& a, u32x4_t& c) {
      constexpr bool HI = decltype(hi_half)::value;
      const int sc = w >= L::kWordsA ? 1 : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = decode2<DT, HI>(raw.v[2 * j][w], raw.vs[2 * j][L::kScales > 1 ? sc : 0] << 23);
        const uint32_t y = decode2<DT, HI>(raw.v[2 * j + 1][w], raw.vs[2 * j + 1][L::kScales > 1 ? sc : 0] << 23);
        a[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        c[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
      }
    };
    auto for_tiles = [&](auto f) {   // f(tile, fragments) over pairs of tiles
#pragma unroll
      for (int w = 0; w < L::kWords; ++w) {
        u32x4_t a, c;
        fragments(w, std::false_type{}, a, c);
        f(4 * w, a); f(4 * w + 1, c);
        if (4 * w + 2 < kTiles) {
          fragments(w, std::true_type{}, a, c);
          f(4 * w + 2, a); f(4 * w + 3, c);
        }
      }
    };
    // A NaN value that some rows of the wave see and others do not: 0 * NaN would reach
    // them all.  Such values are taken out, and put into the outputs of the rows that
    // see them where a product of marks and visibility finds any.
    if (edge) {
      uint32_t nan = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int w = 0; w < L::kWords; ++w)
          nan |= any_nan_code(w >= L::kWordsA && L::kB == 2 ? raw.v[j][w] & 0xFFFFu : raw.v[j][w]);
#pragma unroll
        for (int w = 0; w < L::kScales; ++w) nan |= raw.vs[j][w] == 255u ? 1u : 0u;
      }
      if (__ballot(nan != 0)) {
        Raw keep = raw;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int w = 0; w < L::kWords; ++w) {
            const uint32_t bytes = any_nan_code(raw.v[j][w]) >> 7;      // 1 in every NaN byte
            const bool all = raw.vs[j][L::kScales > 1 && w >= L::kWordsA ? 1 : 0] == 255u;
            const uint32_t mark = all ? 0x01010101u : bytes;
            keep.v[j][w] = raw.v[j][w] & ~(mark * 255u);
            raw.v[j][w] = mark * 0x38u;                                 // E4M3 1.0
          }
#pragma unroll
          for (int w = 0; w < L::kScales; ++w) {
            keep.vs[j][w] = raw.vs[j][w] == 255u ? 127u : raw.vs[j][w];
            raw.vs[j][w] = 127u;
          }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            e[j] = uint32_t(j) - uint32_t(first[n] - key0 - 8 * quarter) < uint32_t(max(min(last[n], hi - 1) - first[n] + 1, 0))
                       ? 1.0f : 0.0f;
          const u32x4_t see = {pack2<DT>(e[0], e[1]), pack2<DT>(e[2], e[3]), pack2<DT>(e[4], e[5]), pack2<DT>(e[6], e[7])};
          for_tiles([&](int t, u32x4_t a) {
            const v4f hits = mfma16<DT>(a, see, v4f{0, 0, 0, 0});
#pragma unroll
            for (int v = 0; v < 4; ++v) {      // a count: all bits of `any` set where it is not zero
              const int any = -__float_as_int(hits[v]) >> 31;
              o[n][t][v] = __uint_as_float(__float_as_uint(o[n][t][v]) | (uint32_t(any) & 0x7FC00000u));
            }
          });
        }
        raw = keep;
      }
    }
    // ---- O^T
    for_tiles([&](int t, u32x4_t a) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) o[n][t] = mfma16<DT>(a, p[n], o[n][t]);
    });
  };

  for (int window0 = start; window0 < hi; window0 += 1024) {
    groups = row_group(g, table, hk, window0 + lane * 16, lo, hi);
    const int steps = (min(hi - window0, 1024) + 31) / 32;
    for (int step = wave; step < steps; step += NW) {
      load(step);
      compute(window0 + 32 * step);
    }
  }

  // ---- sums over the quarters of a row's keys
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
  }
  // ---- waves that split the keys: join them
  {
    __shared__ float sm[NW][NQ * 16], sl[NW][NQ * 16];
    __shared__ v4f so[NQ * kTiles][64];
    if (quarter == 0) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) { sm[wave][n * 16 + r] = mref[n]; sl[wave][n * 16 + r] = l[n]; }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = kLowest, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, sm[w][n * 16 + r]);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float lw = sl[w][n * 16 + r];
        if (lw != 0.0f) sum += lw * (sm[w][n * 16 + r] == top ? 1.0f : __builtin_amdgcn_exp2f(sm[w][n * 16 + r] - top));
      }
      const float a = mref[n] == top ? 1.0f : __builtin_amdgcn_exp2f(mref[n] - top);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o[n][t] *= a;
      mref[n] = top;
      l[n] = sum;
    }
    for (int w = 1; w < NW; ++w) {               // wave 0 adds the others in order
      if (wave == w) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int t = 0; t < kTiles; ++t) so[n * kTiles + t][lane] = o[n][t];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int t = 0; t < kTiles; ++t) o[n][t] += so[n * kTiles + t][lane];
      }
      __syncthreads();
    }
    if (wave != 0) return;
  }

  // ---- outputs: the lane holds channels kA (4 quarter + v) + t of the first run, likewise of the second
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (orow[n] < 0) continue;
    const bool direct = g.splits == 1;
    const float inv = direct ? (l[n] == 0.0f ? 0.0f : 1.0f / l[n]) : 1.0f;
    auto put = [&](int base, int width, int tile0, auto kWidth) {
      constexpr int W = decltype(kWidth)::value;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t d = base + W * (4 * quarter + v);
        if (direct) {
#pragma unroll
          for (int t = 0; t < W; t += 2)
            *reinterpret_cast<uint32_t*>(static_cast<T*>(g.out) + orow[n] * D + d + t) =
                pack2<DT>(o[n][tile0 + t][v] * inv, o[n][tile0 + t + 1][v] * inv);
        } else {
          float* dst = g.part + (orow[n] * g.splits + split) * D + d;
#pragma unroll
          for (int t = 0; t < W; t += 2)
            *reinterpret_cast<float2*>(dst + t) = make_float2(o[n][tile0 + t][v], o[n][tile0 + t + 1][v]);
        }
      }
    };
    put(0, L::kA, 0, std::integral_constant<int, L::kA>{});
    if constexpr (L::kB) put(16 * L::kA, L::kB, L::kA, std::integral_constant<int, L::kB>{});
    if (quarter == 0) put_stats<DT>(g, orow[n], split, mref[n], l[n]);
  }
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
template <int DT, int D, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void attention_tile_kernel(const AttnArgs g) {
  using L = Deal32<D>;
  using T = uint16_t;
  constexpr int kSteps = D / 16;                 // K steps of S^T
  constexpr int kTiles = D / 32;                 // 32-channel tiles of O^T
  constexpr int kFrag = 1040;
  constexpr int kFragsK = 2 * kSteps, kFrags = kFragsK + 4 * kTiles;
  constexpr int kRows = 32 * NW;
  constexpr int kKLoads = (D + 63) / 64;         // 16-byte loads of a lane for 16 keys
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][kFrags * kFrag];
  __shared__ int nan_tile[2][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave & 3;                     // row group of a tile that this wave decodes
  const bool decodes_k = NW == 4 || wave < 4, decodes_v = NW == 4 || wave >= 4;
  const int r = lane & 31, h = lane >> 5;

  int64_t b = blockIdx.x;
  const int hk = int(b % g.kv_heads); b /= g.kv_heads;
  const int split = int(b % g.splits); b /= g.splits;
  const int rt = int(b % g.row_tiles);
  const int64_t req = b / g.row_tiles;
  const int G = g.group;
  const int64_t t0 = min(max(int64_t(g.cu[req]), int64_t(0)), g.tokens);
  const int64_t t1 = min(max(int64_t(g.cu[req + 1]), t0), g.tokens);
  const int m = int(t1 - t0), kv = max(g.lens[req], 0);
  const int64_t rows = int64_t(m) * G, row0 = int64_t(rt) * kRows;
  if (rows <= kFewRows || row0 >= rows) return;  // requests of few rows are attention_kernel's
  if (m > g.max_q || kv > g.max_kv) {            // not what the grid was sized for
    refuse_request<DT, D>(g, t0, rows, hk, rt, split);
    return;
  }
  const int i0 = int(row0 / G), i1 = int((min(row0 + kRows, rows) - 1) / G);
  const int hi_all = max(kv - m + i1 + 1, 0);
  const int lo = g.window ? max(kv - m + i0 - g.window + 1, 0) : 0;
  const int64_t start64 = int64_t(lo & ~31) + int64_t(split) * g.chunk;
  if (split > 0 && start64 >= hi_all) {
    empty_split(g, t0, row0, min(row0 + kRows, rows), hk, split);
    return;
  }
  const int start = int(start64), hi = int(min(int64_t(hi_all), start64 + g.chunk));
  // keys in [all_from, all_to) are seen by every row of the workgroup
  const int all_from = g.window ? max(kv - m + i1 - g.window + 1, 0) : 0, all_to = min(hi, kv - m + i0 + 1);

  int last, first;
  int64_t orow;
  u32x4_t qf[kSteps];
  int wlast_min, wfirst_max;
  {
    const int64_t row = row0 + wave * 32 + r;
    const bool real = row < rows;
    const int64_t rr = real ? row : rows - 1;
    const int i = int(rr / G);
    const int64_t head = int64_t(hk) * G + (rr - int64_t(i) * G);
    orow = real ? (t0 + i) * g.heads + head : -1;
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
  uint4 rk[kKLoads];
  uint32_t rks[kKLoads];
  uint32_t rv[8][L::kA == 8 ? 2 : 1], rvb[8], rvs[8], rvsb[8];
  int groups = -1;
  const int32_t* table = g.table + req * g.table_stride;
  auto load = [&](int tile0) {
    if (((tile0 - start) & 1023) == 0) groups = row_group(g, table, hk, tile0 + lane * 16, lo, hi);
    const int grp = __builtin_amdgcn_readlane(groups, ((tile0 - start) & 1023) / 16 + part);
    if (grp >= 0) {
      const uint8_t* k = g.kc + int64_t(grp) * 16 * D;
      const uint8_t* ks = g.ks + int64_t(grp) * 16 * (D / 32);
      if (decodes_k) {
#pragma unroll
        for (int u = 0; u < kKLoads; ++u) {
          const int c = lane + 64 * u;           // 16-byte chunk of the 16 rows
          if (D % 64 == 0 || c < D) {
            rk[u] = *reinterpret_cast<const uint4*>(k + 16 * c);
            rks[u] = ks[c / 2];                  // two chunks to a block of 32
          }
        }
      }
      if (!decodes_v) return;
      const uint8_t* v = g.vc + int64_t(grp) * 16 * D + 8 * h * D;
      const uint8_t* vs = g.vs + int64_t(grp) * 16 * (D / 32) + 8 * h * (D / 32);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t* a = v + j * D + L::kA * r;
        if constexpr (L::kA == 8) {
          const uint2 w = *reinterpret_cast<const uint2*>(a);
          rv[j][0] = w.x; rv[j][1] = w.y;
        } else if constexpr (L::kA == 4) {
          rv[j][0] = *reinterpret_cast<const uint32_t*>(a);
        } else {
          rv[j][0] = *reinterpret_cast<const uint16_t*>(a);
        }
        rvs[j] = vs[j * (D / 32) + (L::kA * r) / 32];
        if constexpr (L::kB) {
          const uint8_t* e = v + j * D + 32 * L::kA + L::kB * r;
          if constexpr (L::kB == 2) rvb[j] = *reinterpret_cast<const uint16_t*>(e);
          else rvb[j] = *e;
          rvsb[j] = vs[j * (D / 32) + (32 * L::kA + L::kB * r) / 32];
        }
      }
    } else {                                     // keys of a bad page are NaN, and so is what sees them
#pragma unroll
      for (int u = 0; u < kKLoads; ++u) {
        rk[u] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        rks[u] = 127;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rv[j][0] = rvb[j] = 0;
        if constexpr (L::kA == 8) rv[j][1] = 0;
        rvs[j] = rvsb[j] = 127;
      }
    }
  };
  auto decode = [&](int tile0, int buf) {
    uint8_t* base = lds[buf];
    if (decodes_k)
#pragma unroll
    for (int u = 0; u < kKLoads; ++u) {
      const int c = lane + 64 * u;
      const int key = c / kSteps, s = c % kSteps;
      const int row = ((key >> 2) & 1) * 8 + (key >> 3) * 4 + (key & 3) + 16 * (part & 1);
      const uint32_t sc = rks[u] << 23;
      uint8_t* dst = base + ((part >> 1) * kSteps + s) * kFrag + row * 16;
      if (D % 64 == 0 || c < D) {
        *reinterpret_cast<u32x4_t*>(dst) = u32x4_t{decode2<DT, false>(rk[u].x, sc), decode2<DT, true>(rk[u].x, sc),
                                                   decode2<DT, false>(rk[u].y, sc), decode2<DT, true>(rk[u].y, sc)};
        *reinterpret_cast<u32x4_t*>(dst + 512) = u32x4_t{decode2<DT, false>(rk[u].z, sc), decode2<DT, true>(rk[u].z, sc),
                                                         decode2<DT, false>(rk[u].w, sc), decode2<DT, true>(rk[u].w, sc)};
      }
    }
    if (!decodes_v) return;
    // values that no row sees may be anything; the weight 0 must not meet a NaN there
    const int key0 = tile0 + 16 * part;
    uint32_t nan = 0;
    if (tile0 < all_from || tile0 + 64 > all_to) {
      const uint32_t from = uint32_t(lo - key0 - 8 * h), many = uint32_t(max(hi - lo, 0));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool keep = uint32_t(j) - from < many;
        rv[j][0] = keep ? rv[j][0] : 0u;
        if constexpr (L::kA == 8) rv[j][1] = keep ? rv[j][1] : 0u;
        rvs[j] = keep ? rvs[j] : 127u;
        nan |= any_nan_code(rv[j][0]) | (rvs[j] == 255u ? 1u : 0u);
        if constexpr (L::kA == 8) nan |= any_nan_code(rv[j][1]);
        if constexpr (L::kB) {
          rvb[j] = keep ? rvb[j] : 0u;
          rvsb[j] = keep ? rvsb[j] : 127u;
          nan |= any_nan_code(rvb[j]) | (rvsb[j] == 255u ? 1u : 0u);
        }
      }
    }
    const bool any = __ballot(nan != 0) != 0;
    if (lane == 0) nan_tile[buf][part] = any;
    uint8_t* vb = base + (kFragsK + part) * kFrag + lane * 16;   // fragment (tile, step) at kFragsK + 4 tile + step
    auto pair = [&](const uint32_t (&w)[8], const uint32_t (&sc)[8], auto hi_half, int tile, bool both) {
      constexpr bool HI = decltype(hi_half)::value;
      u32x4_t a, c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = decode2<DT, HI>(w[2 * j], sc[2 * j] << 23);
        const uint32_t y = decode2<DT, HI>(w[2 * j + 1], sc[2 * j + 1] << 23);
        a[j] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        c[j] = __builtin_amdgcn_perm(y, x, 0x07060302u);
      }
      *reinterpret_cast<u32x4_t*>(vb + 4 * tile * kFrag) = a;
      if (both) *reinterpret_cast<u32x4_t*>(vb + 4 * (tile + 1) * kFrag) = c;
    };
#pragma unroll
    for (int w = 0; w < (L::kA == 8 ? 2 : 1); ++w) {
      uint32_t x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = rv[j][w];
      pair(x, rvs, std::false_type{}, 4 * w, true);
      if constexpr (L::kA >= 4) pair(x, rvs, std::true_type{}, 4 * w + 2, true);
    }
    if constexpr (L::kB) pair(rvb, rvsb, std::false_type{}, L::kA, L::kB == 2);
  };

  // A tile with NaN values that some rows of the workgroup see and others do not: 0 * NaN would reach
  // those.  The NaNs are put into the outputs of the rows that see them, where a product of marks and
  // visibility finds any, and then taken out of the tile.
  auto take_nans = [&](int tile0, int buf) {
    constexpr uint32_t kInfBits = DT == IN_BF16 ? 0x7F80u : 0x7C00u, kOne = DT == IN_BF16 ? 0x3F80u : 0x3C00u;
    auto nans = [](u32x4_t x) {                  // all bits of the NaN halves
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = ((x[j] & 0x7FFFu) > kInfBits ? 0xFFFFu : 0u) | (((x[j] >> 16) & 0x7FFFu) > kInfBits ? 0xFFFF0000u : 0u);
      return x;
    };
    const uint32_t from = uint32_t(first - tile0 - 8 * h), many = uint32_t(max(min(last, hi - 1) - first + 1, 0));
#pragma nounroll
    for (int u = 0; u < 4; ++u) {
      u32x4_t see;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        see[j] = (uint32_t(16 * u + 2 * j) - from < many ? kOne : 0u) |
                 (uint32_t(16 * u + 2 * j + 1) - from < many ? kOne << 16 : 0u);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        u32x4_t mark = nans(*reinterpret_cast<const u32x4_t*>(lds[buf] + (kFragsK + 4 * t + u) * kFrag + lane * 16));
        mark &= kOne | kOne << 16;
        v16f_t hits;
#pragma unroll
        for (int v = 0; v < 16; ++v) hits[v] = 0.0f;
        hits = mfma32<DT>(mark, see, hits);
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int any = -__float_as_int(hits[v]) >> 31;
          o[t][v] = __uint_as_float(__float_as_uint(o[t][v]) | (uint32_t(any) & 0x7FC00000u));
        }
        __builtin_amdgcn_sched_barrier(0);       // one fragment at a time: this path shall cost no registers
      }
    }
    __syncthreads();
    for (int f = kFragsK + wave; f < kFrags; f += NW) {
      u32x4_t* at = reinterpret_cast<u32x4_t*>(lds[buf] + f * kFrag + lane * 16);
      *at &= ~nans(*at);
    }
    __syncthreads();
  };

  auto compute = [&](int tile0, int buf) {
    const uint8_t* base = lds[buf] + lane * 16;
    // ---- S^T
    v16f_t s[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int v = 0; v < 16; ++v) s[kt][v] = 0.0f;
#pragma unroll
      for (int f = 0; f < kSteps; ++f)
        s[kt] = mfma32<DT>(*reinterpret_cast<const u32x4_t*>(base + (kt * kSteps + f) * kFrag), qf[f], s[kt]);
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
      const float a = mref == next ? 1.0f : __builtin_amdgcn_exp2f(mref - next);
      mref = next;
      l *= a;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) o[t] *= a;
    }
    // ---- weights
    u32x4_t p[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u >> 1][8 * (u & 1) + j], g.c, -mref));
      l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      p[u] = u32x4_t{pack2<DT>(e[0], e[1]), pack2<DT>(e[2], e[3]), pack2<DT>(e[4], e[5]), pack2<DT>(e[6], e[7])};
    }
    // ---- O^T
    const uint8_t* vbase = base + kFragsK * kFrag;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        o[t] = mfma32<DT>(*reinterpret_cast<const u32x4_t*>(vbase + (4 * t + u) * kFrag), p[u], o[t]);
  };

  if (start < hi) {
    load(start);
    decode(start, 0);
    if (start + 64 < hi) load(start + 64);
    __syncthreads();
    int buf = 0;
    for (int tile0 = start; tile0 < hi; tile0 += 64) {
      if (tile0 + 64 < hi) {
        decode(tile0 + 64, buf ^ 1);
        if (tile0 + 128 < hi) load(tile0 + 128);
      }
      if (nan_tile[buf][0] | nan_tile[buf][1] | nan_tile[buf][2] | nan_tile[buf][3]) take_nans(tile0, buf);
      compute(tile0, buf);
      __syncthreads();
      buf ^= 1;
    }
  }

  // ---- outputs: the lane holds channels kA c + t of the first run (c = 8 (v / 4) + 4 h + v % 4), likewise of the second
  l += __shfl_xor(l, 32, 64);
  if (orow < 0) return;
  const bool direct = g.splits == 1;
  const float inv = direct ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
  auto put = [&](int base, int tile0, auto kWidth) {
    constexpr int W = decltype(kWidth)::value;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t d = base + W * (8 * (v >> 2) + 4 * h + (v & 3));
      if (direct) {
        T* dst = static_cast<T*>(g.out) + orow * D + d;
        if constexpr (W == 1) *dst = T(pack2<DT>(o[tile0][v] * inv, 0.0f));
        else
#pragma unroll
          for (int t = 0; t < W; t += 2)
            *reinterpret_cast<uint32_t*>(dst + t) = pack2<DT>(o[tile0 + t][v] * inv, o[tile0 + t + (W > 1)][v] * inv);
      } else {
        float* dst = g.part + (orow * g.splits + split) * D + d;
#pragma unroll
        for (int t = 0; t < W; ++t) dst[t] = o[tile0 + t][v];
      }
    }
  };
  put(0, 0, std::integral_constant<int, L::kA>{});
  if constexpr (L::kB) put(32 * L::kA, L::kA, std::integral_constant<int, L::kB>{});
  if (h == 0) put_stats<DT>(g, orow, split, mref, l);
}

// Joins the splits of one row: o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// One wave per row; a lane takes channels 2 lane, 2 lane + 1 of each 128.
template <int DT, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttnArgs g, int64_t requests) {
  const int lane = threadIdx.x & 63;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= g.tokens * g.heads) return;
  const int64_t token = row / g.heads;
  if (token < g.cu[0] || token >= g.cu[requests]) return;
  const float* ml = g.part_ml + row * g.splits * 2;
  float top = kLowest;
  for (int i = lane; i < g.splits; i += 64)
    if (ml[2 * i + 1] != 0.0f) top = fmaxf(top, ml[2 * i]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  float sum = 0.0f;
  constexpr int kPer = (D + 127) / 128;
  v2f acc[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) acc[u] = v2f{0, 0};
  for (int i = 0; i < g.splits; ++i) {
    const float li = ml[2 * i + 1], mi = ml[2 * i];
    if (li == 0.0f) continue;
    const float w = mi == top ? 1.0f : __builtin_amdgcn_exp2f(mi - top);
    sum += w * li;
    const float* o = g.part + (row * g.splits + i) * D;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int d = u * 128 + 2 * lane;
      if (d < D) {
        const float2 x = *reinterpret_cast<const float2*>(o + d);
        acc[u][0] += w * x.x;
        acc[u][1] += w * x.y;
      }
    }
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
  int nq;                       // 16-row tiles of attention_kernel
  bool tiles;                   // some request may have more than kFewRows rows
  bool few;                     // some request may have no more
  int64_t row_tiles, tile_rows; // of attention_tile_kernel
  int64_t splits, chunk;
  int64_t bytes;                // workspace
};

constexpr int kWaves = 4;

mx_status_t plan_attention(int64_t tokens, int heads, int kv_heads, int dim, int64_t requests, int64_t max_q,
                           int64_t max_kv, int64_t window, Plan& p) {
  const int64_t lim = int64_t(1) << 30;
  if (tokens < 0 || requests < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || heads > 65536) return MX_ERR_SHAPE;
  if (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256) return MX_ERR_SHAPE;
  if (max_q < 0 || max_kv < 0 || window < 0) return MX_ERR_ARG;
  if (tokens > lim || requests > lim || max_kv > lim || max_q > lim) return MX_ERR_SHAPE;
  const int64_t cus = device_cus();
  if (cus <= 0) return MX_ERR_LAUNCH;
  const int64_t group = heads / kv_heads, reqs = std::max<int64_t>(requests, 1);
  const int64_t rows = std::max<int64_t>(std::min(max_q, tokens) * group, 1);
  p.tiles = rows > kFewRows;
  p.few = !p.tiles || requests > 1;
  p.nq = std::min<int64_t>(rows, p.tiles ? kFewRows : rows) <= 16 ? 1 : 2;
  p.tile_rows = dim > 128 ? 128 : 256;
  p.row_tiles = p.tiles ? (rows + p.tile_rows - 1) / p.tile_rows : 1;
  // keys that one row tile can see
  int64_t keys = max_kv;
  if (window > 0) keys = std::min(keys, window + (p.tiles ? p.tile_rows : kFewRows) / group + 33);
  keys = std::max<int64_t>((keys + 31) / 32 * 32, 32);
  // Splits: enough workgroups for three of attention_kernel on every CU, or one and a half of
  // attention_tile_kernel (one fits a CU), but none with less than two steps a wave or four tiles.
  const int64_t base = p.tiles ? std::min(reqs * p.row_tiles, tokens * group / p.tile_rows + reqs) * kv_heads
                               : reqs * kv_heads;
  const int64_t want = std::max<int64_t>(1, (p.tiles ? cus + cus / 2 : 3 * cus) / base);
  p.chunk = std::max<int64_t>((keys + want - 1) / want, 256);
  p.chunk = (p.chunk + 127) / 128 * 128;
  p.splits = (keys + p.chunk - 1) / p.chunk;
  p.bytes = p.splits > 1 ? tokens * heads * p.splits * (dim + 2) * 4 : 0;
  if (reqs * kv_heads * p.row_tiles > 0x7FFFFFFF / p.splits) return MX_ERR_SHAPE;
  return MX_OK;
}

template <int DT, int D>
void launch_attention(const Plan& p, AttnArgs g, int64_t requests, hipStream_t stream) {
  if (p.tiles) {
    constexpr int NW = D > 128 ? 4 : 8;
    const unsigned grid = unsigned(requests * g.kv_heads * p.row_tiles * p.splits);
    attention_tile_kernel<DT, D, NW><<<grid, 64 * NW, 0, stream>>>(g);
  }
  if (p.few) {
    g.few_only = p.tiles;
    g.row_tiles = 1;
    const unsigned grid = unsigned(requests * g.kv_heads * p.splits);
    if (p.nq == 1) attention_kernel<DT, D, 1, kWaves><<<grid, 64 * kWaves, 0, stream>>>(g);
    else attention_kernel<DT, D, 2, kWaves><<<grid, 64 * kWaves, 0, stream>>>(g);
  }
  if (p.splits > 1)
    attention_join_kernel<DT, D><<<unsigned((g.tokens * g.heads + 3) / 4), 256, 0, stream>>>(g, requests);
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
  if (!q || !cu || !lens || !out || (max_kv > 0 && !page_table)) return MX_ERR_NULL;
  if (cache->pages > 0 && (!cache->k || !cache->k_scales || !cache->v || !cache->v_scales)) return MX_ERR_NULL;
  if (misaligned(q) || misaligned(out) || misaligned(cache->k) || misaligned(cache->v) || misaligned(workspace) ||
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
  g.part_ml = g.part ? g.part + tokens * heads * p.splits * cache->dim : nullptr;
  g.tokens = tokens; g.max_q = max_q; g.max_kv = max_kv;
  g.heads = heads; g.kv_heads = cache->kv_heads; g.group = heads / cache->kv_heads; g.page = cache->page;
  g.window = int(std::min<int64_t>(window, int64_t(1) << 30));
  g.row_tiles = int(p.row_tiles); g.splits = int(p.splits); g.chunk = int(p.chunk);
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
