// Rotary positions and the append to a paged MXFP8 key/value cache on gfx950.
//
// A rotary embedding turns channel pair i of a token at position p by the angle
// p f_i: (a, b) -> (a c - b s, b c + a s).  The rotation is orthogonal, so its
// backward pass is the same map with s negated.  All three operators here are
// bound by memory: a table write, one read and one write of the tensor, or one
// read of q, k and v and one write of q and of a little over a byte per element
// of k and v.

#include "mx_device.hpp"
#include "mx_launch.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace mxk {

// ---------------------------------------------------------------------------
// Table
// ---------------------------------------------------------------------------
struct TableArgs {
  float2* out;
  int64_t rows;
  int pairs;
  int scaling;
  double base, rot, factor, lo, hi, turns, m;   // turns = orig_len / (2 pi)
};

// One thread fills kRun consecutive rows of one pair.  The first angle and the
// step of one position go through sincos in FP64; every further row is one
// complex product, z_{n+1} = z_n w, whose error grows by about 2^-52 a step and
// so stays far below the FP32 result's rounding.  Consecutive lanes hold
// consecutive pairs, so a row is written with contiguous 8-byte stores.  Measured:
// 131072 rows of 64 pairs in 12.8 us, 5.2 TB/s written, what the memory takes; 8192 rows
// in 5.5 us, the launch.
template <int kRun>
__global__ __launch_bounds__(256) void rope_table_kernel(const TableArgs g) {
  const int64_t id = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t run = id / g.pairs;
  const int i = int(id - run * g.pairs);
  const int64_t row0 = run * kRun;
  if (row0 >= g.rows) return;
  double f = pow(g.base, -2.0 * double(i) / g.rot);
  if (g.scaling == MX_ROPE_LINEAR) {
    f /= g.factor;
  } else if (g.scaling == MX_ROPE_YARN) {
    const double r = fmin(fmax((double(i) - g.lo) / fmax(g.hi - g.lo, 1e-3), 0.0), 1.0);
    f = f * (1.0 - r) + f / g.factor * r;
  } else if (g.scaling == MX_ROPE_BANDS) {
    const double s = fmin(fmax((g.turns * f - 1.0) / 3.0, 0.0), 1.0);
    f = s * f + (1.0 - s) * f / g.factor;
  }
  double zs, zc, ws, wc;
  sincos(double(row0) * f, &zs, &zc);
  sincos(f, &ws, &wc);
  zs *= g.m;
  zc *= g.m;
  float2* o = g.out + row0 * g.pairs + i;
#pragma unroll
  for (int n = 0; n < kRun; ++n) {
    if (row0 + n >= g.rows) return;
    o[int64_t(n) * g.pairs] = make_float2(float(zc), float(zs));
    const double c = fma(zc, wc, -zs * ws);
    zs = fma(zc, ws, zs * wc);
    zc = c;
  }
}

// ---------------------------------------------------------------------------
// Rotation
// ---------------------------------------------------------------------------
// n / d for n < 2^31 as floor(n m / 2^(31 + s)), s = ceil(log2 d), m = ceil(2^(31 + s) / d) < 2^32: the
// excess m d - 2^(31 + s) is below 2^s, so n times it is below 2^(31 + s).  A thread here moves a few
// dozen bytes, which a division by the compiler (20 instructions, over 100 in 64 bits) would outweigh.
struct Divisor {
  uint32_t m, shift, d;
  Divisor(uint32_t by = 1) : m(0), shift(0), d(by) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < by) ++s;
    if (by > 1) {
      m = uint32_t(((uint64_t(1) << (31 + s)) + by - 1) / by);
      shift = s - 1;
    }
  }
  __device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t& rest) const {
    const uint32_t q = d == 1 ? n : __umulhi(n, m) >> shift;
    rest = n - q * d;
    return q;
  }
};

struct RopeArgs {
  const void* x;
  void* y;
  const int32_t* pos;
  const float2* table;
  int64_t tokens, rows;
  int64_t xt, xh, yt, yh;       // strides in elements
  int heads, dim, rot;
  Divisor chunks;               // V-element accesses a head needs: rot / 2 / V pairs and (dim - rot) / V copies
  Divisor head_groups;
  bool inverse;
};

template <int IN> struct Elem { using T = uint16_t; };
template <> struct Elem<IN_F32> { using T = uint32_t; };

template <int IN>
__device__ __forceinline__ float widen(typename Elem<IN>::T b) {
  if constexpr (IN == IN_F32) return __uint_as_float(b);
  else if constexpr (IN == IN_BF16) return __uint_as_float(uint32_t(b) << 16);
  else return f16_bits_to_f32(b);
}

typedef float v2f_t __attribute__((ext_vector_type(2)));

// RNE narrowing to the storage type.
template <int IN>
__device__ __forceinline__ typename Elem<IN>::T narrow(float v) {
  if constexpr (IN == IN_F32) return __float_as_uint(v);
  else if constexpr (IN == IN_BF16) return __builtin_bit_cast(uint16_t, __bf16(v));
  else return __builtin_bit_cast(uint16_t, _Float16(v));
}

// V storage elements moved with one access of up to 16 bytes, as 32-bit words (words and not elements:
// arrays of 16-bit elements would be kept in LDS by the compiler, not in registers).
template <int IN, int V>
struct Pack {
  using T = typename Elem<IN>::T;
  static constexpr int kBytes = V * int(sizeof(T)), kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 16) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (kBytes == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *p;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *p = T(w[0]);
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (IN == IN_F32) return widen<IN>(w[j]);
    else return widen<IN>(T(w[j / 2] >> (16 * (j & 1))));
  }
  // elements 0 .. V - 1 from FP32 values
  __device__ __forceinline__ void set(const float (&v)[V]) {
    if constexpr (IN == IN_F32) {
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = narrow<IN>(v[j]);
    } else if constexpr (V == 1) {
      w[0] = narrow<IN>(v[0]);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) w[j] = uint32_t(narrow<IN>(v[2 * j])) | uint32_t(narrow<IN>(v[2 * j + 1])) << 16;
    }
  }
};

// The cos / sin pairs of pairs [i, i + V) of a table row; NaN where the position
// has no row.
template <int V>
__device__ __forceinline__ void load_cs(const float2* __restrict__ table, int64_t rows, int pairs, int32_t pos, int i,
                                        bool inverse, float (&c)[V], float (&s)[V]) {
  if (pos < 0 || pos >= rows) {
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = s[j] = __uint_as_float(0x7FC00000u);
    return;
  }
  const float2* row = table + int64_t(pos) * pairs + i;
  if constexpr (V % 2 == 0) {      // V divides pairs, so the address is a multiple of 16 bytes
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float4 t = *reinterpret_cast<const float4*>(row + j);
      c[j] = t.x; s[j] = t.y; c[j + 1] = t.z; s[j + 1] = t.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) { c[j] = row[j].x; s[j] = row[j].y; }
  }
  if (inverse) {
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = -s[j];
  }
}

// One thread: one chunk (V pairs, or V copied channels) of HPT heads of one
// token.  The table entries are loaded once for all its heads (for every head, a
// table row would be twice a BF16 head's bytes).  Measured: 8192 tokens of 32 heads of
// 128 BF16 channels in 28.6 us, 4.8 TB/s, near the rate of a plain copy (5.1).
template <int IN, int V, bool HALF, int HPT>
__device__ __forceinline__ void rope_item(const RopeArgs& g, uint32_t id) {
  using P = Pack<IN, V>;
  using T = typename Elem<IN>::T;
  uint32_t ch, hg;
  const int64_t t = g.head_groups.divide(g.chunks.divide(id, ch), hg);
  if (t >= g.tokens) return;
  const int h0 = int(hg) * HPT, nh = min(HPT, g.heads - h0);
  const T* x = static_cast<const T*>(g.x) + t * g.xt + h0 * g.xh;
  T* y = static_cast<T*>(g.y) + t * g.yt + h0 * g.yh;
  const int pairs = g.rot / 2, i = int(ch) * V;
  if (i >= pairs) {                // channels past the rotation
    const int c = g.rot + (i - pairs);
    P p[HPT];
#pragma unroll
    for (int h = 0; h < HPT; ++h)
      if (h < nh) p[h].load(x + h * g.xh + c);
#pragma unroll
    for (int h = 0; h < HPT; ++h)
      if (h < nh) p[h].store(y + h * g.yh + c);
    return;
  }
  const int ca = HALF ? i : 2 * i, cb = HALF ? i + pairs : 2 * i + V;
  P a[HPT], b[HPT];
#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (h < nh) {
      a[h].load(x + h * g.xh + ca);
      b[h].load(x + h * g.xh + cb);
    }
  float c[V], s[V];
  load_cs<V>(g.table, g.rows, pairs, g.pos[t], i, g.inverse, c, s);
#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (h < nh) {
      float oa[V], ob[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // half: pair j is (a_j, b_j); interleaved: elements 2 j, 2 j + 1 of a followed by b
        const float u = HALF ? a[h].get(j) : 2 * j < V ? a[h].get(2 * j) : b[h].get(2 * j - V);
        const float w = HALF ? b[h].get(j) : 2 * j + 1 < V ? a[h].get(2 * j + 1) : b[h].get(2 * j + 1 - V);
        const float p = u * c[j] - w * s[j], q = w * c[j] + u * s[j];
        if (HALF) {
          oa[j] = p;
          ob[j] = q;
        } else {
          if (2 * j < V) oa[2 * j] = p;
          else ob[2 * j - V] = p;
          if (2 * j + 1 < V) oa[2 * j + 1] = q;
          else ob[2 * j + 1 - V] = q;
        }
      }
      P out;
      out.set(oa);
      out.store(y + h * g.yh + ca);
      out.set(ob);
      out.store(y + h * g.yh + cb);
    }
}

template <int IN, int V, bool HALF, int HPT>
__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs g) {
  rope_item<IN, V, HALF, HPT>(g, blockIdx.x * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
struct AppendArgs {
  RopeArgs q;                   // the rotation of q (q.tokens == 0: none) and the table
  const void* k;
  const void* v;
  int64_t kt, kh, vt, vh;
  const int64_t* slots;
  uint8_t *kc, *ks, *vc, *vs;
  int64_t tokens, slot_count;
  int kv_heads, page, dim;
  double inv_page;
  Divisor per_head, head_groups;
  uint32_t q_blocks, kv_blocks; // workgroups that rotate q, then those of k, then those of v
};

// Channel ch of the rotated key, element by element (any layout and alignment).
template <int IN, bool HALF>
__device__ __forceinline__ float rotated_one(const typename Elem<IN>::T* x, const float2* row, bool ok, int rot, int ch) {
  const float own = widen<IN>(x[ch]);
  if (ch >= rot) return own;
  const int half = rot / 2;
  const int i = HALF ? (ch < half ? ch : ch - half) : ch >> 1;
  const bool first = HALF ? ch < half : (ch & 1) == 0;
  const float other = widen<IN>(x[HALF ? (first ? ch + half : ch - half) : ch ^ 1]);
  const float c = ok ? row[i].x : __uint_as_float(0x7FC00000u), s = ok ? row[i].y : __uint_as_float(0x7FC00000u);
  return first ? own * c - other * s : own * c + other * s;
}

// One thread: 8 consecutive channels from ch on (a multiple of 8) of HPT heads of one
// token's keys (ROTATE) or values.  VEC: rows are 16-byte aligned and, where there is a
// rotation, rot / 2 is a multiple of 8, so a chunk lies in one half (or one run of
// interleaved pairs) and so does its partner.  The four lanes of a quad hold one block of 32.
template <int IN, bool VEC, bool HALF, int HPT, bool ROTATE>
__device__ __forceinline__ void append_item(const AppendArgs& g, const void* base, int64_t ts, int64_t hs, uint8_t* codes,
                                            uint8_t* scales, uint32_t id) {
  using T = typename Elem<IN>::T;
  uint32_t c8, hg;
  const int64_t t = g.head_groups.divide(g.per_head.divide(id, c8), hg);
  if (t >= g.tokens) return;                            // whole quads leave together
  const int ch = int(c8) * 8, h0 = int(hg) * HPT;
  const T* x = static_cast<const T*>(base) + t * ts + h0 * hs;
  const int half = g.q.rot / 2;
  const bool turn = ROTATE && ch < g.q.rot;
  const bool first = !HALF || ch < half;                // of a pair's halves
  const int i = HALF ? (first ? ch : ch - half) : ch / 2;
  float v[HPT][8], c[8], s[8], p[HPT][HALF ? 8 : 1];
  const int64_t slot = g.slots[t];
  const int32_t pos = ROTATE ? g.q.pos[t] : 0;
#pragma unroll
  for (int h = 0; h < HPT; ++h) {
    if (h0 + h >= g.kv_heads) continue;
    if constexpr (VEC) {
      load8<IN>(x + h * hs, ch, v[h]);
      if constexpr (HALF)
        if (turn) load8<IN>(x + h * hs, first ? ch + half : i, p[h]);
    } else {
      const bool ok = ROTATE && pos >= 0 && pos < g.q.rows;
      const float2* row = ok ? g.q.table + int64_t(pos) * half : nullptr;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[h][j] = ROTATE ? rotated_one<IN, HALF>(x + h * hs, row, ok, g.q.rot, ch + j) : widen<IN>(x[h * hs + ch + j]);
    }
  }
  if constexpr (VEC && ROTATE) {
    if (turn) {
      if constexpr (HALF) {
        // first half: own c - other s; second: own c + other s, a subtraction of the negated product
        load_cs<8>(g.q.table, g.q.rows, half, pos, i, !first, c, s);
#pragma unroll
        for (int h = 0; h < HPT; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[h][j] = v[h][j] * c[j] - p[h][j] * s[j];
      } else {
        float c4[4], s4[4];
        load_cs<4>(g.q.table, g.q.rows, half, pos, i, false, c4, s4);
#pragma unroll
        for (int h = 0; h < HPT; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float a = v[h][2 * j], b = v[h][2 * j + 1];
            v[h][2 * j] = a * c4[j] - b * s4[j];
            v[h][2 * j + 1] = b * c4[j] + a * s4[j];
          }
      }
    }
  }
  const bool store = slot >= 0 && slot < g.slot_count;
  const int64_t page = int64_t((double(slot) + 0.5) * g.inv_page);      // slot < 2^34: exact
  const int64_t row0 = (page * g.kv_heads + h0) * g.page + (slot - page * g.page);
#pragma unroll
  for (int h = 0; h < HPT; ++h) {
    if (h0 + h >= g.kv_heads) continue;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(v[h][j]));
    m = quad_max(m);
    uint32_t w[2];
    const uint32_t scale = mx_encode_f32<E4M3, CEIL, 8>(v[h], m, w);
    if (!store) continue;
    const int64_t row = row0 + int64_t(h) * g.page;
    *reinterpret_cast<uint2*>(codes + row * g.dim + ch) = make_uint2(w[0], w[1]);
    if ((c8 & 3) == 0) scales[row * (g.dim / 32) + c8 / 4] = uint8_t(scale);
  }
}

// One launch does all three tensors: the first q_blocks workgroups rotate q, the
// next kv_blocks rotate and encode k, the last kv_blocks encode v.  Measured: 8192
// tokens of 32 + 8 + 8 heads of 128 BF16 channels in 45 us, 4.2 TB/s; one
// token 6.6 us, of which the kernel is 2.4 and the call the rest.
template <int IN, int VQ, bool HALF, int HPT, bool VEC>
__global__ __launch_bounds__(256) void append_kernel(const AppendArgs g) {
  uint32_t b = blockIdx.x;
  if (b < g.q_blocks) {
    rope_item<IN, VQ, HALF, HPT>(g.q, b * 256 + threadIdx.x);
    return;
  }
  b -= g.q_blocks;
  if (b >= g.kv_blocks)
    append_item<IN, VEC, HALF, HPT, false>(g, g.v, g.vt, g.vh, g.vc, g.vs, (b - g.kv_blocks) * 256 + threadIdx.x);
  else if (g.q.table)
    append_item<IN, VEC, HALF, HPT, true>(g, g.k, g.kt, g.kh, g.kc, g.ks, b * 256 + threadIdx.x);
  else
    append_item<IN, VEC, HALF, HPT, false>(g, g.k, g.kt, g.kh, g.kc, g.ks, b * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
inline int elem_size(mx_dtype_t t) { return t == MX_F32 ? 4 : 2; }

// Largest number of elements V in {16 bytes' worth, 2, 1} that every access of the
// rotation can move at once: V divides the pairs and the channels past them, and
// every row starts on a multiple of V elements.
int rope_vector(mx_dtype_t dt, int dim, int rot, const void* x, const void* y, int64_t s0, int64_t s1, int64_t s2,
                int64_t s3) {
  const int size = elem_size(dt);
  for (int v : {16 / size, 2}) {
    const uintptr_t addr = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
    if ((rot / 2) % v == 0 && (dim - rot) % v == 0 && addr % uintptr_t(v * size) == 0 &&
        (s0 | s1 | s2 | s3) % v == 0)
      return v;
  }
  return 1;
}

// Threads that take four heads at once read a table row a quarter as often, but a
// small call then has too few threads to cover the load latency: four from 2^18 chunks
// on, 256 waves for every XCD.
inline int heads_per_thread(int64_t tokens, int heads, int chunks) {
  return tokens * heads >= ((int64_t(1) << 18) + chunks - 1) / chunks && heads >= 4 ? 4 : 1;
}

void fill_rope(RopeArgs& g, const void* x, void* y, int64_t tokens, int heads, int dim, int64_t xt, int64_t xh,
               int64_t yt, int64_t yh, const int32_t* pos, const float* table, int64_t rows, int rot, bool inverse,
               int v, int hpt) {
  g.x = x; g.y = y; g.pos = pos; g.table = reinterpret_cast<const float2*>(table);
  g.tokens = tokens; g.rows = rows; g.xt = xt; g.xh = xh; g.yt = yt; g.yh = yh;
  g.heads = heads; g.dim = dim; g.rot = rot; g.inverse = inverse;
  g.chunks = Divisor(uint32_t((rot / 2 + dim - rot) / v));
  g.head_groups = Divisor(uint32_t((heads + hpt - 1) / hpt));
}

inline mx_status_t launched() { return hipGetLastError() == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

mx_status_t check_rotation(mx_dtype_t dtype, int64_t tokens, int dim, int64_t rows, int rot, mx_rope_layout_t layout) {
  if (dtype != MX_F32 && dtype != MX_BF16 && dtype != MX_F16) return MX_ERR_UNSUPPORTED;
  if (layout != MX_ROPE_HALF && layout != MX_ROPE_INTERLEAVED) return MX_ERR_UNSUPPORTED;
  if (tokens < 0 || tokens > (int64_t(1) << 31) || rows < 0 || dim < 2 || dim > 65536) return MX_ERR_SHAPE;
  if (rot < 2 || rot % 2 || rot > dim) return MX_ERR_SHAPE;
  return MX_OK;
}

// Calls f(integral_constant of V, of HPT) for the run-time pair.
template <int IN, class F>
void with_variant(int v, int hpt, F f) {
  constexpr int kWide = IN == IN_F32 ? 4 : 8;
  auto h = [&](auto vv) {
    if (hpt == 4) f(vv, std::integral_constant<int, 4>{});
    else f(vv, std::integral_constant<int, 1>{});
  };
  if (v == kWide) h(std::integral_constant<int, kWide>{});
  else if (v == 2) h(std::integral_constant<int, 2>{});
  else h(std::integral_constant<int, 1>{});
}

template <class F>
void with_type(mx_dtype_t dt, F f) {
  if (dt == MX_F32) f(std::integral_constant<int, IN_F32>{});
  else if (dt == MX_BF16) f(std::integral_constant<int, IN_BF16>{});
  else f(std::integral_constant<int, IN_F16>{});
}

}  // namespace mxk

using namespace mxk;

extern "C" mx_status_t mx_rope_table(int64_t rows, int rot, double base, mx_rope_scaling_t scaling, double factor,
                                     int64_t orig_len, float* table, hipStream_t stream) {
  if (scaling < MX_ROPE_NONE || scaling > MX_ROPE_BANDS) return MX_ERR_UNSUPPORTED;
  if (rows < 0 || rows > (int64_t(1) << 31) || rot < 2 || rot > 1024 || rot % 2) return MX_ERR_SHAPE;
  if (scaling == MX_ROPE_NTK && rot < 4) return MX_ERR_SHAPE;
  if (!std::isfinite(base) || base <= 1.0) return MX_ERR_ARG;
  if (scaling != MX_ROPE_NONE && (!std::isfinite(factor) || factor < 1.0)) return MX_ERR_ARG;
  const bool needs_len = scaling == MX_ROPE_YARN || scaling == MX_ROPE_BANDS;
  if (needs_len && orig_len < 1) return MX_ERR_ARG;
  if (rows == 0) return MX_OK;
  if (!table) return MX_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(table) & 7u) return MX_ERR_ALIGN;
  TableArgs g = {};
  g.out = reinterpret_cast<float2*>(table);
  g.rows = rows;
  g.pairs = rot / 2;
  g.scaling = scaling;
  g.rot = rot;
  g.base = scaling == MX_ROPE_NTK ? base * std::pow(factor, rot / (rot - 2.0)) : base;
  if (!std::isfinite(g.base)) return MX_ERR_ARG;
  g.factor = factor;
  g.m = 1.0;
  const double two_pi = 6.283185307179586476925286766559;
  if (needs_len) g.turns = double(orig_len) / two_pi;
  if (scaling == MX_ROPE_YARN) {
    auto d = [&](double n) { return rot * std::log(double(orig_len) / (two_pi * n)) / (2.0 * std::log(base)); };
    g.lo = std::fmax(std::floor(d(32.0)), 0.0);
    g.hi = std::fmin(std::ceil(d(1.0)), rot - 1.0);
    g.m = 1.0 + 0.1 * std::log(factor);
  }
  // long tables amortise the two sincos of a thread over 32 rows; short ones need the threads
  const bool wide = rows * g.pairs >= (int64_t(1) << 21);
  const int64_t runs = (rows + (wide ? 31 : 7)) / (wide ? 32 : 8);
  const unsigned blocks = unsigned((runs * g.pairs + 255) / 256);
  if (wide) rope_table_kernel<32><<<blocks, 256, 0, stream>>>(g);
  else rope_table_kernel<8><<<blocks, 256, 0, stream>>>(g);
  return launched();
}

extern "C" mx_status_t mx_rope(const void* x, mx_dtype_t dtype, int64_t tokens, int heads, int dim,
                               int64_t x_token_stride, int64_t x_head_stride, const int32_t* pos, const float* table,
                               int64_t rows, int rot, mx_rope_layout_t layout, int inverse, void* y,
                               int64_t y_token_stride, int64_t y_head_stride, hipStream_t stream) {
  const mx_status_t st = check_rotation(dtype, tokens, dim, rows, rot, layout);
  if (st != MX_OK) return st;
  if (heads < 0 || heads > 65536) return MX_ERR_SHAPE;
  if (tokens == 0 || heads == 0) return MX_OK;
  if (!x || !y || !pos || !table) return MX_ERR_NULL;
  const uintptr_t both = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
  if (both % elem_size(dtype) || misaligned(table) || (reinterpret_cast<uintptr_t>(pos) & 3u)) return MX_ERR_ALIGN;
  const int v = rope_vector(dtype, dim, rot, x, y, x_token_stride, x_head_stride, y_token_stride, y_head_stride);
  const int hpt = heads_per_thread(tokens, heads, (rot / 2 + dim - rot) / v);
  // thread numbers are kept below 2^31: longer inputs go in several launches (a token of 65536 heads of
  // 65536 channels has 2^30 threads, as four heads go to each)
  const int64_t per_token = int64_t((heads + hpt - 1) / hpt) * ((rot / 2 + dim - rot) / v);
  const int64_t slab = int64_t(0x7FFFFE00) / per_token;
  const int64_t size = elem_size(dtype);
  for (int64_t t = 0; t < tokens; t += slab) {
    const int64_t n = std::min(slab, tokens - t);
    RopeArgs g;
    fill_rope(g, static_cast<const uint8_t*>(x) + t * x_token_stride * size, static_cast<uint8_t*>(y) + t * y_token_stride * size,
              n, heads, dim, x_token_stride, x_head_stride, y_token_stride, y_head_stride, pos + t, table, rows, rot,
              inverse != 0, v, hpt);
    const unsigned blocks = unsigned((n * per_token + 255) / 256);
    with_type(dtype, [&](auto in) {
      constexpr int IN = decltype(in)::value;
      with_variant<IN>(v, hpt, [&](auto vv, auto hh) {
        constexpr int V = decltype(vv)::value, H = decltype(hh)::value;
        if (layout == MX_ROPE_HALF) rope_kernel<IN, V, true, H><<<blocks, 256, 0, stream>>>(g);
        else rope_kernel<IN, V, false, H><<<blocks, 256, 0, stream>>>(g);
      });
    });
  }
  return launched();
}

extern "C" mx_status_t mx_kv_append(const void* k, const void* v, mx_dtype_t dtype, int64_t tokens,
                                    int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                    int64_t v_head_stride, const mx_kv_cache_t* cache, const int64_t* slots,
                                    const int32_t* pos, const float* table, int64_t rows, int rot,
                                    mx_rope_layout_t layout, const void* q, int heads, int64_t q_token_stride,
                                    int64_t q_head_stride, void* q_out, hipStream_t stream) {
  if (!cache) return MX_ERR_NULL;
  const int dim = cache->dim;
  mx_status_t st = check_kv_cache(*cache);
  if (st != MX_OK) return st;
  st = check_rotation(dtype, tokens, dim, rows, table ? rot : 2, layout);
  if (st != MX_OK) return st;
  if (q && (heads < 1 || heads > 65536)) return MX_ERR_SHAPE;
  if (tokens == 0) return MX_OK;
  if (!k || !v || !slots || (table && !pos) || (q && (!table || !q_out))) return MX_ERR_NULL;
  if (cache->pages > 0 && (!cache->k || !cache->k_scales || !cache->v || !cache->v_scales)) return MX_ERR_NULL;
  const int size = elem_size(dtype);
  const uintptr_t kv = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
  if (kv % size || misaligned(table) || (reinterpret_cast<uintptr_t>(pos) & 3u) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) || misaligned(cache->k) || misaligned(cache->v) ||
      misaligned(cache->k_scales) || misaligned(cache->v_scales))
    return MX_ERR_ALIGN;
  if (q && (reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out)) % size) return MX_ERR_ALIGN;
  const int kv_heads = cache->kv_heads;
  int vq = 16 / size, hpt = heads_per_thread(tokens, kv_heads, dim / 8);
  int64_t q_threads = 0;                                // of a token
  if (q) {
    vq = rope_vector(dtype, dim, rot, q, q_out, q_token_stride, q_head_stride, int64_t(heads) * dim, dim);
    const int chunks = (rot / 2 + dim - rot) / vq;
    hpt = std::max(hpt, heads_per_thread(tokens, heads, chunks));
    q_threads = int64_t((heads + hpt - 1) / hpt) * chunks;
  }
  const int64_t kv_threads = int64_t((kv_heads + hpt - 1) / hpt) * (dim / 8);
  // 16-byte loads of keys and values: aligned rows, and no 8-channel chunk across the rotation's borders
  const int64_t strides = k_token_stride | k_head_stride | v_token_stride | v_head_stride;
  const bool vec = (kv & 15u) == 0 && strides % (16 / size) == 0 && (!table || (rot / 2) % 8 == 0);
  // thread numbers, and those of all three tensors together, are kept below 2^31: longer inputs go in several
  // launches (a token of 65536 heads of 256 channels has 2^23 threads)
  const int64_t slab = int64_t(0x7FFFFC00) / (q_threads + 2 * kv_threads);
  for (int64_t t = 0; t < tokens; t += slab) {
    const int64_t n = std::min(slab, tokens - t);
    AppendArgs g = {};
    if (q) {
      fill_rope(g.q, static_cast<const uint8_t*>(q) + t * q_token_stride * size, static_cast<uint8_t*>(q_out) + t * heads * dim * size,
                n, heads, dim, q_token_stride, q_head_stride, int64_t(heads) * dim, dim, pos + t, table, rows, rot, false, vq, hpt);
    } else {
      g.q.table = reinterpret_cast<const float2*>(table);
      g.q.pos = table ? pos + t : nullptr;
      g.q.rows = rows;
      g.q.rot = rot;
    }
    g.k = static_cast<const uint8_t*>(k) + t * k_token_stride * size;
    g.v = static_cast<const uint8_t*>(v) + t * v_token_stride * size;
    g.kt = k_token_stride; g.kh = k_head_stride; g.vt = v_token_stride; g.vh = v_head_stride;
    g.slots = slots + t;
    g.kc = cache->k; g.ks = cache->k_scales; g.vc = cache->v; g.vs = cache->v_scales;
    g.tokens = n;
    g.slot_count = cache->pages * cache->page;
    g.kv_heads = kv_heads; g.page = cache->page; g.dim = dim;
    g.inv_page = 1.0 / cache->page;
    g.per_head = Divisor(uint32_t(dim / 8));            // a multiple of 4, so a quad stays in one block of 32
    g.head_groups = Divisor(uint32_t((kv_heads + hpt - 1) / hpt));
    g.q_blocks = uint32_t((n * q_threads + 255) / 256);
    g.kv_blocks = uint32_t((n * kv_threads + 255) / 256);
    const unsigned blocks = g.q_blocks + 2 * g.kv_blocks;
    with_type(dtype, [&](auto in) {
      constexpr int IN = decltype(in)::value;
      with_variant<IN>(vq, hpt, [&](auto vv, auto hh) {
        constexpr int V = decltype(vv)::value, H = decltype(hh)::value;
        const bool half = layout == MX_ROPE_HALF;
        if (vec && half) append_kernel<IN, V, true, H, true><<<blocks, 256, 0, stream>>>(g);
        else if (vec) append_kernel<IN, V, false, H, true><<<blocks, 256, 0, stream>>>(g);
        else if (half) append_kernel<IN, V, true, H, false><<<blocks, 256, 0, stream>>>(g);
        else append_kernel<IN, V, false, H, false><<<blocks, 256, 0, stream>>>(g);
      });
    });
  }
  return launched();
}
