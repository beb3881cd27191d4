// Beam search's selection over beams and vocabulary on gfx950.
//
// A candidate (b, v) of a request has score S_b + x_bv - ln sum_u exp x_bu.  Within a beam the order of scores is
// the order of logits, so one read of the logits gives both things that are needed: the sum, kept with its running
// maximum, and the beam's best `width` logits.  A wave reads a segment of one beam's logits; a second launch joins the
// segments of a request's beams, scores their candidates in 64 bits and takes the best, reorders the token
// histories and appends the tokens.
//
// It is bound by the read of the logits where there are many, by the two launches and their latency where there are few.

#include "mx_launch.hpp"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

namespace mxk {

constexpr int kMostBeams = 64;              // a lane for each when they are merged
constexpr int kMostWidth = 64;              // a lane for each of a beam's candidates
constexpr int kMostSplits = 64;             // a lane for each segment of a beam's logits
constexpr int kFew = 128;                   // candidates of a request that are all compared with each other
constexpr int kGood = 512;                  // and of more, those that can be
constexpr int kBuffer = 512;                // candidates a wave sets aside before it sorts them in
constexpr int64_t kMostBlocks = 1 << 23;    // of 256 threads in a launch, which has fewer than 2^32 threads

typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));      // of logits, at any place of their type
typedef int32_t Vector __attribute__((ext_vector_type(4)));

// Sum and maximum of a segment: sum exp(x - m).
struct Part {
  double s;
  float m;
  uint32_t pad;
};

struct BeamArgs {
  const void* x;
  const float* scores;
  const uint8_t* finished;
  const int32_t *history, *lens;
  float* scores_out;
  int32_t *parents, *tokens, *history_out, *lens_out;
  uint8_t* finished_out;
  Part* parts;                              // [rows][splits]
  uint64_t* best;                           // [rows][splits][keep]
  int64_t request_stride, beam_stride, rows, segment, first;           // first: the workgroup that a launch begins with
  int requests, beams, vocab, width, keep, splits, eos, pad, cols, vector;
};

// Whole numbers in the order of floats (-0 below +0: callers add 0 first).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// The higher the better: the logit, of equal ones the lower token.  0 stands for none.
__device__ __forceinline__ uint64_t candidate(float x, uint32_t token) {
  return uint64_t(ordered(x + 0.0f)) << 32 | uint32_t(~token);
}

// The value of lane ^ D, by moves inside the vector unit: a shuffle through LDS takes some 60 clocks more, and a sort
// is 27 of them one behind the other.
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t x) {
  if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false);             // quads 1 0 3 2
  else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false);        // quads 2 3 0 1
  else if constexpr (D == 4) {
    const uint32_t y = __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false);                    // mirrored eights: lane ^ 7
    return __builtin_amdgcn_mov_dpp(y, 0x1B, 0xF, 0xF, false);                                 // mirrored quads: lane ^ 3
  } else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(x, 0x128, 0xF, 0xF, false);     // sixteens turned by 8
  else if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return threadIdx.x & 16u ? r[0] : r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return threadIdx.x & 32u ? r[0] : r[1];
  }
}

template <int D>
__device__ __forceinline__ uint64_t across(uint64_t x) {
  return uint64_t(across<D>(uint32_t(x >> 32))) << 32 | across<D>(uint32_t(x));
}
template <int D>
__device__ __forceinline__ float across(float x) { return __uint_as_float(across<D>(__float_as_uint(x))); }
template <int D>
__device__ __forceinline__ double across(double x) {
  return __longlong_as_double(int64_t(across<D>(uint64_t(__double_as_longlong(x)))));
}

// f(x of this lane, x of lane ^ D) for D = From, From / 2 .. 1.
template <int From, class T, class F>
__device__ __forceinline__ T fold(T x, F f) {
  x = f(x, across<From>(x), std::integral_constant<int, From>{});
  if constexpr (From > 1) return fold<From / 2>(x, f);
  else return x;
}

template <class T>
__device__ __forceinline__ T wave_sum(T x) {
  return fold<32>(x, [](T a, T b, auto) { return a + b; });
}
__device__ __forceinline__ float wave_max(float x) {
  return fold<32>(x, [](float a, float b, auto) { return fmaxf(a, b); });
}

__device__ __forceinline__ uint64_t lane_value(uint64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(x), lane), hi = __builtin_amdgcn_readlane(uint32_t(x >> 32), lane);
  return uint64_t(hi) << 32 | lo;
}

template <int Size>
__device__ __forceinline__ uint64_t sorted(uint64_t x) {
  const int lane = threadIdx.x & 63;
  if constexpr (Size > 2) x = sorted<Size / 2>(x);
  return fold<Size / 2>(x, [&](uint64_t a, uint64_t b, auto d) {
    const bool small = ((lane & Size) == 0) == ((lane & decltype(d)::value) == 0);
    return (a < b) == small ? a : b;
  });
}

// list: 64 candidates, the best in lane 0; takes in 64 more in any order: these are sorted the other way round, so
// that lane by lane the better of the two are the best 64 of all, up and down once, which six steps put in order.
__device__ __forceinline__ uint64_t absorb(uint64_t list, uint64_t x) {
  const int lane = threadIdx.x & 63;
  x = sorted<64>(x);
  x = x > list ? x : list;
  return fold<32>(x, [&](uint64_t a, uint64_t b, auto d) {
    return (a < b) == ((lane & decltype(d)::value) != 0) ? a : b;
  });
}

// Lanes of a wave hand candidates to each other through LDS: what was written before is read after.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave's best `keep` candidates of what it has seen.
struct Best {
  uint64_t list = 0;                        // a lane each, the best in lane 0
  uint64_t least = 0;                       // the keep-th of the list
  float floor = -FLT_MAX;                   // no logit below it can enter
  int waiting = 0;                          // candidates set aside in the buffer

  __device__ __forceinline__ void take_in(uint64_t* buffer, int keep) {
    const int lane = threadIdx.x & 63;
    wave_fence();
    const int all = waiting + __popcll(__ballot(list != 0));
    if (all <= 64) {
      // few, as almost always: each one's place is the number of better ones (no two are alike).  20 clocks a
      // candidate, where the sort of 64 takes 3000 with its code fetched
      if (list) buffer[waiting + lane] = list;
      wave_fence();
      const uint64_t x = lane < all ? buffer[lane] : 0;
      int place = 0;
      for (int i = 0; i < all; ++i) place += lane_value(x, i) > x;
      if (lane < all) buffer[place] = x;
      wave_fence();
      list = lane < min(all, keep) ? buffer[lane] : 0;
      waiting = 0;
    }
    while (waiting > 0) {
      const int n = min(waiting, 64);
      waiting -= n;
      list = absorb(list, lane < n ? buffer[waiting + lane] : 0);
      if (lane >= keep) list = 0;
    }
    least = lane_value(list, keep - 1);
    if (least) floor = unordered(uint32_t(least >> 32));
    wave_fence();                           // read before the next ones are written
  }
};

// A bound that the keys of at least `keep` lanes reach (0 where not so many have one): the keep-th largest of them to
// 16 bits, a float's sign, exponent and seven more.
__device__ __forceinline__ uint32_t bound_of(uint32_t key, int keep) {
  uint32_t bound = 0;
#pragma unroll
  for (int bit = 31; bit >= 16; --bit)
    if (__popcll(__ballot(key >= (bound | 1u << bit))) >= keep) bound |= 1u << bit;
  return bound;
}

template <int DT>
struct Elements;
template <>
struct Elements<MX_F32> {
  static constexpr int kVec = 4;
  using Type = float;
  static __device__ __forceinline__ float at(const Words& v, int j) {
    return __uint_as_float(v[j]);
  }
  static __device__ __forceinline__ float one(float x) { return x; }
  static constexpr uint32_t kNone = 0xFF800000u;
};
template <>
struct Elements<MX_BF16> {
  static constexpr int kVec = 8;
  using Type = uint16_t;
  static __device__ __forceinline__ float at(const Words& v, int j) {
    const uint32_t w = v[j / 2];
    return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ float one(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
  static constexpr uint32_t kNone = 0xFF80FF80u;
};
template <>
struct Elements<MX_F16> {
  static constexpr int kVec = 8;
  using Type = uint16_t;
  static __device__ __forceinline__ float one(uint16_t x) {
    return float(__builtin_bit_cast(_Float16, x));
  }
  static __device__ __forceinline__ float at(const Words& v, int j) {
    const uint32_t w = v[j / 2];
    return one(uint16_t(j & 1 ? w >> 16 : w & 0xFFFFu));
  }
  static constexpr uint32_t kNone = 0xFC00FC00u;
};

// A beam that can be continued.
__device__ __forceinline__ bool live(const BeamArgs& g, int64_t row) {
  return !(g.finished && g.finished[row]) && isfinite(g.scores[row]);
}

constexpr float kLog2e = 1.44269504088896340736f;

// A wave for each segment of each beam's logits.  Eight loads of 16 bytes a lane are in flight, past the caches (which
// spares 8%); a chunk's maximum moves each lane's own reference before its exponentials are added, in 32 bits within a
// chunk and in 64 across chunks.  The first chunk's keep-th largest lane maximum is a bound that at least keep logits
// reach: those that reach it, some more than keep, are set aside and sorted.  2048 rows of 131072 BF16 logits take 100 us
// at best and 108 to 112 on average over 30 calls, 5.4 and 4.8 to 5.0 TB/s, as a copy does, with the vector unit busy 74% of
// the time.  Tried: each granule's registers reloaded for the next chunk as soon as it is worked off, 128 us: the compiler
// waits for all of them at the loop's head.
template <int DT, int kLoads>
__global__ __launch_bounds__(256) void beam_scan_kernel(const BeamArgs g) {
  using E = Elements<DT>;
  using T = typename E::Type;
  constexpr int kVec = E::kVec, kChunk = 64 * kVec * kLoads;
  __shared__ uint64_t buffers[4][kBuffer];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t* buffer = buffers[wave];
  const int64_t id = (g.first + blockIdx.x) * 4 + wave;
  const int64_t row = id / g.splits;
  const int split = int(id - row * g.splits);
  if (row >= g.rows || !live(g, row)) return;
  const int64_t request = row / g.beams;
  const T* x = static_cast<const T*>(g.x) + request * g.request_stride + (row - request * g.beams) * g.beam_stride;
  const int begin = int(split * g.segment), end = int(min(int64_t(g.vocab), (split + 1) * g.segment));
  Best best;
  float m = -FLT_MAX;
  double s = 0.0;
  for (int at = begin; at < end; at += kChunk) {
    Words v[kLoads];
    float odd = -INFINITY;                  // of the elements behind the last whole 16 bytes, a lane has one
    const int whole = end - (end - begin) % kVec;          // only a row's last segment has others
    if (at + kChunk <= whole) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) v[u] = __builtin_nontemporal_load(reinterpret_cast<const Words*>(x + at + (u * 64 + lane) * kVec));
    } else {
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        v[u] = Words{E::kNone, E::kNone, E::kNone, E::kNone};
        const int i = at + (u * 64 + lane) * kVec;
        if (i < whole) v[u] = __builtin_nontemporal_load(reinterpret_cast<const Words*>(x + i));
      }
      if (whole + lane < end && at + kChunk >= whole) odd = E::one(x[whole + lane]);
    }
    float top = odd;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
#pragma unroll
      for (int j = 0; j < kVec; ++j) top = fmaxf(top, E::at(v[u], j));
    if (top > m) {
      s *= double(__builtin_amdgcn_exp2f((m - top) * kLog2e));
      m = top;
    }
    float sum = __builtin_amdgcn_exp2f((odd - m) * kLog2e);
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) part += __builtin_amdgcn_exp2f((E::at(v[u], j) - m) * kLog2e);
      sum += part;
    }
    s += double(sum);
    if (at == begin) {
      const uint32_t bound = bound_of(ordered(top + 0.0f), g.keep);
      best.floor = bound ? fmaxf(unordered(bound), -FLT_MAX) : -FLT_MAX;
      // bit patterns of NaN order above all numbers; the row is then passed over whatever is kept
      if (!(best.floor <= FLT_MAX)) best.floor = FLT_MAX;
    }
    if (__ballot(top >= best.floor) == 0) continue;
    const int before = best.waiting;
    {
      auto set_aside = [&](float y, uint32_t token) {
        const bool hit = y >= best.floor;
        const uint64_t mask = __ballot(hit);
        if (mask == 0) return;
        const int to = best.waiting + __popcll(mask & ((uint64_t(1) << lane) - 1));
        if (hit && to < kBuffer) buffer[to] = candidate(y, token);
        best.waiting += __popcll(mask);
      };
      set_aside(odd, uint32_t(whole + lane));
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
#pragma unroll
        for (int j = 0; j < kVec; ++j) set_aside(E::at(v[u], j), uint32_t(at + (u * 64 + lane) * kVec + j));
    }
    if (best.waiting > kBuffer) {
      // very many equal logits: 64 at a time in the order of the tokens, so that the list soon holds the lowest
      best.waiting = before;
      best.take_in(buffer, g.keep);
      for (int i = at; i < min(end, at + kChunk); i += 64) {
        const uint64_t c = i + lane < end && i + lane < at + kChunk ? candidate(E::one(x[i + lane]), uint32_t(i + lane)) : 0;
        const bool hit = c > best.least && c >= uint64_t(ordered(-FLT_MAX)) << 32;
        const uint64_t mask = __ballot(hit);
        if (mask == 0) continue;
        if (hit) buffer[best.waiting + __popcll(mask & ((uint64_t(1) << lane) - 1))] = c;
        best.waiting += __popcll(mask);
        if (best.waiting >= 64) best.take_in(buffer, g.keep);
      }
    } else if (best.waiting >= 64) {
      best.take_in(buffer, g.keep);
    }
  }
  best.take_in(buffer, g.keep);
  const float all = wave_max(m);
  s = wave_sum(s * double(__builtin_amdgcn_exp2f((m - all) * kLog2e)));
  if (lane == 0) g.parts[id] = {s, all, 0};
  if (lane < g.keep) g.best[id * g.keep + lane] = best.list;
}

// A workgroup for each request, several where long histories are copied (each takes the same decision and copies
// some of the columns).  A wave for each beam joins its segments; then each candidate counts those better than it.
// One request of four beams takes 5.6 us, nearly all of it latency: 1.7 for what the first launch left in other XCDs' caches,
// 1 for a beam's best, 1 for the choice, 1 to 2 for a history; 256 requests of eight beams with histories of 2048
// tokens (33 MB read and written) 12 to 13.  One candidate chosen after the other, by a wave, took 700 clocks each.
// kMany: of more than 128 candidates only those are compared that reach a bound, and 16 waves share the beams: 4
// requests of 16 beams, 32 to be chosen, take 25 us (39 with eight waves that compare all), where one request of four
// beams would take 6.6.  The segments' lists come in order; that order is not used, and of more than 64 candidates that
// reach the bound each 64 are sorted again.
template <int kWaves, bool kMany>
__global__ __launch_bounds__(64 * kWaves) void beam_merge_kernel(const BeamArgs g) {
  __shared__ uint64_t buffers[kWaves][kBuffer];
  extern __shared__ double score[];         // [beams][keep], and the tokens behind them
  uint32_t* token = reinterpret_cast<uint32_t*>(score + g.beams * g.keep);
  __shared__ int passed[32];                // of each bit of a bound: how many reach it; 0: candidates that reach the bound
  __shared__ int chosen_beam[kMostWidth];
  __shared__ int chosen_token[kMostWidth];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int request = blockIdx.x;
  const int64_t row0 = int64_t(request) * g.beams;
  __shared__ int length[kMostBeams];
  __shared__ bool was[kMostBeams];
  if (kMany && threadIdx.x < 32) passed[threadIdx.x] = 0;
  // all that does not depend on the choice is read before it
  if (int(threadIdx.x) < g.beams) {
    const int n = g.lens ? g.lens[row0 + threadIdx.x] : 0;
    was[threadIdx.x] = g.finished && g.finished[row0 + threadIdx.x];
    length[threadIdx.x] = min(max(n, 0), g.cols);
  }
  for (int b = wave; b < g.beams; b += kWaves) {
    const int64_t row = row0 + b;
    const float before = g.scores[row];
    const bool done = g.finished && g.finished[row];
    // (of a beam without a scan, what the workspace holds is read and not used)
    const int count = g.splits * g.keep;
    const uint64_t* from = g.best + row * count;
    uint64_t c[kBuffer / 64];
    auto load = [&](int i) {
#pragma unroll
      for (int u = 0; u < kBuffer / 64; ++u) c[u] = from[min(i + u * 64 + lane, count - 1)];
#pragma unroll
      for (int u = 0; u < kBuffer / 64; ++u) c[u] = i + u * 64 + lane < count ? c[u] : 0;
    };
    load(0);
    Part p = g.parts[row * g.splits + min(lane, g.splits - 1)];
    // without this the loads move down to where each value is needed, one behind the other
#pragma unroll
    for (int u = 0; u < kBuffer / 64; ++u) asm volatile("" : "+v"(c[u]));
    if (lane >= g.splits) p = {0.0, -FLT_MAX, 0};
    double mine = -INFINITY;
    uint32_t v = 0;
    if (isfinite(before) && !done) {
      Best best;
      const float all = wave_max(p.m);
      const double s = wave_sum(p.s * double(__builtin_amdgcn_exp2f((p.m - all) * kLog2e)));
      const double log_s = log(s);            // apart from the maximum, beside which it could vanish
      for (int i = 0; i < count; i += kBuffer) {
        if (i) load(i);
        if (i == 0 && count > 64) {
          // as in the scan, a bound that keep lanes reach
          uint32_t key = 0;
#pragma unroll
          for (int u = 0; u < kBuffer / 64; ++u) key = max(key, uint32_t(c[u] >> 32));
          best.least = uint64_t(bound_of(key, g.keep)) << 32;
        }
#pragma unroll
        for (int u = 0; u < kBuffer / 64; ++u) {
          if (i + u * 64 >= count) break;
          const bool hit = c[u] && c[u] >= best.least;
          const uint64_t mask = __ballot(hit);
          if (hit) buffers[wave][best.waiting + __popcll(mask & ((uint64_t(1) << lane) - 1))] = c[u];
          best.waiting += __popcll(mask);
        }
        best.take_in(buffers[wave], g.keep);
      }
      const uint64_t list = best.list;
      // a row with NaN or +inf, or without a finite logit, has no candidates
      if (list && isfinite(log_s) && isfinite(all)) {
        mine = double(before) + ((double(unordered(uint32_t(list >> 32))) - double(all)) - log_s);
        v = ~uint32_t(list);
      }
    } else if (isfinite(before) && lane == 0) {
      mine = before;                        // finished: itself
      v = uint32_t(g.pad);
    }
    if (lane < g.keep) {
      score[b * g.keep + lane] = mine;
      token[b * g.keep + lane] = v;
    }
  }
  __syncthreads();
  auto choose = [&](int place, int beam, double z, int t) {
    chosen_beam[place] = beam;
    chosen_token[place] = t;
    if (blockIdx.y == 0) g.scores_out[int64_t(request) * g.width + place] = float(z);
  };
  // A candidate's place is the number of better ones: a higher score, or the same and a lower beam, or a better logit of
  // the same beam.
  constexpr int step = 64 * kWaves;
  const int candidates = g.beams * g.keep, me = threadIdx.x;
  double* good = reinterpret_cast<double*>(&buffers[0][0]);
  int* which = reinterpret_cast<int*>(good + kGood);
  if constexpr (kMany) {
    // only those that reach a bound which at least width do: the width-th largest score to 20 bits
    constexpr int kEach = kMostBeams * kMostWidth / step;
    uint32_t key[kEach], bound = 0;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int i = u * step + me;
      // (+ 0: a score of -0, which a finished beam can have, equals one of 0)
      key[u] = i < candidates && score[i] > -INFINITY ? ordered(float(score[i]) + 0.0f) : 0;
    }
    for (int bit = 31; bit >= 12; --bit) {
      const uint32_t next = bound | 1u << bit;
      int n = 0;
#pragma unroll
      for (int u = 0; u < kEach; ++u)
        if (u * step < candidates) n += __popcll(__ballot(key[u] >= next));
      if (lane == 0 && n) atomicAdd(&passed[bit], n);
      __syncthreads();
      if (passed[bit] >= g.width) bound = next;
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      if (key[u] == 0 || key[u] < bound) continue;
      const int to = atomicAdd(&passed[0], 1);             // in any order: their places do not depend on it
      if (to < kGood) {
        good[to] = score[u * step + me];
        which[to] = u * step + me;
      }
    }
    __syncthreads();
  }
  if constexpr (!kMany) {
    const double mine = me < candidates ? score[me] : -INFINITY;
    int place = 0;
    if (wave * 64 < candidates) {
#pragma unroll 8
      for (int i = 0; i < candidates; ++i) {
        const double other = score[i];
        place += other > mine || (other == mine && i < me);
      }
    }
    if (mine > -INFINITY && place < g.width) choose(place, me / g.keep, mine, int(token[me]));
    const int real = __syncthreads_count(mine > -INFINITY);
    if (me >= real && me < g.width) choose(me, -1, -INFINITY, g.pad);
  } else if (passed[0] <= kGood) {
    const int some = passed[0];
    if (me < some) {
      const double mine = good[me];
      const int at = which[me];
      int place = 0;
#pragma unroll 8
      for (int i = 0; i < some; ++i) {
        const double other = good[i];
        place += other > mine || (other == mine && which[i] < at);
      }
      if (place < g.width) choose(place, at / g.keep, mine, int(token[at]));
    }
    if (me >= some && me < g.width) choose(me, -1, -INFINITY, g.pad);
  } else if (wave == 0) {
    // very many that are nearly alike: one after the other, lane b with the best candidate of beam b that is left
    int at = 0;
    double head = lane < g.beams ? score[lane * g.keep] : -INFINITY;
    for (int j = 0; j < g.width; ++j) {
      const double top = fold<32>(head, [](double a, double b, auto) { return fmax(a, b); });
      const int from = __ffsll(__ballot(head == top)) - 1;          // of equal ones the lower beam
      if (lane != from) continue;
      if (top > -INFINITY) {
        choose(j, lane, top, int(token[lane * g.keep + at]));
        ++at;
        head = at < g.keep ? score[lane * g.keep + at] : -INFINITY;
      } else {
        choose(j, -1, top, g.pad);
      }
    }
  }
  __syncthreads();
  if (blockIdx.y == 0 && int(threadIdx.x) < g.width) {
    const int j = threadIdx.x, b = chosen_beam[j], v = chosen_token[j];
    const int64_t row = row0 + max(b, 0), o = int64_t(request) * g.width + j;
    const bool stays = b < 0 || was[b];
    g.parents[o] = int32_t(row);
    g.tokens[o] = v;
    g.finished_out[o] = b >= 0 && (was[b] || v == g.eos);
    if (g.lens) {
      const int n = length[max(b, 0)];
      g.lens_out[o] = stays || n == g.cols ? n : n + 1;
    }
  }
  if (!g.history || g.cols == 0) return;
  for (int j = wave; j < g.width; j += kWaves) {
    const int b = chosen_beam[j];
    const int64_t row = row0 + max(b, 0);
    const int32_t* from = g.history + row * g.cols;
    int32_t* to = g.history_out + (int64_t(request) * g.width + j) * g.cols;
    const bool grows = b >= 0 && !was[b];
    const int n = length[max(b, 0)], t = chosen_token[j];
    // 16 bytes at once where rows start on such borders, eight of them in flight
    const int vectors = g.vector ? g.cols / 4 : 0;
    for (int i = blockIdx.y * 512; i < vectors; i += gridDim.y * 512) {
      Vector v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = reinterpret_cast<const Vector*>(from)[min(i + u * 64 + lane, vectors - 1)];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = i + u * 64 + lane;
        if (at >= vectors) continue;
        if (grows && n / 4 == at) {
          v[u].x = n % 4 == 0 ? t : v[u].x;
          v[u].y = n % 4 == 1 ? t : v[u].y;
          v[u].z = n % 4 == 2 ? t : v[u].z;
          v[u].w = n % 4 == 3 ? t : v[u].w;
        }
        reinterpret_cast<Vector*>(to)[at] = v[u];
      }
    }
    for (int64_t i = int64_t(vectors) * 4 + blockIdx.y * 64 + lane; i < g.cols; i += gridDim.y * 64) to[i] = grows && i == n ? t : from[i];
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// Segments of a beam's logits: enough waves for eight on every SIMD, but of at least 4096 logits where that leaves one
// for every SIMD, else of 1024: the bound, the sorts and the sums at the end of a segment cost a wave as much as some
// thousand logits, and the second launch reads what each leaves.  (32 x 4 beams of 50001 F16 logits, both launches: 9.7 +
// 6.8 us with segments of 4096, 9.0 + 7.4 with 2048, 11.3 + 9.8 with 1024; 2048 rows of 131072 BF16 logits, the first
// launch: 108 us with eight waves on a SIMD, 111 with four.)
mx_status_t plan(BeamArgs& g, mx_dtype_t dtype, int64_t requests, int64_t beams, int64_t vocab, int64_t width) {
  if (dtype != MX_F32 && dtype != MX_BF16 && dtype != MX_F16) return MX_ERR_UNSUPPORTED;
  if (requests < 0 || requests > (int64_t(1) << 20) || beams < 1 || beams > kMostBeams || width < 1 || width > kMostWidth ||
      vocab < 1 || vocab > (int64_t(1) << 30))
    return MX_ERR_SHAPE;
  g.requests = int(requests);
  g.beams = int(beams);
  g.rows = requests * beams;
  g.vocab = int(vocab);
  g.width = int(width);
  g.keep = int(std::min(width, vocab));
  const int64_t cus = std::max<int64_t>(device_cus(), 1), rows = std::max<int64_t>(g.rows, 1);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kMostSplits, 32 * cus / rows));
  const int64_t shortest = rows * ((vocab + 4095) / 4096) >= 4 * cus ? 4096 : 1024;
  const int64_t least = std::max<int64_t>(shortest, (vocab + want - 1) / want);
  g.segment = least <= 1024 ? 1024 : least <= 2048 ? 2048 : (least + 4095) / 4096 * 4096;
  g.splits = int((vocab + g.segment - 1) / g.segment);
  return MX_OK;
}

inline int64_t parts_bytes(const BeamArgs& g) { return g.rows * g.splits * int64_t(sizeof(Part)); }
inline int64_t best_bytes(const BeamArgs& g) { return g.rows * g.splits * g.keep * int64_t(sizeof(uint64_t)); }

}  // namespace mxk

using namespace mxk;

extern "C" mx_status_t mx_beam_select_workspace(int64_t requests, int64_t beams, int64_t vocab, int64_t width,
                                                int64_t* bytes) {
  if (!bytes) return MX_ERR_NULL;
  BeamArgs g = {};
  const mx_status_t st = plan(g, MX_F32, requests, beams, vocab, width);
  if (st != MX_OK) return st;
  *bytes = parts_bytes(g) + best_bytes(g);
  return MX_OK;
}

extern "C" mx_status_t mx_beam_select(const void* logits, mx_dtype_t dtype, int64_t requests, int64_t beams,
                                      int64_t vocab, int64_t request_stride, int64_t beam_stride, const float* scores,
                                      const uint8_t* finished, int64_t width, int64_t eos, int64_t pad,
                                      const int32_t* history, const int32_t* lens, int64_t history_cols,
                                      float* scores_out, int32_t* parents, int32_t* tokens, uint8_t* finished_out,
                                      int32_t* history_out, int32_t* lens_out, void* workspace,
                                      int64_t workspace_bytes, hipStream_t stream) {
  BeamArgs g = {};
  const mx_status_t st = plan(g, dtype, requests, beams, vocab, width);
  if (st != MX_OK) return st;
  if (history_cols < 0 || history_cols > INT32_MAX) return MX_ERR_SHAPE;
  if (eos < INT32_MIN || eos > INT32_MAX || pad < INT32_MIN || pad > INT32_MAX) return MX_ERR_ARG;
  if (requests == 0) return MX_OK;
  if (!logits || !scores || !scores_out || !parents || !tokens || !finished_out) return MX_ERR_NULL;
  const bool with_history = history || lens || history_out || lens_out;
  if (with_history && (!lens || !lens_out || (history_cols && (!history || !history_out)))) return MX_ERR_NULL;
  auto off4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == MX_F32 ? 4 : 2)) return MX_ERR_ALIGN;
  if (off4(scores) || off4(scores_out) || off4(parents) || off4(tokens) || off4(history) || off4(lens) ||
      off4(history_out) || off4(lens_out))
    return MX_ERR_ALIGN;
  if (workspace_bytes < parts_bytes(g) + best_bytes(g)) return MX_ERR_SHAPE;
  if (!workspace) return MX_ERR_NULL;
  if (misaligned(workspace)) return MX_ERR_ALIGN;
  g.x = logits; g.scores = scores; g.finished = finished; g.history = history; g.lens = lens;
  g.scores_out = scores_out; g.parents = parents; g.tokens = tokens; g.finished_out = finished_out;
  g.history_out = history_out; g.lens_out = lens_out;
  g.parts = static_cast<Part*>(workspace);
  g.best = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + parts_bytes(g));
  g.request_stride = request_stride; g.beam_stride = beam_stride;
  g.eos = int(eos); g.pad = int(pad); g.cols = int(history_cols);
  const int64_t all_blocks = (g.rows * g.splits + 3) / 4;
  auto scan = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const int64_t loads = (g.segment + 64 * Elements<DT>::kVec - 1) / (64 * Elements<DT>::kVec);
    const unsigned blocks = unsigned(std::min(kMostBlocks, all_blocks - g.first));
    if (loads <= 2) beam_scan_kernel<DT, 2><<<blocks, 256, 0, stream>>>(g);
    else if (loads <= 4) beam_scan_kernel<DT, 4><<<blocks, 256, 0, stream>>>(g);
    else beam_scan_kernel<DT, 8><<<blocks, 256, 0, stream>>>(g);
  };
  for (; g.first < all_blocks; g.first += kMostBlocks) {
    if (dtype == MX_F32) scan(std::integral_constant<int, MX_F32>{});
    else if (dtype == MX_BF16) scan(std::integral_constant<int, MX_BF16>{});
    else scan(std::integral_constant<int, MX_F16>{});
    // what was not scanned is not merged
    if (hipGetLastError() != hipSuccess) return MX_ERR_LAUNCH;
  }
  g.vector = g.cols % 4 == 0 && !misaligned(history) && !misaligned(history_out);
  // 32 KiB of history a workgroup, up to two of them on a CU
  const int64_t wide = with_history ? g.width * int64_t(g.cols) * 4 / 32768 : 0;
  const int64_t most = std::max<int64_t>(1, 2 * std::max<int64_t>(device_cus(), 1) / requests);
  const unsigned y = unsigned(std::max<int64_t>(1, std::min(wide, most)));
  const dim3 grid(static_cast<unsigned>(requests), y);
  const int64_t candidates = beams * g.keep;
  if (candidates <= kFew) beam_merge_kernel<8, false><<<grid, 512, size_t(candidates) * 12, stream>>>(g);
  else beam_merge_kernel<16, true><<<grid, 1024, size_t(candidates) * 12, stream>>>(g);
  return hipGetLastError() == hipSuccess ? MX_OK : MX_ERR_LAUNCH;
}
