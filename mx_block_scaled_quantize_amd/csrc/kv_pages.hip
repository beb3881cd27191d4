// Pages of the paged MXFP8 key/value cache on gfx950: copied, forked, freed and moved together.
//
// A pool of pages has a count of holders for every page (0: free).  All plans are made on the
// device from the counts and the page table: which pages a sequence keeps, which it gets, and
// what has to be copied.  Pages are dealt by rank (the nth page needed is the nth free one), found
// by counting in blocks and summing the blocks before, so nothing depends on the order in which
// workgroups run; atomics are used for counts only, which any order adds up to the same.
//
// What bounds them: the copies are bound by memory (one read and one write of each page); the plans
// read the counts and the tables once, which takes a few microseconds, and so are bound by the
// chain of launches that their dependent steps need.

#include "mx_launch.hpp"

#include <algorithm>

namespace mxk {

constexpr int kLayersPerLaunch = 32;        // 4 pointers each: 1 KiB of a launch's arguments
constexpr int kPartLoads = 8;               // 16-byte granules that a lane copies at once
constexpr int kPartGranules = 64 * kPartLoads;
constexpr int kPerThread = 16;              // counts that a thread of a counting block reads
constexpr int kCountBlock = 256 * kPerThread;
constexpr int kMostCountBlocks = 4096;      // every block sums the blocks before it: 16 loads a thread

struct Layers {
  uint8_t* p[kLayersPerLaunch][4];          // k, k_scales, v, v_scales
};

typedef uint32_t Granule __attribute__((ext_vector_type(4)));

struct PageShape {
  int kv_heads, page, dim;
};

// n / d for quotients below 2^51, with inv = 1.0 / d: the product is off by less than one, which one step mends.
__device__ __forceinline__ int64_t divide(int64_t n, int64_t d, double inv, int64_t& rest) {
  int64_t q = int64_t(double(n) * inv);
  rest = n - q * d;
  if (rest < 0) { --q; rest += d; }
  if (rest >= d) { ++q; rest -= d; }
  return q;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// ---------------------------------------------------------------------------
// Copies
// ---------------------------------------------------------------------------
// A wave copies part `part` of the first `tokens` tokens (a multiple of 16) of page src to page dst: 8 KiB of the
// keys, the values, the key scales and the value scales in a row.  Eight loads of 16 bytes a lane are in flight
// before the first store, past the caches, as no part is read twice.  A whole page is one run of bytes in each array;
// of a part of one, each head is a run.  Measured on 1.1 GB read and written: 205 to 213 us (5.2 to 5.4 TB/s); with four loads
// 213, through the caches 227, with 2048 instead of up to 16384 workgroups 216; 300 with an address worked out for each
// 16 bytes, as now only in parts that are not of one array.
__device__ __forceinline__ void copy_part(uint8_t* const (&from)[4], uint8_t* const (&to)[4], const PageShape& s,
                                          int64_t src, int64_t dst, int tokens, uint32_t part) {
  const bool whole = tokens == s.page;
  const uint32_t heads = whole ? 1u : uint32_t(s.kv_heads);
  const uint32_t head_codes = (whole ? uint32_t(s.kv_heads) * uint32_t(s.page) : uint32_t(tokens)) * uint32_t(s.dim) / 16u;
  const uint32_t head_scales = head_codes / 32u, codes = heads * head_codes, scales = heads * head_scales;
  const int64_t page_codes = int64_t(s.kv_heads) * s.page * s.dim;
  const uint32_t lane = threadIdx.x & 63u;
  const uint32_t first = part * kPartGranules, last = first + kPartGranules - 1;
  Granule v[kPartLoads];
  if (whole && last < 2u * codes && (last < codes || first >= codes)) {
    const bool is_value = first >= codes;
    const int64_t off = int64_t(first - (is_value ? codes : 0u)) * 16;
    const Granule* f = reinterpret_cast<const Granule*>((is_value ? from[2] : from[0]) + src * page_codes + off) + lane;
    Granule* t = reinterpret_cast<Granule*>((is_value ? to[2] : to[0]) + dst * page_codes + off) + lane;
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) v[i] = __builtin_nontemporal_load(f + i * 64);
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) __builtin_nontemporal_store(v[i], t + i * 64);
    return;
  }
  // four at a time: 256 registers for eight of them and their addresses
  uint8_t* const from0 = from[0];
  uint8_t* const from1 = from[1];
  uint8_t* const from2 = from[2];
  uint8_t* const from3 = from[3];
  uint8_t* const to0 = to[0];
  uint8_t* const to1 = to[1];
  uint8_t* const to2 = to[2];
  uint8_t* const to3 = to[3];
#pragma unroll 1
  for (int half = 0; half < kPartLoads; half += 4) {
    if (first + half * 64 >= 2u * (codes + scales)) break;
    uint8_t* at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t g = first + (half + i) * 64 + lane;
      const bool is_scale = g >= 2u * codes;
      uint32_t o = is_scale ? g - 2u * codes : g;
      const uint32_t n = is_scale ? scales : codes, run = is_scale ? head_scales : head_codes;
      const bool is_value = o >= n;
      o -= is_value ? n : 0u;
      const int64_t page_bytes = is_scale ? page_codes / 32 : page_codes;
      int64_t off = int64_t(o) * 16;
      if (!whole) {
        const uint32_t head = o / run;
        off = int64_t(head) * (int64_t(s.page) * s.dim / (is_scale ? 32 : 1)) + int64_t(o - head * run) * 16;
      }
      const uint8_t* f = is_scale ? (is_value ? from3 : from1) : (is_value ? from2 : from0);
      uint8_t* t = is_scale ? (is_value ? to3 : to1) : (is_value ? to2 : to0);
      const bool real = g < 2u * (codes + scales);
      v[i] = Granule{};
      if (real) v[i] = __builtin_nontemporal_load(reinterpret_cast<const Granule*>(f + src * page_bytes + off));
      at[i] = real ? t + dst * page_bytes + off : nullptr;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at[i]) __builtin_nontemporal_store(v[i], reinterpret_cast<Granule*>(at[i]));
  }
}

struct Item {
  int64_t copy;
  int layer;
  uint32_t part;
};

// Items of work of a launch: (copy, layer, part), the parts of a page in a row.
struct Items {
  int layers, parts;
  double inv_layers, inv_parts;
  __device__ __forceinline__ Item at(int64_t i) const {
    int64_t part, layer;
    const int64_t unit = divide(i, parts, inv_parts, part);
    const int64_t copy = divide(unit, layers, inv_layers, layer);
    return {copy, int(layer), uint32_t(part)};
  }
};

struct CopyArgs {
  Layers from, to;
  const int32_t *src, *dst;
  int64_t count, src_pages, dst_pages;
  PageShape shape;
  Items items;
};

__global__ __launch_bounds__(256) void page_copy_kernel(const CopyArgs g) {
  const int64_t waves = int64_t(gridDim.x) * 4;
  const int64_t total = g.count * g.items.layers * g.items.parts;
  for (int64_t i = int64_t(blockIdx.x) * 4 + uniform(threadIdx.x >> 6); i < total; i += waves) {
    const Item it = g.items.at(i);
    const int32_t src = g.src[it.copy], dst = g.dst[it.copy];
    if (src < 0 || src >= g.src_pages || dst < 0 || dst >= g.dst_pages) continue;
    const int layer = uniform(it.layer);
    copy_part(g.from.p[layer], g.to.p[layer], g.shape, src, dst, g.shape.page, it.part);
  }
}

// ---------------------------------------------------------------------------
// Sums over a workgroup
// ---------------------------------------------------------------------------
// x of a lane some way before this one, 0 where there is none: by moves inside the vector unit.
template <int Ctrl, int Rows>
__device__ __forceinline__ int32_t before_lane(int32_t x) { return __builtin_amdgcn_update_dpp(0, x, Ctrl, Rows, 0xF, false); }
template <int Ctrl, int Rows>
__device__ __forceinline__ int64_t before_lane(int64_t x) {
  const uint32_t lo = before_lane<Ctrl, Rows>(int32_t(x)), hi = before_lane<Ctrl, Rows>(int32_t(x >> 32));
  return int64_t(uint64_t(hi) << 32 | lo);
}

// Sum of x over the lanes up to this one: within each sixteen lanes, then the last lanes of sixteens, of halves.
template <class T>
__device__ __forceinline__ T wave_scan(T x) {
  x += before_lane<0x111, 0xF>(x);
  x += before_lane<0x112, 0xF>(x);
  x += before_lane<0x114, 0xF>(x);
  x += before_lane<0x118, 0xF>(x);
  x += before_lane<0x142, 0xA>(x);
  x += before_lane<0x143, 0xC>(x);
  return x;
}

// Sum of x over the threads before this one, and over all of them, in a workgroup of W waves.
template <int W = 4, class T>
__device__ __forceinline__ T block_scan(T x, T& total) {
  __shared__ T part[W];
  const T mine = wave_scan(x);
  const int w = threadIdx.x >> 6;
  __syncthreads();                          // the last call's sums are read
  if ((threadIdx.x & 63u) == 63u) part[w] = mine;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < w) before += part[i];
    total += part[i];
  }
  return before + mine - x;
}

// Sum of the first `before` and of all `count` entries.
template <class T, class U>
__device__ __forceinline__ T sum_before(const U* a, int count, int before, T& total) {
  T x = 0, y = 0;
  for (int i = threadIdx.x; i < count; i += 256) {
    const T v = T(a[i]);
    y += v;
    if (i < before) x += v;
  }
  T sum;
  block_scan(x, sum);
  block_scan(y, total);
  return sum;
}

// Counting blocks: block b has the pages [b, b + 1) * per_block.
struct Blocks {
  int64_t pages, per_block;                 // per_block a multiple of kCountBlock
  int count;
  __device__ __forceinline__ int64_t begin(int b) const { return int64_t(b) * per_block; }
  __device__ __forceinline__ int64_t end(int b) const { return min(pages, int64_t(b + 1) * per_block); }
};

// Keeps loads where they are asked for: without it they move down to where each value is first needed, and each waits.
template <int N>
__device__ __forceinline__ void hold(int32_t (&r)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+v"(r[k]));
}

// A run: 1024 pages in a row of a wave, lane l with those at 64 k + l (so that loads and stores are of whole lines, and
// a ballot counts 64 pages).  Pages behind the pool read as `other`.
struct Run {
  uint32_t at;                              // below 2^31 + 2^14
  int32_t r[kPerThread];
  __device__ __forceinline__ void load(const int32_t* refs, int64_t first, int64_t pages, int32_t other) {
    at = uint32_t(first) + (threadIdx.x >> 6) * (64 * kPerThread) + (threadIdx.x & 63u);
    if (pages == 0) {
#pragma unroll
      for (int k = 0; k < kPerThread; ++k) r[k] = other;
      return;
    }
    // without a condition on a lane, so that all sixteen are in flight
    const uint32_t wave_at = uint32_t(uniform(int(at)));
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      r[k] = other;
      if (wave_at + 64 * k < pages) r[k] = refs[min(int64_t(at + 64 * k), pages - 1)];
    }
    hold(r);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) r[k] = at + 64 * k < pages ? r[k] : other;
  }
  template <class P>
  __device__ __forceinline__ int count(P p) const {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) n += __popcll(__ballot(p(r[k])));
    return n;
  }
  // Calls f(k, page, how many pages before it p holds for), with `before` of them before this wave's run.
  template <class P, class F>
  __device__ __forceinline__ void each(int before, P p, F f) const {
    const uint64_t below = (uint64_t(1) << (threadIdx.x & 63u)) - 1;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const uint64_t mask = __ballot(p(r[k]));
      f(k, at + 64 * k, before + __popcll(mask & below));
      before += __popcll(mask);
    }
  }
};

__device__ __forceinline__ bool is_free(int32_t n) { return n == 0; }
__device__ __forceinline__ bool is_used(int32_t n) { return n != 0; }

// Sum of the waves' counts before this wave's, and of all.
template <int W>
__device__ __forceinline__ int waves_before(int n, int& total) {
  __shared__ int part[W];
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63u) == 0) part[w] = n;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < w) before += part[i];
    total += part[i];
  }
  return before;
}

// ---------------------------------------------------------------------------
// Forking
// ---------------------------------------------------------------------------
struct ForkArgs {
  Layers caches;
  const int32_t *refs, *table, *lens, *parents, *cu;
  int32_t *refs_out, *table_out, *lens_out;
  int64_t* slots;
  int64_t pages, stride, rows, children, tokens, capacity;
  int cols, out_cols, release;
  PageShape shape;
  Items items;
  Blocks blocks;
  int child_blocks;
  // workspace
  int64_t *start, *child_sum;               // first new page of a child (-1: it gets none); pages that a block of children needs
  int32_t *kids, *writers, *first;          // of each row: children, those that write into its last page, the first of these
  int32_t *info;                            // of each child: 2 * new pages + whether the first is a copy; -1: too many for a row
  int32_t *child_copies, *block_free, *list, *copies;
  int4* copy;                               // source page (-1: none), place of the new page in the list, tokens
};

struct Child {
  int64_t row;                              // -1: starts empty
  int had, fresh, from;                     // cached tokens, new tokens, the first one's number
  int held, partly;                         // pages, and tokens in the last one if it is partly filled
};

__device__ __forceinline__ int row_length(const ForkArgs& g, int64_t row) {
  return min(max(g.lens[row], 0), g.cols * g.shape.page);
}

// The child of row `row` (-1: none) of length `had`, with new tokens from lo up to hi.
__device__ __forceinline__ Child child_of(const ForkArgs& g, int64_t row, int had, int64_t lo, int64_t hi) {
  Child c;
  c.row = row;
  c.had = had;
  lo = min(max(lo, int64_t(0)), g.tokens);
  c.from = int(lo);
  c.fresh = int(min(max(hi, lo), g.tokens) - lo);
  c.held = (c.had + g.shape.page - 1) / g.shape.page;
  c.partly = c.had % g.shape.page;
  return c;
}

__device__ __forceinline__ Child child_of(const ForkArgs& g, int64_t i) {
  int64_t row = g.parents ? int64_t(g.parents[i]) : i;
  if (row < 0 || row >= g.rows) row = -1;
  return child_of(g, row, row < 0 ? 0 : row_length(g, row), g.cu ? g.cu[i] : 0, g.cu ? g.cu[i + 1] : 0);
}

__device__ __forceinline__ bool in_pool(const ForkArgs& g, int32_t page) { return page >= 0 && page < g.pages; }

// The rows' children, counted in LDS by the first workgroup, while the others copy the counts of pages (64 x 4 beams over
// 15000 pages: 2.7 us against 2.2 + 2.5 in two launches).
constexpr int kBeginRows = 4096, kBeginChildren = 16384;

__global__ __launch_bounds__(1024) void fork_begin_kernel(const ForkArgs g) {
  __shared__ int32_t kids[kBeginRows], writers[kBeginRows], first[kBeginRows];
  if (blockIdx.x > 0) {
    const int64_t step = int64_t(gridDim.x - 1) * 1024;
    for (int64_t i = int64_t(blockIdx.x - 1) * 1024 + threadIdx.x; i < g.pages; i += step) g.refs_out[i] = g.refs[i];
    return;
  }
  for (int i = threadIdx.x; i < g.rows; i += 1024) {
    kids[i] = writers[i] = 0;
    first[i] = INT32_MAX;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g.children; i += 1024) {
    const Child c = child_of(g, i);
    if (c.row < 0) continue;
    atomicAdd(&kids[c.row], 1);
    if (c.fresh && c.partly) {
      atomicAdd(&writers[c.row], 1);
      atomicMin(&first[c.row], i);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g.rows; i += 1024) {
    g.kids[i] = kids[i];
    g.writers[i] = writers[i];
    g.first[i] = first[i];
  }
}

// The same where there are more rows or children, in two launches.
__global__ __launch_bounds__(256) void fork_init_kernel(const ForkArgs g) {
  const int64_t step = int64_t(gridDim.x) * 256;
  const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (g.refs_out != g.refs)
    for (int64_t i = at; i < g.pages; i += step) g.refs_out[i] = g.refs[i];
  for (int64_t i = at; i < g.rows; i += step) {
    g.kids[i] = g.writers[i] = 0;
    g.first[i] = INT32_MAX;
  }
}

__global__ __launch_bounds__(256) void fork_kids_kernel(const ForkArgs g) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= g.children) return;
  const Child c = child_of(g, i);
  if (c.row < 0) return;
  atomicAdd(&g.kids[c.row], 1);
  if (c.fresh && c.partly) {
    atomicAdd(&g.writers[c.row], 1);
    atomicMin(&g.first[c.row], int32_t(i));
  }
}

// Every page of a row gains the row's children and loses the row itself if it is released.  A thread takes one column of
// eight rows: beams of a request lie next to each other and share their first pages, whose gains and losses add up to
// nothing before they would go to memory (256 x 8 beams of some 380 pages: 22.3 -> 8.6 us).
constexpr int kRowGroup = 8;

__global__ __launch_bounds__(256) void fork_counts_kernel(const ForkArgs g) {
  for (int64_t row0 = int64_t(blockIdx.x) * kRowGroup; row0 < g.rows; row0 += int64_t(gridDim.x) * kRowGroup) {
    int32_t d[kRowGroup], held[kRowGroup];
    int most = 0;
#pragma unroll
    for (int u = 0; u < kRowGroup; ++u) {
      const int64_t row = min(row0 + u, g.rows - 1);
      d[u] = g.kids[row];
      held[u] = row_length(g, row);
    }
#pragma unroll
    for (int u = 0; u < kRowGroup; ++u) {
      d[u] = row0 + u < g.rows ? d[u] - g.release : 0;
      held[u] = d[u] == 0 ? 0 : (held[u] + g.shape.page - 1) / g.shape.page;
      most = max(most, held[u]);
    }
    for (int j = blockIdx.y * 256 + threadIdx.x; j < most; j += gridDim.y * 256) {
      int32_t page[kRowGroup];
#pragma unroll
      for (int u = 0; u < kRowGroup; ++u) {
        page[u] = -1;
        if (uniform(held[u]) > 0) page[u] = g.table[(row0 + u) * g.stride + min(j, held[u] - 1)];
      }
      hold(page);
      int32_t last = -1, sum = 0;
#pragma unroll
      for (int u = 0; u < kRowGroup; ++u) {
        if (j >= held[u] || !in_pool(g, page[u])) continue;
        if (page[u] != last) {
          if (sum != 0) atomicAdd(&g.refs_out[last], sum);
          last = page[u];
          sum = 0;
        }
        sum += d[u];
      }
      if (sum != 0) atomicAdd(&g.refs_out[last], sum);
    }
  }
}

// Blocks of children: the pages that each needs; blocks of pages: how many are free.
__global__ __launch_bounds__(256) void fork_needs_kernel(const ForkArgs g) {
  if (int(blockIdx.x) >= g.child_blocks) {
    const int b = blockIdx.x - g.child_blocks;
    int n = 0, total;
    // without parents and with the rows released the counts stay, and are copied here
    const bool copy = !g.parents && g.release && g.refs_out != g.refs;
    for (int64_t at = g.blocks.begin(b); at < g.blocks.end(b); at += kCountBlock) {
      Run run;
      run.load(copy ? g.refs : g.refs_out, at, g.pages, 1);
      n += run.count(is_free);
      if (copy) run.each(0, is_free, [&](int k, uint32_t page, int) { if (page < g.pages) g.refs_out[page] = run.r[k]; });
    }
    waves_before<4>(n, total);
    if (threadIdx.x == 0) g.block_free[b] = total;
    return;
  }
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  int need = 0, info = 0;
  bool copy = false;
  if (i < g.children) {
    const Child c = child_of(g, i);
    const int64_t after = (int64_t(c.had) + c.fresh + g.shape.page - 1) / g.shape.page;
    if (c.fresh && c.partly) {
      const int32_t tail = g.table[c.row * g.stride + c.held - 1];
      if (in_pool(g, tail)) {
        const bool alone = !g.parents && g.release;
        const int32_t count = (alone ? g.refs : g.refs_out)[tail];
        const int32_t writers = alone ? 1 : g.writers[c.row];
        copy = !(count == writers && (alone || g.first[c.row] == i));
      }
    }
    need = int(after) - c.held + copy;
    info = 2 * need + copy;
    if (after > g.out_cols) info = -1, copy = false;        // gets none, and what it needs still counts
    g.info[i] = info;
  }
  int64_t total;
  const int64_t before = block_scan(int64_t(need), total);
  int copies;
  block_scan(int(copy), copies);
  if (i < g.children) g.start[i] = before;
  if (threadIdx.x == 0) {
    g.child_sum[blockIdx.x] = total;
    g.child_copies[blockIdx.x] = copies;
  }
}

// Blocks of children: where each one's new pages begin in the list, or that there are too few, and the copies;
// blocks of pages: the free ones into the list, as many as can be needed.
__global__ __launch_bounds__(256) void fork_list_kernel(const ForkArgs g) {
  if (int(blockIdx.x) >= g.child_blocks) {
    const int b = blockIdx.x - g.child_blocks;
    int all, rank = sum_before<int>(g.block_free, g.blocks.count, b, all);
    if (rank >= g.capacity) return;
    for (int64_t at = g.blocks.begin(b); at < g.blocks.end(b); at += kCountBlock) {
      Run run;
      run.load(g.refs_out, at, g.pages, 1);
      int total;
      const int before = waves_before<4>(run.count(is_free), total);
      run.each(rank + before, is_free, [&](int k, uint32_t page, int nth) {
        if (run.r[k] == 0 && nth < g.capacity) g.list[nth] = int32_t(page);
      });
      rank += total;
    }
    return;
  }
  int64_t all_free, all_needed;
  sum_before<int64_t>(g.block_free, g.blocks.count, 0, all_free);
  const int64_t base = sum_before<int64_t>(g.child_sum, g.child_blocks, blockIdx.x, all_needed);
  int all_copies;
  const int copies = sum_before<int>(g.child_copies, g.child_blocks, blockIdx.x, all_copies);
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int info = i < g.children ? g.info[i] : 0;
  const bool copy = info > 0 && (info & 1);
  int total;
  const int nth = copies + block_scan(int(copy), total);
  if (blockIdx.x == 0 && threadIdx.x == 0) *g.copies = all_copies;
  if (i >= g.children) return;
  const Child c = child_of(g, i);
  const int64_t start = base + g.start[i];
  const int need = info >> 1;
  const bool fits = c.fresh && info >= 0 && (need == 0 || start + need <= min(all_free, g.capacity));
  g.start[i] = fits ? start : -1;
  if (copy) {
    const int32_t tail = g.table[c.row * g.stride + c.held - 1];
    g.copy[nth] = make_int4(fits ? tail : -1, fits ? int(start) : 0, (c.partly + 15) / 16 * 16, 0);
  }
}

// Small pools: one workgroup of 16 waves plans alone, with the counts in LDS, instead of four or five launches behind
// each other: 6.7 us for four beams against 12.9.  Its one CU reads the table, though: 33000 entries take it 20 us,
// the launches 14, so that it takes tables of up to 8192.
constexpr int kSmallPages = 16384, kSmallRows = 1024, kSmallEntries = 8192;

// Entries of a table, eight of a thread at once; read before it is known which of them count.
struct Entries {
  int32_t page[8];
  __device__ __forceinline__ static int row_of(int e, int cols, float inv) {
    int row = int(float(e) * inv);          // off by one at most: e < 2^16
    if (row * cols > e) --row;
    if ((row + 1) * cols <= e) ++row;
    return row;
  }
  __device__ __forceinline__ void load(const int32_t* table, int64_t stride, int base, int entries, int cols, float inv) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      page[u] = -1;
      if (base + u * 1024 + uniform(int(threadIdx.x & ~63u)) >= entries) continue;
      const int e = min(base + u * 1024 + int(threadIdx.x), entries - 1);
      const int row = row_of(e, cols, inv);
      page[u] = table[row * stride + e - row * cols];
    }
    hold(page);
  }
  // Adds weight[r] to the counts of the entries [from[r], to[r]) of every row r.
  __device__ __forceinline__ void add(int32_t* count, int pages, int base, int entries, int cols, float inv,
                                      const int32_t* weight, const int32_t* from, const int32_t* to) const {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int e = base + u * 1024 + int(threadIdx.x);
      if (e >= entries || page[u] < 0 || page[u] >= pages) continue;
      const int row = row_of(e, cols, inv), j = e - row * cols;
      if (weight[row] != 0 && j >= from[row] && j < to[row]) atomicAdd(&count[page[u]], weight[row]);
    }
  }
};

__global__ __launch_bounds__(1024) void fork_small_kernel(const ForkArgs g) {
  __shared__ int32_t count[kSmallPages];
  __shared__ int32_t kids[kSmallRows], zero[kSmallRows], length[kSmallRows], held[kSmallRows], writers[kSmallRows],
      first[kSmallRows];
  const int t = threadIdx.x, pages = int(g.pages), entries = int(g.rows) * g.cols;
  const float inv = g.cols ? 1.0f / float(g.cols) : 0.0f;
  const bool alone = !g.parents && g.release;             // every row goes on: no count changes but by copies
  // all that is read at places known beforehand
  Run run;
  run.load(g.refs, 0, pages, 1);
  Entries some;
  if (!alone && entries) some.load(g.table, g.stride, 0, entries, g.cols, inv);
  const bool is_child = t < g.children;
  int64_t parent = is_child ? g.parents ? int64_t(g.parents[t]) : t : -1;
  if (parent < 0 || parent >= g.rows) parent = -1;
  int64_t lo = 0, hi = 0;
  if (is_child && g.cu) {
    lo = g.cu[t];
    hi = g.cu[t + 1];
  }
  const int mine = t < g.rows ? row_length(g, t) : 0;
  run.each(0, is_free, [&](int k, uint32_t page, int) { count[page] = run.r[k]; });
  kids[t] = g.release ? -1 : 0;
  zero[t] = writers[t] = 0;
  first[t] = INT32_MAX;
  length[t] = mine;
  held[t] = (mine + g.shape.page - 1) / g.shape.page;
  __syncthreads();
  const Child c = child_of(g, parent, parent < 0 ? 0 : length[parent], lo, hi);
  int32_t tail = -1;
  if (c.fresh && c.partly) tail = g.table[c.row * g.stride + c.held - 1];
  if (c.row >= 0) {
    atomicAdd(&kids[c.row], 1);
    if (c.fresh && c.partly) {
      atomicAdd(&writers[c.row], 1);
      atomicMin(&first[c.row], t);
    }
  }
  __syncthreads();
  if (!alone) {
    for (int base = 0; base < entries; base += 8 * 1024) {
      if (base) some.load(g.table, g.stride, base, entries, g.cols, inv);
      some.add(count, pages, base, entries, g.cols, inv, kids, zero, held);
    }
    __syncthreads();
  }
  // pages that each child needs
  const int64_t after = (int64_t(c.had) + c.fresh + g.shape.page - 1) / g.shape.page;
  const bool wide = after > g.out_cols;
  const bool shared = in_pool(g, tail) && !(count[tail] == writers[c.row] && first[c.row] == t);
  const bool copy = shared && !wide;                      // too many for a row: gets none, and what it needs still counts
  const int64_t need = after - c.held + shared;
  int64_t sums;                             // of pages, and of copies in the lowest bits (1024 at most)
  const int64_t both = block_scan<16>(need * 2048 + copy, sums);
  const int64_t start = both >> 11;
  const int nth = int(both & 2047), copies = int(sums & 2047);
  int all_free;
  run.each(0, is_free, [&](int k, uint32_t page, int) { run.r[k] = count[page]; });
  const int before = waves_before<16>(run.count(is_free), all_free);
  run.each(before, is_free, [&](int k, uint32_t page, int rank) {
    if (run.r[k] == 0 && rank < g.capacity) g.list[rank] = int32_t(page);
    if (page < pages && (g.refs_out != g.refs || !alone)) g.refs_out[page] = run.r[k];
  });
  if (t == 0) *g.copies = copies;
  if (!is_child) return;
  const bool fits = c.fresh && !wide && (need == 0 || start + need <= min(int64_t(all_free), g.capacity));
  g.info[t] = int(2 * need + copy);
  g.start[t] = fits ? start : -1;
  if (copy) g.copy[nth] = make_int4(fits ? tail : -1, fits ? int(start) : 0, (c.partly + 15) / 16 * 16, 0);
}

// The partly filled pages, 8 KiB a wave at a time, by workgroup `block` of `blocks`.
__device__ __forceinline__ void copy_tails(const ForkArgs& g, int64_t block, int64_t blocks) {
  const int64_t total = int64_t(*g.copies) * g.items.layers * g.items.parts;
  for (int64_t i = block * 4 + uniform(threadIdx.x >> 6); i < total; i += blocks * 4) {
    const Item it = g.items.at(i);
    const int4 c = g.copy[it.copy];
    if (c.x < 0) continue;
    const int layer = uniform(it.layer);
    copy_part(g.caches.p[layer], g.caches.p[layer], g.shape, c.x, g.list[c.y], uniform(c.z), it.part);
  }
}

// A workgroup for each child writes its row of the table, its slots and the counts of its pages; the workgroups
// behind them copy the partly filled pages.  64 x 4 beams in eight layers, some 80 pages of 34 KB each: 11 us, of which
// the copies' bytes need 9.
__global__ __launch_bounds__(256) void fork_rows_kernel(const ForkArgs g) {
  const int64_t i = blockIdx.x;
  if (i > 0 && i >= g.children) {
    copy_tails(g, i - g.children, int64_t(gridDim.x) - g.children);
    return;
  }
  if (i == 0 && g.tokens) {                 // tokens before the first child and behind the last are padding
    const int64_t lo = g.cu ? min(max(int64_t(g.cu[0]), int64_t(0)), g.tokens) : g.tokens;
    const int64_t hi = g.cu ? min(max(int64_t(g.cu[g.children]), int64_t(0)), g.tokens) : g.tokens;
    for (int64_t t = threadIdx.x; t < lo; t += 256) g.slots[t] = -1;
    for (int64_t t = hi + threadIdx.x; t < g.tokens; t += 256) g.slots[t] = -1;
  }
  if (g.children == 0) return;              // launched for the padding
  const Child c = child_of(g, i);
  const int64_t start = g.start[i];
  const bool fits = start >= 0;
  const int copy = fits ? g.info[i] & 1 : 0;
  const int after = fits ? int((int64_t(c.had) + c.fresh + g.shape.page - 1) / g.shape.page) : c.held;
  const int32_t* row = g.table + c.row * g.stride;        // read up to held, which is 0 without a row
  const int kept = c.held - copy;                          // pages that stay
  int32_t* out = g.table_out + i * g.out_cols;
  for (int j = threadIdx.x; j < g.out_cols; j += 256) {
    int32_t page = -1;
    if (j < kept) {
      page = row[j];
    } else if (j < after) {
      page = g.list[start + j - kept];
      g.refs_out[page] = 1;
    }
    out[j] = page;
  }
  if (threadIdx.x == 0) {
    g.lens_out[i] = c.had + (fits ? c.fresh : 0);
    if (copy) atomicSub(&g.refs_out[row[c.held - 1]], 1);
  }
  for (int64_t t = threadIdx.x; t < c.fresh; t += 256) {
    int64_t slot = -1;
    if (fits) {
      const int at = int(c.had + t), j = at / g.shape.page;
      const int32_t page = j < kept ? row[j] : g.list[start + j - kept];
      if (in_pool(g, page)) slot = int64_t(page) * g.shape.page + at % g.shape.page;
    }
    g.slots[c.from + t] = slot;
  }
}

// Copies of further layers than those of one launch.
__global__ __launch_bounds__(256) void fork_copy_kernel(const ForkArgs g) {
  copy_tails(g, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------------
// Freeing
// ---------------------------------------------------------------------------
struct FreeArgs {
  const int32_t *refs, *table, *lens, *keep;
  int32_t *refs_out, *lens_out;
  int64_t pages, stride, rows;
  int cols, page;
  // many entries: `tiles` tiles of 8192, buckets of 2^shift pages
  int tiles, buckets, shift;
  uint16_t* ends;                           // [tiles][kBuckets + 1]: where a bucket's entries begin in a tile
  int32_t* sorted;                          // [tiles][8192]: pages that lose a hold, bucket after bucket
};

__global__ __launch_bounds__(256) void refs_copy_kernel(const int32_t* from, int32_t* to, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) to[i] = from[i];
}

__device__ __forceinline__ int kept_tokens(const FreeArgs& g, int64_t row, int had) {
  return min(had, g.keep ? max(g.keep[row], 0) : 0);
}

// A workgroup for a row, or for some of its entries.  It is bound by the atomics where the pages of a row lie anywhere:
// they are worked off behind the L2s, 22 a nanosecond; leaving each page to workgroups of one XCD changed nothing.  So
// tables of many entries go the way below.
__global__ __launch_bounds__(256) void free_pages_kernel(const FreeArgs g) {
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const int had = min(max(g.lens[row], 0), g.cols * g.page), left = kept_tokens(g, row, had);
    const int end = (had + g.page - 1) / g.page;
    for (int j = (left + g.page - 1) / g.page + blockIdx.y * 256 + threadIdx.x; j < end; j += gridDim.y * 256) {
      const int32_t page = g.table[row * g.stride + j];
      if (page >= 0 && page < g.pages) atomicSub(&g.refs_out[page], 1);
    }
    if (g.lens_out != g.lens && blockIdx.y == 0 && threadIdx.x == 0) g.lens_out[row] = left;
  }
}

// Tables of many entries: the pages that lose a hold are put in order of buckets of 2^shift pages, a tile of 8192
// entries in LDS at a time; then a workgroup for each bucket counts them in LDS and subtracts: no atomics in memory.
// 4096 rows of 1025 entries over 1.4 million pages that lie anywhere, copy of the counts included: 20 us where 790000
// entries lose a hold, 32 where all 3.1 million do; 38 and 124 by atomics.  Of rows whose pages follow each other, 32 counts
// a line, 23 and 32, by atomics 10 and 16: pages come in such order from a fresh pool only.
constexpr int kTile = 8192, kBuckets = 256;

__global__ __launch_bounds__(1024, 8) void free_sort_kernel(const FreeArgs g) {
  __shared__ int32_t begin[kBuckets + 1];
  __shared__ int32_t order[kTile];
  const int t = threadIdx.x;
  const int64_t base = int64_t(blockIdx.x) * kTile;
  const int cols = g.cols, last = int(g.rows) - 1, wide = kTile / 8 / cols, rest = kTile / 8 % cols;
  int at = int((base + t) / cols), place = int(base + t - int64_t(at) * cols);
  int32_t had[8], keep[8], page[8], j[8];
  int row[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {             // entry base + t + 1024 u
    row[u] = at;
    j[u] = place;
    had[u] = g.lens[min(at, last)];
    keep[u] = g.keep ? g.keep[min(at, last)] : 0;
    at += wide;
    place += rest;
    if (place >= cols) {
      place -= cols;
      ++at;
    }
  }
  hold(had);
  hold(keep);
  if (t <= kBuckets) begin[t] = 0;
  bool gone[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int n = min(max(had[u], 0), cols * g.page), left = min(n, max(keep[u], 0));
    const bool real = row[u] <= last;
    if (real && j[u] == 0 && g.lens_out != g.lens) g.lens_out[row[u]] = left;
    const int token = j[u] * g.page;        // the page's first
    gone[u] = real && token >= left && token < n;
    page[u] = -1;
    if (__ballot(gone[u])) page[u] = g.table[min(row[u], last) * g.stride + j[u]];
  }
  hold(page);
  __syncthreads();
  int rank[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (!gone[u] || page[u] >= g.pages) page[u] = -1;
    const bool real = page[u] >= 0;
    const uint64_t all = __ballot(real);
    if (all == 0) continue;
    const int bucket = page[u] >> g.shift, one = __builtin_amdgcn_readlane(bucket, __ffsll((unsigned long long)all) - 1);
    if (__ballot(real && bucket == one) == all) {
      // pages that follow each other: one addition for all
      int start = 0;
      if ((t & 63) == 0) start = atomicAdd(&begin[one], __popcll(all));
      rank[u] = uniform(start) + __popcll(all & ((uint64_t(1) << (t & 63)) - 1));
    } else if (real) {
      rank[u] = atomicAdd(&begin[bucket], 1);
    }
  }
  __syncthreads();
  const int mine = t < g.buckets ? begin[t] : 0;
  int total;
  const int start = block_scan<16>(mine, total);
  if (t <= g.buckets) {
    begin[t] = start;
    g.ends[int64_t(blockIdx.x) * (kBuckets + 1) + t] = uint16_t(start);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (page[u] >= 0) order[begin[page[u] >> g.shift] + rank[u]] = page[u];
  __syncthreads();
  for (int i = t; i < total; i += 1024) g.sorted[base + i] = order[i];
}

__global__ __launch_bounds__(1024) void free_apply_kernel(const FreeArgs g) {
  extern __shared__ int32_t count[];        // of 2^shift pages
  const int t = threadIdx.x, span = 1 << g.shift;
  const int64_t base = int64_t(blockIdx.x) * span;
  const int pages = int(min(int64_t(span), g.pages - base));
  int32_t refs[8];                          // those of the first 8192 pages are read meanwhile
  auto load = [&](int first) {
#pragma unroll
    for (int u = 0; u < 8; ++u) refs[u] = g.refs[base + min(first + u * 1024 + t, pages - 1)];
  };
  load(0);
  for (int i = t; i < span; i += 1024) count[i] = 0;
  __syncthreads();
  // a lane for each tile, the tiles dealt to the waves in turn: its first 64 entries; of tiles that have more, the rest
  // by the wave together
  const int lane = t & 63;
  auto add = [&](const int32_t* from, int i, int step, int hi) {
    int32_t page[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) page[u] = from[min(i + u * step, hi - 1)];
    hold(page);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u * step < hi) atomicAdd(&count[page[u] & (span - 1)], 1);
  };
  for (int first = 0; first < g.tiles; first += 1024) {
    const int tile = first + lane * 16 + (t >> 6);
    const uint16_t* ends = g.ends + int64_t(min(tile, g.tiles - 1)) * (kBuckets + 1) + blockIdx.x;
    const int lo = ends[0], hi = tile < g.tiles ? ends[1] : lo;
    const int32_t* from = g.sorted + int64_t(tile) * kTile;
    const int some = min(hi, lo + 64);
    for (int i = lo; i < some; i += 8) add(from, i, 1, some);
    for (uint64_t more = __ballot(some < hi); more; more &= more - 1) {
      const int who = __ffsll((unsigned long long)more) - 1;
      const int end = __builtin_amdgcn_readlane(hi, who);
      const int32_t* it = g.sorted + int64_t(first + who * 16 + (t >> 6)) * kTile;
      for (int i = __builtin_amdgcn_readlane(some, who) + lane; i < end; i += 8 * 64) add(it, i, 64, end);
    }
  }
  __syncthreads();
  for (int first = 0; first < pages; first += 8 * 1024) {
    if (first) load(first);
    hold(refs);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = first + u * 1024 + t;
      if (i < pages) g.refs_out[base + i] = refs[u] - count[i];
    }
  }
}

// Small pools: one launch, with the counts in LDS, instead of a copy of the counts and the launch above (3.2 us against
// 1.4 + 2.4 and the time between).
__global__ __launch_bounds__(1024) void free_small_kernel(const FreeArgs g) {
  __shared__ int32_t count[kSmallPages];
  __shared__ int32_t minus[kSmallRows], from[kSmallRows], to[kSmallRows];
  const int t = threadIdx.x, pages = int(g.pages), entries = int(g.rows) * g.cols;
  const float inv = g.cols ? 1.0f / float(g.cols) : 0.0f;
  Run run;
  run.load(g.refs, 0, pages, 1);
  Entries some;
  if (entries) some.load(g.table, g.stride, 0, entries, g.cols, inv);
  int left = 0;
  if (t < g.rows) {
    const int had = min(max(g.lens[t], 0), g.cols * g.page);
    left = kept_tokens(g, t, had);
    minus[t] = -1;
    from[t] = (left + g.page - 1) / g.page;
    to[t] = (had + g.page - 1) / g.page;
  }
  run.each(0, is_free, [&](int k, uint32_t page, int) { count[page] = run.r[k]; });
  __syncthreads();
  for (int base = 0; base < entries; base += 8 * 1024) {
    if (base) some.load(g.table, g.stride, base, entries, g.cols, inv);
    some.add(count, pages, base, entries, g.cols, inv, minus, from, to);
  }
  __syncthreads();
  run.each(0, is_free, [&](int, uint32_t page, int) { if (page < pages) g.refs_out[page] = count[page]; });
  if (t < g.rows) g.lens_out[t] = left;
}

// Lengths changed in place change after every workgroup has read them.
__global__ __launch_bounds__(256) void free_lens_kernel(const FreeArgs g) {
  const int64_t row = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (row < g.rows) g.lens_out[row] = kept_tokens(g, row, min(max(g.lens[row], 0), g.cols * g.page));
}

// ---------------------------------------------------------------------------
// Moving pages together
// ---------------------------------------------------------------------------
// With U pages in use, those at or above U move into the free ones below: the nth free page takes the nth used one
// from the top.  A page p has n used ones before it, so a free one is number p - n of the free, and a used one is
// number U - 1 - n from the top; both follow from one running count, and no source is a target.
struct CompactArgs {
  Layers caches;
  const int32_t *refs, *table, *lens;
  int32_t *refs_out, *table_out, *used;
  int64_t pages, stride, rows;
  int cols;
  PageShape shape;
  Items items;
  Blocks blocks;
  int64_t table_blocks;
  // workspace
  int32_t *block_used, *hole, *mover, *mover_refs, *nth, *moves;
};

__global__ __launch_bounds__(256) void compact_count_kernel(const CompactArgs g) {
  int n = 0, total;
  for (int64_t at = g.blocks.begin(blockIdx.x); at < g.blocks.end(blockIdx.x); at += kCountBlock) {
    Run run;
    run.load(g.refs, at, g.pages, 0);
    n += run.count(is_used);
  }
  waves_before<4>(n, total);
  if (threadIdx.x == 0) g.block_used[blockIdx.x] = total;
}

// What becomes of a page with count `count` and u used ones before it.
__device__ __forceinline__ void compact_page(const CompactArgs& g, int page, int32_t count, int u, int used) {
  const bool live = count != 0;
  if (page < used) {
    if (!live) g.hole[page - u] = int32_t(page);
    else g.refs_out[page] = count;                         // a hole's count comes with its page
  } else {
    g.nth[page] = live ? int32_t(used - 1 - u) : -1;
    if (live) {
      g.mover[used - 1 - u] = int32_t(page);
      g.mover_refs[used - 1 - u] = count;
    }
    g.refs_out[page] = 0;
  }
  if (page == used - 1) *g.moves = int32_t(used - u - live);
}

__global__ __launch_bounds__(256) void compact_plan_kernel(const CompactArgs g) {
  int used, before = sum_before<int>(g.block_used, g.blocks.count, blockIdx.x, used);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *g.used = used;
    if (used == 0) *g.moves = 0;
  }
  for (int64_t at = g.blocks.begin(blockIdx.x); at < g.blocks.end(blockIdx.x); at += kCountBlock) {
    Run run;
    run.load(g.refs, at, g.pages, 0);
    int total;
    const int first = waves_before<4>(run.count(is_used), total);
    run.each(before + first, is_used, [&](int k, uint32_t page, int u) {
      if (page < g.pages) compact_page(g, page, run.r[k], u, used);
    });
    before += total;
  }
}

// Small pools: count and plan in one launch (15000 pages: 7 us, 4.7 + 8.0 in two).
__global__ __launch_bounds__(1024) void compact_small_kernel(const CompactArgs g) {
  const int t = threadIdx.x;
  Run run;
  run.load(g.refs, 0, g.pages, 0);
  int used;
  const int before = waves_before<16>(run.count(is_used), used);
  run.each(before, is_used, [&](int k, uint32_t page, int u) {
    if (page < g.pages) compact_page(g, page, run.r[k], u, used);
  });
  if (t == 0) {
    *g.used = used;
    if (used == 0) *g.moves = 0;
  }
}

__global__ __launch_bounds__(256) void compact_move_kernel(const CompactArgs g) {
  const int64_t moves = *g.moves, used = *g.used;
  if (int64_t(blockIdx.x) < g.table_blocks) {
    const int64_t step = g.table_blocks * 256, at = int64_t(blockIdx.x) * 256 + threadIdx.x;
    for (int64_t i = at; i < moves; i += step) g.refs_out[g.hole[i]] = g.mover_refs[i];
    for (int64_t row = blockIdx.x; row < g.rows; row += g.table_blocks) {
      const int held = (min(max(g.lens[row], 0), g.cols * g.shape.page) + g.shape.page - 1) / g.shape.page;
      for (int j = threadIdx.x; j < g.cols; j += 256) {
        int32_t page = g.table[row * g.stride + j];
        if (j < held && page >= used && page < g.pages) {
          const int32_t n = g.nth[page];
          if (n >= 0) page = g.hole[n];
        }
        g.table_out[row * g.cols + j] = page;
      }
    }
    return;
  }
  const int64_t waves = (int64_t(gridDim.x) - g.table_blocks) * 4;
  const int64_t total = moves * g.items.layers * g.items.parts;
  for (int64_t i = (int64_t(blockIdx.x) - g.table_blocks) * 4 + uniform(threadIdx.x >> 6); i < total; i += waves) {
    const Item it = g.items.at(i);
    const int layer = uniform(it.layer);
    copy_part(g.caches.p[layer], g.caches.p[layer], g.shape, g.mover[it.copy], g.hole[it.copy], g.shape.page, it.part);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
inline mx_status_t launched() { return hipGetLastError() == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

inline bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
inline bool off8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) != 0; }

// Caches of all layers: alike, with all their pointers, pages of at most 2^30 bytes of codes.
mx_status_t check_layers(const mx_kv_cache_t* c, int layers) {
  if (layers < 1 || layers > 65536) return MX_ERR_SHAPE;
  if (!c) return MX_ERR_NULL;
  for (int l = 0; l < layers; ++l) {
    const mx_status_t st = check_kv_cache(c[l]);
    if (st != MX_OK) return st;
    if (c[l].pages != c[0].pages || c[l].kv_heads != c[0].kv_heads || c[l].page != c[0].page || c[l].dim != c[0].dim)
      return MX_ERR_SHAPE;
  }
  if (int64_t(c->kv_heads) * c->page > (int64_t(1) << 30) / c->dim) return MX_ERR_SHAPE;
  if (c->pages > INT32_MAX) return MX_ERR_SHAPE;
  if (c->pages == 0) return MX_OK;
  for (int l = 0; l < layers; ++l) {
    if (!c[l].k || !c[l].k_scales || !c[l].v || !c[l].v_scales) return MX_ERR_NULL;
    if (misaligned(c[l].k) || misaligned(c[l].k_scales) || misaligned(c[l].v) || misaligned(c[l].v_scales))
      return MX_ERR_ALIGN;
  }
  return MX_OK;
}

PageShape shape_of(const mx_kv_cache_t& c) { return {c.kv_heads, c.page, c.dim}; }

void fill_layers(Layers& to, const mx_kv_cache_t* c, int n) {
  for (int l = 0; l < n; ++l) {
    uint8_t* p[4] = {c[l].k, c[l].k_scales, c[l].v, c[l].v_scales};
    std::copy(p, p + 4, to.p[l]);
  }
}

// 8 KiB parts of a page, the last one short.
Items items_of(const mx_kv_cache_t& c, int layers) {
  const int64_t codes = int64_t(c.kv_heads) * c.page * c.dim / 16;
  Items it;
  it.layers = layers;
  it.parts = int((2 * (codes + codes / 32) + kPartGranules - 1) / kPartGranules);
  it.inv_layers = 1.0 / it.layers;
  it.inv_parts = 1.0 / it.parts;
  return it;
}

// LDS that nothing uses: it keeps the copying workgroups to two on a CU, with which the memory does more (1.1 GB read and
// written: 213 us, with eight 218; 1.0 GB moved in a pool: 178 and 188).
constexpr size_t kTwoOnACu = 80000;

// Pages of less than a part leave most of a wave's loads undone, so that all the waves that fit are wanted (120000 pages of 2 KB
// moved: 169 us with two workgroups on a CU, 101 with eight).
size_t copy_lds(const Items& it) { return it.parts > 1 ? kTwoOnACu : 0; }

// Workgroups of four waves for `copies` copies, which walk the work where there are more than 64 for each CU.
unsigned copy_grid(int64_t copies, const Items& it) {
  const int64_t cus = std::max<int64_t>(device_cus(), 1);
  const double waves = double(copies) * it.layers * it.parts;
  return unsigned(std::max(1.0, std::min(double(64 * cus), std::ceil(waves / 4.0))));
}

Blocks blocks_of(int64_t pages) {
  Blocks b;
  b.pages = pages;
  const int64_t runs = (pages + kCountBlock - 1) / kCountBlock;
  b.per_block = std::max<int64_t>(1, (runs + kMostCountBlocks - 1) / kMostCountBlocks) * kCountBlock;
  b.count = int((pages + b.per_block - 1) / b.per_block);
  return b;
}

// Hands out parts of a workspace, each on a 16-byte border.
struct Space {
  uint8_t* base;
  int64_t used = 0;
  template <class T>
  T* take(int64_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += (n * int64_t(sizeof(T)) + 15) / 16 * 16;
    return p;
  }
};

constexpr int64_t kMostRows = int64_t(1) << 20;

// Whether one workgroup holds the counts of a pool and reads a table in a few steps.
bool is_small(int64_t pages, int64_t rows, int64_t cols) {
  return pages <= kSmallPages && rows <= kSmallRows && rows * cols <= kSmallEntries;
}

// Pages that all children together can need: a copy and a started page each, and one a page's worth of new tokens.
int64_t fork_capacity(int64_t pages, int64_t children, int64_t tokens, int page) {
  return std::min(pages, 2 * children + tokens / page);
}

int64_t fork_space(ForkArgs& g, uint8_t* base) {
  Space s{base};
  g.start = s.take<int64_t>(g.children);
  g.child_sum = s.take<int64_t>(g.child_blocks);
  g.copy = s.take<int4>(g.children);
  g.kids = s.take<int32_t>(g.rows);
  g.writers = s.take<int32_t>(g.rows);
  g.first = s.take<int32_t>(g.rows);
  g.info = s.take<int32_t>(g.children);
  g.child_copies = s.take<int32_t>(g.child_blocks);
  g.block_free = s.take<int32_t>(g.blocks.count);
  g.list = s.take<int32_t>(g.capacity);
  g.copies = s.take<int32_t>(1);
  return s.used;
}

mx_status_t fork_sizes(ForkArgs& g, int64_t pages, int64_t rows, int64_t children, int64_t tokens, int page) {
  if (pages < 0 || pages > INT32_MAX || rows < 0 || rows > kMostRows || children < 0 || children > kMostRows || tokens < 0 ||
      tokens > INT32_MAX || page < 16 || page > 65536 || page % 16)
    return MX_ERR_SHAPE;
  g.pages = pages;
  g.rows = rows;
  g.children = children;
  g.tokens = tokens;
  g.blocks = blocks_of(pages);
  g.child_blocks = int((children + 255) / 256);
  g.capacity = fork_capacity(pages, children, tokens, page);
  return MX_OK;
}

// Whether the entries of a table are put in order first, and in what.  The host knows the table's size alone, not how many
// rows end nor where their pages lie.  Microseconds by atomics and in order, rows of 512 entries over 100000 pages, counts
// copied, captured (those of 1.5 million pages within 9 of these):
//   entries                            2^18          2^19          2^20          2^21          2^22
//   pages anywhere, all rows end       14.4   14.6   24.8   15.6   45.6   17.2   86.9   21.8   171    32.4
//                   a quarter           6.8   10.7   10.4   11.1   15.7   11.8   27.1   13.3   48.9   19.5
//                   8 rows              5.0    8.3    5.5    8.5    5.7    8.4    6.4    8.7    7.9   11.1
//   pages in a row, all rows end        4.9   15.9    5.8   17.9    7.0   19.8   10.2   21.6   17.5   29.0
//                   8 rows              4.4   11.6    4.9   11.4    5.2   11.6    5.9   11.7    7.4   14.2
// In place the atomics take 1 to 5 less (8 rows, anywhere: 3.9 against 8.3 with 2^19, 6.6 against 11.0 with 2^22).  So from 2^19
// entries on, where all rows that end first gain: what it can save grows with the table, what it can cost stays at 3 to 18.
// Up to 2^28 entries for the workspace's sake; buckets of up to 2^15 pages fit LDS.
bool free_plan(FreeArgs& g, int64_t pages, int64_t rows, int64_t cols) {
  if (rows * cols < (int64_t(1) << 19) || rows * cols > (int64_t(1) << 28)) return false;
  if (pages <= kSmallPages || pages > int64_t(kBuckets) << 15) return false;
  g.shift = 0;
  while (int64_t(kBuckets) << g.shift < pages) ++g.shift;
  g.buckets = int((pages + (int64_t(1) << g.shift) - 1) >> g.shift);
  g.tiles = int((rows * cols + kTile - 1) / kTile);
  return true;
}

int64_t free_space(FreeArgs& g, uint8_t* base) {
  Space s{base};
  g.sorted = s.take<int32_t>(int64_t(g.tiles) * kTile);
  g.ends = s.take<uint16_t>(int64_t(kBuckets + 1) * g.tiles);
  return s.used;
}

mx_status_t free_sizes(int64_t pages, int64_t rows, int64_t cols, int page) {
  if (pages < 0 || pages > INT32_MAX || rows < 0 || rows > kMostRows || page < 16 || page > 65536 || page % 16)
    return MX_ERR_SHAPE;
  return cols < 0 || cols > INT32_MAX / page ? MX_ERR_SHAPE : MX_OK;
}

int64_t compact_space(CompactArgs& g, uint8_t* base) {
  Space s{base};
  g.block_used = s.take<int32_t>(g.blocks.count);
  g.hole = s.take<int32_t>(g.pages / 2);
  g.mover = s.take<int32_t>(g.pages / 2);
  g.mover_refs = s.take<int32_t>(g.pages / 2);
  g.nth = s.take<int32_t>(g.pages);
  g.moves = s.take<int32_t>(1);
  return s.used;
}

}  // namespace mxk

using namespace mxk;

extern "C" mx_status_t mx_kv_copy(const mx_kv_cache_t* src, const mx_kv_cache_t* dst, int layers,
                                  const int32_t* src_pages, const int32_t* dst_pages, int64_t count,
                                  hipStream_t stream) {
  mx_status_t st = check_layers(src, layers);
  if (st != MX_OK) return st;
  st = check_layers(dst, layers);
  if (st != MX_OK) return st;
  if (src->kv_heads != dst->kv_heads || src->page != dst->page || src->dim != dst->dim) return MX_ERR_SHAPE;
  if (count < 0 || count > INT32_MAX) return MX_ERR_SHAPE;
  if (count == 0 || src->pages == 0 || dst->pages == 0) return MX_OK;
  if (!src_pages || !dst_pages) return MX_ERR_NULL;
  if (off4(src_pages) || off4(dst_pages)) return MX_ERR_ALIGN;
  for (int l = 0; l < layers; l += kLayersPerLaunch) {
    const int n = std::min(kLayersPerLaunch, layers - l);
    CopyArgs g = {};
    fill_layers(g.from, src + l, n);
    fill_layers(g.to, dst + l, n);
    g.src = src_pages;
    g.dst = dst_pages;
    g.count = count;
    g.src_pages = src->pages;
    g.dst_pages = dst->pages;
    g.shape = shape_of(*src);
    g.items = items_of(*src, n);
    page_copy_kernel<<<copy_grid(count, g.items), 256, copy_lds(g.items), stream>>>(g);
  }
  return launched();
}

extern "C" mx_status_t mx_kv_fork_workspace(int64_t pages, int64_t rows, int64_t children, int64_t tokens, int page,
                                            int64_t* bytes) {
  if (!bytes) return MX_ERR_NULL;
  ForkArgs g = {};
  const mx_status_t st = fork_sizes(g, pages, rows, children, tokens, page);
  if (st != MX_OK) return st;
  *bytes = fork_space(g, nullptr);
  return MX_OK;
}

extern "C" mx_status_t mx_kv_fork(const mx_kv_cache_t* caches, int layers, const int32_t* refs,
                                  const int32_t* page_table, int64_t table_stride, int64_t table_cols,
                                  const int32_t* lens, int64_t rows, const int32_t* parents, int64_t children,
                                  const int32_t* cu, int64_t tokens, int release, int32_t* refs_out,
                                  int32_t* table_out, int64_t out_cols, int32_t* lens_out, int64_t* slots,
                                  void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  mx_status_t st = check_layers(caches, layers);
  if (st != MX_OK) return st;
  ForkArgs g = {};
  const int page = caches->page;
  st = fork_sizes(g, caches->pages, rows, children, tokens, page);
  if (st != MX_OK) return st;
  if (table_cols < 0 || out_cols < table_cols || out_cols > INT32_MAX / page || (table_stride < table_cols && rows > 1))
    return MX_ERR_SHAPE;
  if (!parents && children != rows) return MX_ERR_SHAPE;
  if (!cu && tokens) return MX_ERR_NULL;
  if (g.pages && (!refs || !refs_out)) return MX_ERR_NULL;
  if (rows && (!lens || (table_cols && !page_table))) return MX_ERR_NULL;
  if (children && (!lens_out || (out_cols && !table_out))) return MX_ERR_NULL;
  if (tokens && !slots) return MX_ERR_NULL;
  if (off4(refs) || off4(refs_out) || off4(lens) || off4(lens_out) || off4(page_table) || off4(table_out) ||
      off4(parents) || off4(cu) || off8(slots))
    return MX_ERR_ALIGN;
  if (children && ((table_out && table_out == page_table) || lens_out == lens)) return MX_ERR_ARG;
  const int64_t need = fork_space(g, nullptr);
  if (workspace_bytes < need) return MX_ERR_SHAPE;
  if (!workspace) return MX_ERR_NULL;
  if (misaligned(workspace)) return MX_ERR_ALIGN;
  fork_space(g, static_cast<uint8_t*>(workspace));
  g.refs = refs; g.table = page_table; g.lens = lens; g.parents = parents; g.cu = cu;
  g.refs_out = refs_out; g.table_out = table_out; g.lens_out = lens_out; g.slots = slots;
  g.stride = table_stride;
  g.cols = int(table_cols); g.out_cols = int(out_cols); g.release = release != 0;
  g.shape = shape_of(*caches);
  const int64_t cus = std::max<int64_t>(device_cus(), 1);
  const bool small = is_small(g.pages, rows, table_cols) && children <= kSmallRows;
  const unsigned both = unsigned(g.child_blocks + g.blocks.count);
  if (small) {
    fork_small_kernel<<<1, 1024, 0, stream>>>(g);
  } else if (parents || !release) {
    const int64_t copied = refs_out != refs ? g.pages : 0, n = std::max(rows, copied);
    if (rows <= kBeginRows && children <= kBeginChildren) {
      fork_begin_kernel<<<unsigned(1 + std::min(2 * cus, (copied + 1023) / 1024)), 1024, 0, stream>>>(g);
    } else {
      if (n) fork_init_kernel<<<unsigned(std::min(8 * cus, (n + 255) / 256)), 256, 0, stream>>>(g);
      if (children) fork_kids_kernel<<<unsigned(g.child_blocks), 256, 0, stream>>>(g);
    }
    if (rows && table_cols) {
      // a workgroup for eight rows, several where there are few rows
      const int64_t x = std::min((rows + kRowGroup - 1) / kRowGroup, 8 * cus), y = std::min((table_cols + 255) / 256, std::max<int64_t>(1, 8 * cus / x));
      fork_counts_kernel<<<dim3(unsigned(x), unsigned(y)), 256, 0, stream>>>(g);
    }
  }
  if (!small && both) fork_needs_kernel<<<both, 256, 0, stream>>>(g);
  if (children == 0) {
    if (tokens) fork_rows_kernel<<<1, 256, 0, stream>>>(g);
    return launched();
  }
  if (!small) fork_list_kernel<<<both, 256, 0, stream>>>(g);
  for (int l = 0; l < layers; l += kLayersPerLaunch) {
    const int n = std::min(kLayersPerLaunch, layers - l);
    fill_layers(g.caches, caches + l, n);
    g.items = items_of(*caches, n);
    const unsigned copiers = tokens && g.pages ? copy_grid(children, g.items) : 0;
    if (l == 0) fork_rows_kernel<<<unsigned(children) + copiers, 256, 0, stream>>>(g);
    else if (copiers) fork_copy_kernel<<<copiers, 256, 0, stream>>>(g);
  }
  return launched();
}

extern "C" mx_status_t mx_kv_free_workspace(int64_t pages, int64_t rows, int64_t table_cols, int page, int64_t* bytes) {
  if (!bytes) return MX_ERR_NULL;
  const mx_status_t st = free_sizes(pages, rows, table_cols, page);
  if (st != MX_OK) return st;
  FreeArgs g = {};
  *bytes = free_plan(g, pages, rows, table_cols) ? free_space(g, nullptr) : 0;
  return MX_OK;
}

extern "C" mx_status_t mx_kv_free(const int32_t* refs, int64_t pages, int page, const int32_t* page_table,
                                  int64_t table_stride, int64_t table_cols, const int32_t* lens, int64_t rows,
                                  const int32_t* keep, int32_t* refs_out, int32_t* lens_out, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
  const mx_status_t st = free_sizes(pages, rows, table_cols, page);
  if (st != MX_OK) return st;
  if (table_stride < table_cols && rows > 1) return MX_ERR_SHAPE;
  if (pages && (!refs || !refs_out)) return MX_ERR_NULL;
  if (rows && (!lens || !lens_out || (table_cols && !page_table))) return MX_ERR_NULL;
  if (keep && keep == lens_out) return MX_ERR_ARG;
  if (off4(refs) || off4(refs_out) || off4(lens) || off4(lens_out) || off4(page_table) || off4(keep)) return MX_ERR_ALIGN;
  FreeArgs g = {};
  const bool many = free_plan(g, pages, rows, table_cols);
  if (many) {
    if (workspace_bytes < free_space(g, nullptr)) return MX_ERR_SHAPE;
    if (!workspace) return MX_ERR_NULL;
    if (misaligned(workspace)) return MX_ERR_ALIGN;
    free_space(g, static_cast<uint8_t*>(workspace));
  }
  if (rows == 0 && (pages == 0 || refs_out == refs)) return MX_OK;
  g.refs = refs; g.table = page_table; g.lens = lens; g.keep = keep; g.refs_out = refs_out; g.lens_out = lens_out;
  g.pages = pages; g.stride = table_stride; g.rows = rows; g.cols = int(table_cols); g.page = page;
  if (refs_out != refs && is_small(pages, rows, table_cols)) {
    free_small_kernel<<<1, 1024, 0, stream>>>(g);
    return launched();
  }
  const int64_t cus = std::max<int64_t>(device_cus(), 1);
  if (many) {
    free_sort_kernel<<<unsigned(g.tiles), 1024, 0, stream>>>(g);
    free_apply_kernel<<<unsigned(g.buckets), 1024, size_t(4) << g.shift, stream>>>(g);
  } else {
    if (refs_out != refs && pages)
      refs_copy_kernel<<<unsigned(std::min(8 * cus, (pages + 255) / 256)), 256, 0, stream>>>(refs, refs_out, pages);
    if (rows) {
      const int64_t x = std::min(rows, 8 * cus);
      const int64_t y = std::min(std::max<int64_t>(1, (table_cols + 255) / 256), std::max<int64_t>(1, 8 * cus / x));
      free_pages_kernel<<<dim3(unsigned(x), unsigned(y)), 256, 0, stream>>>(g);
    }
  }
  if (rows && lens_out == lens) free_lens_kernel<<<unsigned((rows + 255) / 256), 256, 0, stream>>>(g);
  return launched();
}

extern "C" mx_status_t mx_kv_compact_workspace(int64_t pages, int64_t* bytes) {
  if (!bytes) return MX_ERR_NULL;
  if (pages < 0 || pages > INT32_MAX) return MX_ERR_SHAPE;
  CompactArgs g = {};
  g.pages = pages;
  g.blocks = blocks_of(pages);
  *bytes = compact_space(g, nullptr);
  return MX_OK;
}

extern "C" mx_status_t mx_kv_compact(const mx_kv_cache_t* caches, int layers, const int32_t* refs,
                                     const int32_t* page_table, int64_t table_stride, int64_t table_cols,
                                     const int32_t* lens, int64_t rows, int32_t* refs_out, int32_t* table_out,
                                     int32_t* used, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const mx_status_t st = check_layers(caches, layers);
  if (st != MX_OK) return st;
  const int page = caches->page;
  if (rows < 0 || rows > kMostRows || table_cols < 0 || table_cols > INT32_MAX / page ||
      (table_stride < table_cols && rows > 1))
    return MX_ERR_SHAPE;
  CompactArgs g = {};
  g.pages = caches->pages;
  g.blocks = blocks_of(g.pages);
  if (!used || (g.pages && (!refs || !refs_out))) return MX_ERR_NULL;
  if (rows && (!lens || (table_cols && (!page_table || !table_out)))) return MX_ERR_NULL;
  if (off4(refs) || off4(refs_out) || off4(lens) || off4(page_table) || off4(table_out) || off4(used)) return MX_ERR_ALIGN;
  // a table changed in place has the same rows
  if (table_out == page_table && table_stride != table_cols && rows > 1) return MX_ERR_ARG;
  const int64_t need = compact_space(g, nullptr);
  if (workspace_bytes < need) return MX_ERR_SHAPE;
  if (!workspace) return MX_ERR_NULL;
  if (misaligned(workspace)) return MX_ERR_ALIGN;
  compact_space(g, static_cast<uint8_t*>(workspace));
  g.refs = refs; g.table = page_table; g.lens = lens;
  g.refs_out = refs_out; g.table_out = table_out; g.used = used;
  g.stride = table_stride; g.rows = rows; g.cols = int(table_cols);
  g.shape = shape_of(*caches);
  const int64_t cus = std::max<int64_t>(device_cus(), 1);
  if (g.pages <= kSmallPages) {
    compact_small_kernel<<<1, 1024, 0, stream>>>(g);
  } else {
    compact_count_kernel<<<unsigned(g.blocks.count), 256, 0, stream>>>(g);
    compact_plan_kernel<<<unsigned(g.blocks.count), 256, 0, stream>>>(g);
  }
  for (int l = 0; l < layers; l += kLayersPerLaunch) {
    const int n = std::min(kLayersPerLaunch, layers - l);
    fill_layers(g.caches, caches + l, n);
    g.items = items_of(*caches, n);
    const unsigned copiers = g.pages > 1 ? copy_grid(g.pages / 2, g.items) : 0;
    g.table_blocks = l == 0 ? std::max<int64_t>(1, std::min(4 * cus, std::max(rows, g.pages / 2048))) : 0;
    if (g.table_blocks + copiers) compact_move_kernel<<<unsigned(g.table_blocks) + copiers, 256, copy_lds(g.items), stream>>>(g);
  }
  return launched();
}
