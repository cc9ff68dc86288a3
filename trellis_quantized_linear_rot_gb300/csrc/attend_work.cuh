// How the attention kernels divide their work, and how the parts of a row are
// joined.
//
// An item is one (sequence, kv head). The tiles of all items, sequence by
// sequence, form one line that is cut into equal runs, so that ragged lengths
// and few long sequences fill the GPU alike. A run has a team of blocks, one
// for each block of rows (one if the rows of a kv head fit one): they read the
// same keys at about the same time, so that memory gives them once and L2 the
// other times. Lengths are on the device, so every block finds its run itself.
// A run holds whole items but for its first and its last, which other runs may
// share: those leave (max, sum, weighted sum) of their part in the workspace,
// and the parts are joined in an order that the sizes and lengths fix, by the
// block that arrives last at the item or by a launch of its own. No block waits for another.
#pragma once

#include <algorithm>

#include "ptx.cuh"
#include "spec.cuh"

namespace tfx {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Going from one item to the next costs a block about as much as kGap tiles
// (its sums are joined and written, another q comes), so an item has kGap
// places in the line after those of its tiles. On tcgen05, us with two, four
// and six: a tree of 64 nodes over 50,001 slots 81.6, 80.0, 78.9; 19 trees of
// 25 over up to 6,000 118.5, 116.0, 116.1; 19 of 53 over up to 798 29.5, 29.1,
// 29.8. With mma.sync an item is less: 32 tokens over up to 300 slots 15.4
// with one, 16.6 with two.
//
// The line of places (below 2^31: checked on the host) and one run of it: the
// first `longer` runs have per + 1 places, the others per. No more runs than
// places, so that no run between two others is empty.
struct Line {
  int runs, per, longer;
  int begin, end;
  __device__ __forceinline__ void cut(int total, int most, int run) {
    runs = min(total, most);
    per = total / runs;
    longer = total - per * runs;
    const int i = min(run, runs);
    begin = begin_of(i);
    end = i < runs ? begin_of(i + 1) : begin;
  }
  __device__ __forceinline__ int begin_of(int run) const { return run * per + min(run, longer); }
  // The run that holds place f.
  __device__ __forceinline__ int run_of(int f) const {
    const int border = longer * (per + 1);
    return f < border ? f / (per + 1) : longer + (f - border) / per;
  }
};

// Position of a tile: item `item` (kv head) of sequence b, tile t of its nt;
// first is the place of the item's tile 0 in the line.
struct Cursor {
  int b, item, t, nt;
  int first;
  Span span;
};

template <int kTile>
__device__ __forceinline__ int tiles_of(const Span& s) {
  return s.slots <= kTile ? 1 : (s.slots + kTile - 1) / kTile;
}

template <int kTile, int kGap>
__device__ __forceinline__ void advance(const AttendArgs& a, Cursor* c) {
  if (++c->t < c->nt) return;
  c->t = 0;
  c->first += c->nt + kGap;
  if (++c->item < a.c.kv_heads) return;
  c->item = 0;
  if (++c->b >= a.c.batch) return;
  c->span = sequence_span(a.c, c->b, a.nodes);
  c->nt = tiles_of<kTile>(c->span);
}

// Block-wide: the line, run number `run` of at most `most`, the cursor at its
// begin and its number of tiles (0: nothing to do, the cursor is not set).
// `scratch` has room for 2 * (kThreads / 32) + 6 ints. Batches of up to 32
// sequences are scanned by every warp for itself, without meeting; of up to
// kThreads once by the block; larger ones twice (length, then place).
template <int kTile, int kGap, int kThreads>
__device__ int find_run(const AttendArgs& a, int most, int run, int* scratch, Line* line, Cursor* cur) {
  const int items = a.c.kv_heads;
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int batch = a.c.batch;
  if (batch <= 32) {
    const Span span = lane < batch ? sequence_span(a.c, lane, a.nodes) : Span{};
    const int nt = lane < batch ? tiles_of<kTile>(span) : 0, places = lane < batch ? nt + kGap : 0;
    int upto = places * items, tiles = nt * items;
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(~0u, upto, o), z = __shfl_up_sync(~0u, tiles, o);
      if (lane >= o) upto += y, tiles += z;
    }
    const int from = upto - places * items;
    line->cut(__shfl_sync(~0u, upto, 31), most, run);
    if (line->begin >= line->end) return 0;
    // The sequences that begin and end lie in, their items and places in those.
    const int b = __ffs(__ballot_sync(~0u, line->begin < upto)) - 1;
    const int last = __ffs(__ballot_sync(~0u, line->end <= upto)) - 1;
    const int nt_b = __shfl_sync(~0u, nt, b), nt_last = __shfl_sync(~0u, nt, last);
    const int in_b = line->begin - __shfl_sync(~0u, from, b), in_last = line->end - __shfl_sync(~0u, from, last);
    const int item = in_b / (nt_b + kGap), t = in_b - item * (nt_b + kGap);
    const int item_last = in_last / (nt_last + kGap), t_last = in_last - item_last * (nt_last + kGap);
    const int before = __shfl_sync(~0u, tiles - nt * items, b) + item * nt_b + min(t, nt_b);
    const int n = __shfl_sync(~0u, tiles - nt * items, last) + item_last * nt_last + min(t_last, nt_last) - before;
    if (n == 0) return 0;
    const Span own{__shfl_sync(~0u, span.context, b), __shfl_sync(~0u, span.slots, b)};
    *cur = Cursor{b, item, t, nt_b, line->begin - t, own};
    if (t >= nt_b) {   // in a gap: on to the next item
      cur->t = nt_b - 1;
      advance<kTile, kGap>(a, cur);
    }
    return n;
  }
  // Sequence of the run's begin, its first place; tiles before begin and end;
  // the sequence's span.
  int* found = scratch + 2 * kWarps;
  for (int pass = batch <= kThreads ? 1 : 0; pass < 2; ++pass) {
    int before = 0, tiles_before = 0;
    for (int b0 = 0; b0 < batch; b0 += kThreads) {
      const int b = b0 + tid;
      const Span span = b < batch ? sequence_span(a.c, b, a.nodes) : Span{};
      const int nt = b < batch ? tiles_of<kTile>(span) : 0;
      const int n = b < batch ? (nt + kGap) * items : 0;
      int upto = n, tiles = nt * items;
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(~0u, upto, o), z = __shfl_up_sync(~0u, tiles, o);
        if (lane >= o) upto += y, tiles += z;
      }
      if (lane == 31) scratch[warp] = upto, scratch[kWarps + warp] = tiles;
      __syncthreads();
      int prior = before, tiles_prior = tiles_before;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) prior += scratch[w], tiles_prior += scratch[kWarps + w];
        before += scratch[w], tiles_before += scratch[kWarps + w];
      }
      upto += prior, tiles += tiles_prior;
      if (b0 + kThreads >= batch && (pass == 0 || batch <= kThreads)) line->cut(before, most, run);
      if (pass == 1 && n > 0) {
        // Tiles of the line before a place of this sequence.
        auto tiles_to = [&](int place) {
          const int in = place - (upto - n), item = in / (nt + kGap);
          return tiles - nt * items + item * nt + min(in - item * (nt + kGap), nt);
        };
        if (line->begin >= upto - n && line->begin < upto) {
          found[0] = b;
          found[1] = upto - n;
          found[2] = tiles_to(line->begin);
          found[4] = span.context;
          found[5] = span.slots;
        }
        if (line->end > upto - n && line->end <= upto) found[3] = tiles_to(line->end);
      }
      __syncthreads();
    }
  }
  if (line->begin >= line->end) return 0;
  const int n_tiles = found[3] - found[2];
  if (n_tiles == 0) return 0;
  cur->b = found[0];
  cur->span = Span{found[4], found[5]};
  cur->nt = tiles_of<kTile>(cur->span);
  const int in = line->begin - found[1];
  cur->item = in / (cur->nt + kGap);
  cur->t = in - cur->item * (cur->nt + kGap);
  cur->first = line->begin - cur->t;
  if (cur->t >= cur->nt) {   // in a gap: on to the next item
    cur->t = cur->nt - 1;
    advance<kTile, kGap>(a, cur);
  }
  return n_tiles;
}

// Place of run `run`'s part of the item at `first`, for row block rb of
// row_blocks. A run has two parts for each row block in the workspace: of the
// item it begins in, and of a later item it ends in. A part is kRows rows of D
// sums, kRows maxima (in units of log 2) and kRows sums of weights.
struct Rows {
  int rb, row_blocks;
};
__device__ __forceinline__ int part_index(const Line& l, const Rows& w, int run, int first) {
  return 2 * (run * w.row_blocks + w.rb) + (l.begin_of(run) < first ? 1 : 0);
}
template <int kRows, int D>
constexpr size_t kPartFloats = static_cast<size_t>(kRows) * (D + 2);

// Counts this block's part of the item (nt tiles from `first`); true in the
// block that arrives last. An item cut between runs is counted at the place of
// its first part, so that the counters' number does not depend on the call's
// sizes and a workspace serves any of them.
__device__ __forceinline__ bool arrives_last(const AttendArgs& a, const Line& l, const Rows& w, int first, int nt) {
  const int p0 = l.run_of(first), parts = l.run_of(first + nt - 1) - p0 + 1;
  int* counter = a.counters + part_index(l, w, p0, first);
  const bool last = atomicAdd(counter, 1) + 1 == parts;
  if (last) *counter = 0;   // ready for the next call
  return last;
}

// Row r of an item: node and head.
struct RowOf {
  int node, head;
};
__device__ __forceinline__ RowOf row_of(const AttendArgs& a, int kvh, int r) {
  const int node = r / a.group;
  return {node, kvh * a.group + r - node * a.group};
}

// kThreads threads (this one is number tid): joins the parts of the item at
// `first` (nt tiles) and writes its rows, which start at row0 of its kv head.
// Parts are added in run order.
template <typename T, int kRows, int D, int kThreads>
__device__ void join_parts(const AttendArgs& a, const Line& line, const Rows& w, int b, int kvh, int row0,
                           int rows, int first, int nt, bool idle, int tid) {
  constexpr size_t kPart = kPartFloats<kRows, D>;
  const int p0 = line.run_of(first), n = line.run_of(first + nt - 1) - p0 + 1;
  // Every part but the first is the one its run begins with.
  const float* part0 = a.partials + part_index(line, w, p0, first) * kPart;
  const float* part1 = a.partials + 2 * (static_cast<size_t>(p0 + 1) * w.row_blocks + w.rb) * kPart;
  const size_t step = 2 * static_cast<size_t>(w.row_blocks) * kPart;
  // A thread takes four columns of kBatch rows at a time, kGroup parts of each
  // at once, so that many loads are in flight; few rows have many parts and
  // many rows few.
  constexpr int kBatch = kRows > 16 ? 4 : 1, kGroup = kRows > 16 ? 2 : 6, kStep = kThreads / (D / 4);
  const int e = tid % (D / 4) * 4;
  for (int r0 = tid / (D / 4); r0 < rows; r0 += kBatch * kStep) {
    float top[kBatch], l[kBatch];
    float4 o[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top[k] = -INFINITY, l[k] = 0.f, o[k] = float4{0.f, 0.f, 0.f, 0.f};
    for (int q0 = 0; q0 < n; q0 += kGroup) {
      float m[kBatch][kGroup], u[kBatch][kGroup];
      float4 x[kBatch][kGroup];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const float* part = q0 + i == 0 ? part0 : part1 + (q0 + i - 1) * step;
          const int r = r0 + k * kStep;
          const bool real = q0 + i < n && r < rows;
          m[k][i] = real ? __ldcg(part + kRows * D + r) : -INFINITY;
          u[k][i] = real ? __ldcg(part + kRows * D + kRows + r) : 0.f;
          x[k][i] = real ? __ldcg(reinterpret_cast<const float4*>(part + r * D + e)) : float4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        float high = top[k];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) high = fmaxf(high, m[k][i]);
        const float base = high == -INFINITY ? 0.f : high;
        const float keep = exp2_approx(top[k] - base);
        top[k] = high;
        l[k] *= keep, o[k].x *= keep, o[k].y *= keep, o[k].z *= keep, o[k].w *= keep;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const float f = exp2_approx(m[k][i] - base);
          l[k] += f * u[k][i];
          o[k].x += f * x[k][i].x, o[k].y += f * x[k][i].y, o[k].z += f * x[k][i].z, o[k].w += f * x[k][i].w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kStep;
      if (r >= rows) continue;
      const RowOf ro = row_of(a, kvh, row0 + r);
      const int up = a.parents[b * a.stride_parents + ro.node];
      const bool present = !idle && up >= -1 && up < ro.node;
      const bool empty = !present || l[k] == 0.f;
      const float inv = empty ? 0.f : 1.f / l[k];
      const size_t at = (static_cast<size_t>(b) * a.nodes + ro.node) * a.heads + ro.head;
      const float y[4] = {o[k].x, o[k].y, o[k].z, o[k].w};
      alignas(8) T t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = from_f32<T>(empty ? 0.f : y[i] * inv);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + e) = *reinterpret_cast<const uint2*>(t);
      if (e == 0) a.lse[at] = empty ? -INFINITY : (top[k] + log2f(l[k])) * kLn2;
    }
  }
}

// The same for parts of 128 rows, which are stored by column (column c of row
// r at c * 128 + r: there a thread has a row, and a warp's writes lie
// together): the block's kThreads / 128 groups share out the parts, kGroup at
// once, and this thread joins kColumns columns from c0 on of row tid % 128.
template <typename T, int D, int kColumns, int kGroup, int kThreads>
__device__ void join_row(const AttendArgs& a, const Line& line, const Rows& w, int b, int kvh, int row0, int rows,
                         int c0, int first, int nt, bool idle, int up) {
  constexpr int kGroups = kThreads / 128;
  __shared__ float others[kGroups > 1 ? kGroups - 1 : 1][kGroups > 1 ? kColumns + 2 : 1][128];
  const int r = threadIdx.x % 128, g = threadIdx.x / 128;
  constexpr size_t kPart = kPartFloats<128, D>;
  const int p0 = line.run_of(first), n = line.run_of(first + nt - 1) - p0 + 1;
  const float* part0 = a.partials + part_index(line, w, p0, first) * kPart + r;
  const float* part1 = a.partials + 2 * (static_cast<size_t>(p0 + 1) * w.row_blocks + w.rb) * kPart + r;
  const size_t step = 2 * static_cast<size_t>(w.row_blocks) * kPart;
  float top = -INFINITY, l = 0.f, o[kColumns] = {};
#pragma unroll 1
  for (int q0 = g * kGroup; q0 < n; q0 += kGroups * kGroup) {
    float m[kGroup], u[kGroup], x[kGroup][kColumns];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const bool real = q0 + i < n && r < rows;
      const float* from = q0 + i == 0 || !real ? part0 : part1 + (q0 + i - 1) * step;
      m[i] = real ? __ldcg(from + 128 * D) : -INFINITY;
      u[i] = real ? __ldcg(from + 128 * D + 128) : 0.f;
#pragma unroll
      for (int c = 0; c < kColumns; ++c) x[i][c] = real ? __ldcg(from + (c0 + c) * 128) : 0.f;
    }
    float high = top;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) high = fmaxf(high, m[i]);
    const float base = high == -INFINITY ? 0.f : high, keep = exp2_approx(top - base);
    top = high;
    l *= keep;
#pragma unroll
    for (int c = 0; c < kColumns; ++c) o[c] *= keep;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const float f = exp2_approx(m[i] - base);
      l += f * u[i];
#pragma unroll
      for (int c = 0; c < kColumns; ++c) o[c] += f * x[i][c];
    }
  }
  if constexpr (kGroups > 1) {
    if (g > 0) {
#pragma unroll
      for (int c = 0; c < kColumns; ++c) others[g - 1][c][r] = o[c];
      others[g - 1][kColumns][r] = top;
      others[g - 1][kColumns + 1][r] = l;
    }
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float m = others[k][kColumns][r], high = fmaxf(top, m), base = high == -INFINITY ? 0.f : high;
      const float keep = exp2_approx(top - base), f = exp2_approx(m - base);
      top = high;
      l = l * keep + f * others[k][kColumns + 1][r];
#pragma unroll
      for (int c = 0; c < kColumns; ++c) o[c] = o[c] * keep + f * others[k][c][r];
    }
  }
  if (r >= rows) return;
  const RowOf ro = row_of(a, kvh, row0 + r);
  const bool empty = idle || up < -1 || up >= ro.node || l == 0.f;
  const float inv = empty ? 0.f : 1.f / l;
  const size_t at = (static_cast<size_t>(b) * a.nodes + ro.node) * a.heads + ro.head;
  T* out = static_cast<T*>(a.out) + at * D;
#pragma unroll
  for (int c = 0; c < kColumns; c += 8) {
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(empty ? 0.f : o[c + i] * inv);
    *reinterpret_cast<uint4*>(out + c0 + c) = *reinterpret_cast<const uint4*>(t);
  }
  if (c0 == 0) a.lse[at] = empty ? -INFINITY : (top + log2f(l)) * kLn2;
}

// The join as a launch of its own: in the main launch one block reads all
// parts of an item after everybody else has left, here the whole GPU does.
// Block (x, y): an item and row block, or, where there are more of those than
// the main launch had blocks, the item that a run begins inside of, if it is
// the first run to do so. y is a row, whose parts the block's groups of D / 4
// threads share out (kRows of 16 or 64), or kColumns columns of all 128 rows.
template <typename T, int kRows, int D, int kTile, int kGap, int kColumns, int kGroup, int kThreads>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ AttendArgs a, int row_blocks,
                                                        int block_rows, int runs) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int scratch[2 * kWarps + 6];
  __shared__ int sums[2][kWarps];
  const int tid = threadIdx.x, team = blockIdx.x / row_blocks;
  const Rows w{static_cast<int>(blockIdx.x) - team * row_blocks, row_blocks};
  Line line;
  Cursor cur = {};
  int p0 = 0, n = 1;
  if (gridDim.x == runs * row_blocks) {
    if (find_run<kTile, kGap, kThreads>(a, runs, team, scratch, &line, &cur) && cur.t > 0) {
      p0 = line.run_of(cur.first);
      if (team == p0 + 1) n = line.run_of(cur.first + cur.nt - 1) - p0 + 1;
    }
  } else {
    cur.b = team / a.c.kv_heads;
    cur.item = team - cur.b * a.c.kv_heads;
    int before = 0, all = 0;   // places of the sequences before b, and of all
    for (int i = tid; i < a.c.batch; i += kThreads) {
      const int places = (tiles_of<kTile>(sequence_span(a.c, i, a.nodes)) + kGap) * a.c.kv_heads;
      all += places;
      if (i < cur.b) before += places;
    }
    before = __reduce_add_sync(~0u, before);
    all = __reduce_add_sync(~0u, all);
    if (tid % 32 == 0) sums[0][tid / 32] = before, sums[1][tid / 32] = all;
    __syncthreads();
    cur.span = sequence_span(a.c, cur.b, a.nodes);
    cur.nt = tiles_of<kTile>(cur.span);
    before = all = 0;
    for (int i = 0; i < kWarps; ++i) before += sums[0][i], all += sums[1][i];
    cur.first = before + cur.item * (cur.nt + kGap);
    line.cut(all, runs, 0);
    p0 = line.run_of(cur.first);
    n = line.run_of(cur.first + cur.nt - 1) - p0 + 1;
  }
  const int first = cur.first, nt = cur.nt, b = cur.b, kvh = cur.item, row0 = w.rb * block_rows;
  const int rows = min(block_rows, a.nodes * a.group - row0);
  const Span span = cur.span;
  const int my_row = kRows == 128 ? tid % 128 : blockIdx.y;
  const int up = n > 1 && my_row < rows ? __ldcg(a.parents + b * a.stride_parents + (row0 + my_row) / a.group) : -2;
  // Lengths and parents (from L2) are older than the main launch, which let
  // this one begin only after its own wait for what came before it.
  chain();
  if (n == 1) return;   // whole, or another block's
  if constexpr (kRows == 128) {
    join_row<T, D, kColumns, kGroup, kThreads>(a, line, w, b, kvh, row0, rows, blockIdx.y * kColumns, first, nt,
                                               span.context < 0, up);
  } else {
    constexpr int kLanes = D / 4, kGroups = kThreads / kLanes, kAhead = 6;
    constexpr size_t kPart = kPartFloats<kRows, D>;
    __shared__ float4 others[kGroups][kLanes];
    __shared__ float tops[kGroups], ls[kGroups];
    const int r = blockIdx.y, g = tid / kLanes, e = tid % kLanes * 4;
    if (r >= rows) return;
    const float* part0 = a.partials + part_index(line, w, p0, first) * kPart;
    const float* part1 = a.partials + 2 * (static_cast<size_t>(p0 + 1) * row_blocks + w.rb) * kPart;
    const size_t step = 2 * static_cast<size_t>(row_blocks) * kPart;
    float top = -INFINITY, l = 0.f;
    float4 o = {0.f, 0.f, 0.f, 0.f};
    for (int q0 = g; q0 < n; q0 += kGroups * kAhead) {
      float m[kAhead], u[kAhead];
      float4 x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int p = q0 + i * kGroups;
        const float* part = p == 0 ? part0 : part1 + (p - 1) * step;
        m[i] = p < n ? __ldcg(part + kRows * D + r) : -INFINITY;
        u[i] = p < n ? __ldcg(part + kRows * D + kRows + r) : 0.f;
        x[i] = p < n ? __ldcg(reinterpret_cast<const float4*>(part + r * D + e)) : float4{0.f, 0.f, 0.f, 0.f};
      }
      float high = top;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) high = fmaxf(high, m[i]);
      const float base = high == -INFINITY ? 0.f : high, keep = exp2_approx(top - base);
      top = high;
      l *= keep, o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float f = exp2_approx(m[i] - base);
        l += f * u[i], o.x += f * x[i].x, o.y += f * x[i].y, o.z += f * x[i].z, o.w += f * x[i].w;
      }
    }
    others[g][tid % kLanes] = o;
    if (e == 0) tops[g] = top, ls[g] = l;
    __syncthreads();
    if (g > 0) return;
    for (int k = 1; k < kGroups; ++k) top = fmaxf(top, tops[k]);
    const float base = top == -INFINITY ? 0.f : top;
    l = 0.f, o = float4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < kGroups; ++k) {
      const float f = exp2_approx(tops[k] - base);
      const float4 x = others[k][tid % kLanes];
      l += f * ls[k], o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
    }
    const RowOf ro = row_of(a, kvh, row0 + r);
    const bool empty = span.context < 0 || up < -1 || up >= ro.node || l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    const size_t out_at = (static_cast<size_t>(b) * a.nodes + ro.node) * a.heads + ro.head;
    const float y[4] = {o.x, o.y, o.z, o.w};
    alignas(8) T t[4];
    for (int i = 0; i < 4; ++i) t[i] = from_f32<T>(empty ? 0.f : y[i] * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + out_at * D + e) = *reinterpret_cast<const uint2*>(t);
    if (e == 0) a.lse[out_at] = empty ? -INFINITY : (top + log2f(l)) * kLn2;
  }
}

template <typename T, int kRows, int D, int kTile, int kGap, int kColumns, int kGroup, int kThreads>
cudaError_t launch_join_as(const AttendArgs& a, int runs, int row_blocks, int block_rows, cudaStream_t s) {
  const dim3 grid(std::min(a.c.batch * a.c.kv_heads, runs) * row_blocks,
                  kRows == 128 ? D / kColumns : std::min(block_rows, a.nodes * a.group));
  return launch_chained(join_kernel<T, kRows, D, kTile, kGap, kColumns, kGroup, kThreads>, grid, dim3(kThreads), 0, 1,
                        s, a, row_blocks, block_rows, runs);
}

// Parts of an item where the lengths are alike: its share of the runs, or its
// tiles if the page table has room for fewer.
inline int64_t parts_of(const AttendArgs& a, int runs, int tile) {
  const int64_t tiles = (static_cast<int64_t>(a.c.table_width) * a.c.page_size + tile - 1) / tile;
  return std::min<int64_t>(runs / (static_cast<int64_t>(a.c.batch) * a.c.kv_heads), tiles);
}

// The more parts an item has, the more of them are read at once. Whole calls,
// us, D = 128, rows of 16: 304 parts 15.4 with blocks of 512 threads, 17.2
// with 256, 23.5 with 128; 38 parts 15.2, 14.9, 16.0. Rows of 128: 152 parts
// 21.6, 28.5, 42.5; 19 parts 41.9, 43.0, 44.1; 9 parts 25.2, 22.3, 23.2; 6
// parts 89.7, 83.0, 80.9; 3 parts 56.1 with 8 columns a block, 51.6 with 32.
template <typename T, int kRows, int D, int kTile, int kGap>
cudaError_t launch_join(const AttendArgs& a, int runs, int row_blocks, int block_rows, cudaStream_t s) {
  const int64_t parts = parts_of(a, runs, kTile);
  if constexpr (kRows < 128) {
    if (parts < 64) return launch_join_as<T, kRows, D, kTile, kGap, 8, 8, 256>(a, runs, row_blocks, block_rows, s);
    return launch_join_as<T, kRows, D, kTile, kGap, 8, 8, 512>(a, runs, row_blocks, block_rows, s);
  } else {
    if (parts < 4) return launch_join_as<T, kRows, D, kTile, kGap, 32, 2, 128>(a, runs, row_blocks, block_rows, s);
    if (parts < 16) return launch_join_as<T, kRows, D, kTile, kGap, 8, 8, 128>(a, runs, row_blocks, block_rows, s);
    return launch_join_as<T, kRows, D, kTile, kGap, 8, 8, 512>(a, runs, row_blocks, block_rows, s);
  }
}

}  // namespace tfx
