// How the attention kernels divide their work, and how the parts of a row are
// joined.
//
// An item is one (sequence, kv head, block of rows): its rows all read the
// same keys. The tiles of all items, sequence by sequence, form one line that
// is cut into equal runs, one for each block of the launch, so that ragged
// lengths and few long sequences fill the GPU alike. Lengths are on the
// device, so every block finds its run itself. A run holds whole items but
// for its first and its last, which other blocks may share: those leave
// (max, sum, weighted sum) of their part in the workspace, and the block that
// arrives last at the item joins the parts in the order of the runs. No block
// waits for another.
#pragma once

#include "ptx.cuh"
#include "spec.cuh"

namespace tfx {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The line of tiles and this block's run of it.
struct Line {
  long long total;   // tiles of all items
  long long begin, end;
  int blocks;        // runs: blocks of the launch, at most one a tile
};

// Position of a tile: item `item` (kv head, row block) of sequence b, tile t
// of its nt. first = place of the item's tile 0 in the line.
struct Cursor {
  int b, item, t, nt;
  long long first;
  Span span;
};

template <int kTile>
__device__ __forceinline__ int tiles_of(const Span& s) {
  return s.slots <= kTile ? 1 : (s.slots + kTile - 1) / kTile;
}

// Block-wide: the line's length, this block's run and the cursor at its
// begin. `scratch` has room for kThreads / 32 + 3 long longs. False where the
// run is empty. Batches of up to kThreads sequences are scanned once, larger
// ones twice (length, then place).
template <int kTile, int kThreads>
__device__ bool find_run(const AttendArgs& a, int items, int blocks, long long* scratch, Line* line, Cursor* cur) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int batch = a.c.batch;
  long long* found = scratch + kWarps + 1;   // [0] first tile of the sequence, [1] sequence
  long long before = 0;
  // No more runs than tiles, so that no run between two others is empty.
  auto cut = [&](long long all) {
    line->total = all;
    line->blocks = all < blocks ? static_cast<int>(all) : blocks;
    const int i = min(static_cast<int>(blockIdx.x), line->blocks);
    line->begin = all * i / line->blocks;
    line->end = i < line->blocks ? all * (i + 1) / line->blocks : all;
  };
  for (int pass = 0; pass < 2; ++pass) {
    before = 0;
    for (int b0 = 0; b0 < batch; b0 += kThreads) {
      const int b = b0 + tid;
      long long n = 0;
      if (b < batch) n = static_cast<long long>(tiles_of<kTile>(sequence_span(a.c, b, a.nodes))) * items;
      long long run = n;
      for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += y;
      }
      if (lane == 31) scratch[warp] = run;
      __syncthreads();
      long long prior = before, all = before;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) prior += scratch[w];
        all += scratch[w];
      }
      run += prior;
      const bool last = b0 + kThreads >= batch;
      if (pass == 0 && last) cut(all);
      if ((pass == 1 || batch <= kThreads) && line->begin >= run - n && line->begin < run) {
        found[0] = run - n;
        found[1] = b;
      }
      before = all;
      __syncthreads();
    }
    if (batch <= kThreads) break;
  }
  if (line->begin >= line->end) return false;
  cur->b = static_cast<int>(found[1]);
  cur->span = sequence_span(a.c, cur->b, a.nodes);
  cur->nt = tiles_of<kTile>(cur->span);
  const long long in = line->begin - found[0];
  cur->item = static_cast<int>(in / cur->nt);
  cur->t = static_cast<int>(in - static_cast<long long>(cur->item) * cur->nt);
  cur->first = line->begin - cur->t;
  return true;
}

template <int kTile>
__device__ __forceinline__ void advance(const AttendArgs& a, int items, Cursor* c) {
  if (++c->t < c->nt) return;
  c->t = 0;
  c->first += c->nt;
  if (++c->item < items) return;
  c->item = 0;
  if (++c->b >= a.c.batch) return;
  c->span = sequence_span(a.c, c->b, a.nodes);
  c->nt = tiles_of<kTile>(c->span);
}

// The block whose run holds tile f of the line, and where its run begins.
__device__ __forceinline__ int block_of(const Line& l, long long f) {
  return static_cast<int>(((f + 1) * l.blocks - 1) / l.total);
}
__device__ __forceinline__ long long begin_of(const Line& l, int block) { return l.total * block / l.blocks; }

// Place of a block's part of the item at `first`.
__device__ __forceinline__ size_t part_index(const Line& l, int block, long long first) {
  return 2 * static_cast<size_t>(block) + (begin_of(l, block) < first ? 1 : 0);
}

// A block has two parts in the workspace: of the item its run begins in, and
// of a later item it ends in. A part is kRows rows of D sums, kRows maxima
// (in units of log 2) and kRows sums of weights.
template <int kRows, int D>
struct Part {
  static constexpr size_t kFloats = static_cast<size_t>(kRows) * (D + 2);
  static __device__ __forceinline__ float* at(const AttendArgs& a, const Line& l, int block, long long first) {
    return a.partials + part_index(l, block, first) * kFloats;
  }
};

// Counts this block's part of the item (nt tiles from `first`); true in the
// block that arrives last. An item cut between blocks is counted at the place
// of its first part, so that the counters' number does not depend on the
// call's sizes and a workspace serves any of them.
__device__ __forceinline__ bool arrives_last(const AttendArgs& a, const Line& l, long long first, int nt) {
  const int b0 = block_of(l, first), parts = block_of(l, first + nt - 1) - b0 + 1;
  int* counter = a.counters + part_index(l, b0, first);
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

// Whole block: joins the parts of the item at `first` (nt tiles) and writes
// rows row0 .. row0 + rows - 1 of its kv head. Parts are added in run order.
template <typename T, int kRows, int D, int kThreads>
__device__ void join_parts(const AttendArgs& a, const Line& line, const TreeMasks& masks, int b, int kvh, int row0,
                           int rows, long long first, int nt, bool idle) {
  const int b0 = block_of(line, first), b1 = block_of(line, first + nt - 1);
  for (int id = threadIdx.x; id < rows * (D / 4); id += kThreads) {
    const int r = id / (D / 4), e = (id - r * (D / 4)) * 4;
    float top = -INFINITY;
    for (int p = b0; p <= b1; ++p) top = fmaxf(top, __ldcg(Part<kRows, D>::at(a, line, p, first) + kRows * D + r));
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = b0; p <= b1; ++p) {
      const float* part = Part<kRows, D>::at(a, line, p, first);
      const float w = exp2_approx(__ldcg(part + kRows * D + r) - base);
      l += w * __ldcg(part + kRows * D + kRows + r);
      const float4 x = __ldcg(reinterpret_cast<const float4*>(part + r * D + e));
      o.x += w * x.x, o.y += w * x.y, o.z += w * x.z, o.w += w * x.w;
    }
    const RowOf ro = row_of(a, kvh, row0 + r);
    const bool present = !idle && (masks.anc[ro.node][ro.node >> 5] >> (ro.node & 31) & 1);
    const bool empty = !present || l == 0.f;
    const float inv = empty ? 0.f : 1.f / l;
    const size_t at = (static_cast<size_t>(b) * a.nodes + ro.node) * a.heads + ro.head;
    T* out = static_cast<T*>(a.out) + at * D + e;
    const float y[4] = {o.x, o.y, o.z, o.w};
    T t[4];
    for (int i = 0; i < 4; ++i) t[i] = from_f32<T>(empty ? 0.f : y[i] * inv);
    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(t);
    if (e == 0) a.lse[at] = empty ? -INFINITY : (top + log2f(l)) * kLn2;
  }
}

}  // namespace tfx
