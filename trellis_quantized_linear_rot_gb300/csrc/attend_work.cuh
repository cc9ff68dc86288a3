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

// The line of tiles (below 2^31: checked on the host) and this block's run of
// it: the first `longer` runs have per + 1 tiles, the others per. No more
// runs than tiles, so that no run between two others is empty.
struct Line {
  int blocks, per, longer;
  int begin, end;
  __device__ __forceinline__ void cut(int total, int launched) {
    blocks = min(total, launched);
    per = total / blocks;
    longer = total - per * blocks;
    const int i = min(static_cast<int>(blockIdx.x), blocks);
    begin = begin_of(i);
    end = i < blocks ? begin_of(i + 1) : begin;
  }
  __device__ __forceinline__ int begin_of(int block) const { return block * per + min(block, longer); }
  // The block whose run holds tile f.
  __device__ __forceinline__ int block_of(int f) const {
    const int border = longer * (per + 1);
    return f < border ? f / (per + 1) : longer + (f - border) / per;
  }
};

// Position of a tile: item `item` (kv head, row block) of sequence b, tile t
// of its nt. first = place of the item's tile 0 in the line.
struct Cursor {
  int b, item, t, nt;
  int first;
  Span span;
};

template <int kTile>
__device__ __forceinline__ int tiles_of(const Span& s) {
  return s.slots <= kTile ? 1 : (s.slots + kTile - 1) / kTile;
}

// Block-wide: the line, this block's run and the cursor at its begin.
// `scratch` has room for kThreads / 32 + 2 ints. False where the run is
// empty. Batches of up to kThreads sequences are scanned once, larger ones
// twice (length, then place).
template <int kTile, int kThreads>
__device__ bool find_run(const AttendArgs& a, int items, int* scratch, Line* line, Cursor* cur) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int batch = a.c.batch;
  int* found = scratch + kWarps;   // [0] first tile of the sequence, [1] sequence
  for (int pass = batch <= kThreads ? 1 : 0; pass < 2; ++pass) {
    int before = 0;
    for (int b0 = 0; b0 < batch; b0 += kThreads) {
      const int b = b0 + tid;
      const int n = b < batch ? tiles_of<kTile>(sequence_span(a.c, b, a.nodes)) * items : 0;
      int run = n;
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += y;
      }
      if (lane == 31) scratch[warp] = run;
      __syncthreads();
      int prior = before, all = before;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) prior += scratch[w];
        all += scratch[w];
      }
      run += prior;
      if (b0 + kThreads >= batch && (pass == 0 || batch <= kThreads)) line->cut(all, gridDim.x);
      if (pass == 1 && line->begin >= run - n && line->begin < run) {
        found[0] = run - n;
        found[1] = b;
      }
      before = all;
      __syncthreads();
    }
  }
  if (line->begin >= line->end) return false;
  cur->b = found[1];
  cur->span = sequence_span(a.c, cur->b, a.nodes);
  cur->nt = tiles_of<kTile>(cur->span);
  const int in = line->begin - found[0];
  cur->item = in / cur->nt;
  cur->t = in - cur->item * cur->nt;
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

// Place of a block's part of the item at `first`. A block has two parts in
// the workspace: of the item its run begins in, and of a later item it ends
// in. A part is kRows rows of D sums, kRows maxima (in units of log 2) and
// kRows sums of weights.
__device__ __forceinline__ int part_index(const Line& l, int block, int first) {
  return 2 * block + (l.begin_of(block) < first ? 1 : 0);
}
template <int kRows, int D>
constexpr size_t kPartFloats = static_cast<size_t>(kRows) * (D + 2);

// Counts this block's part of the item (nt tiles from `first`); true in the
// block that arrives last. An item cut between blocks is counted at the place
// of its first part, so that the counters' number does not depend on the
// call's sizes and a workspace serves any of them.
__device__ __forceinline__ bool arrives_last(const AttendArgs& a, const Line& l, int first, int nt) {
  const int b0 = l.block_of(first), parts = l.block_of(first + nt - 1) - b0 + 1;
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

// kThreads threads (this one is number tid): joins the parts of the item at `first` (nt tiles) and writes
// rows row0 .. row0 + rows - 1 of its kv head. Parts are added in run order.
template <typename T, int kRows, int D, int kThreads, typename Masks>
__device__ void join_parts(const AttendArgs& a, const Line& line, const Masks& masks, int b, int kvh, int row0,
                           int rows, int first, int nt, bool idle, int tid) {
  constexpr size_t kPart = kPartFloats<kRows, D>;
  const int b0 = line.block_of(first), n = line.block_of(first + nt - 1) - b0 + 1;
  // Every part but the first is the one its block begins with.
  const float* part0 = a.partials + part_index(line, b0, first) * kPart;
  const float* part1 = a.partials + 2 * static_cast<size_t>(b0 + 1) * kPart;
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
    for (int p0 = 0; p0 < n; p0 += kGroup) {
      float m[kBatch][kGroup], w[kBatch][kGroup];
      float4 x[kBatch][kGroup];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const float* part = p0 + i == 0 ? part0 : part1 + (p0 + i - 1) * 2 * kPart;
          const int r = r0 + k * kStep;
          const bool real = p0 + i < n && r < rows;
          m[k][i] = real ? __ldcg(part + kRows * D + r) : -INFINITY;
          w[k][i] = real ? __ldcg(part + kRows * D + kRows + r) : 0.f;
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
          l[k] += f * w[k][i];
          o[k].x += f * x[k][i].x, o[k].y += f * x[k][i].y, o[k].z += f * x[k][i].z, o[k].w += f * x[k][i].w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kStep;
      if (r >= rows) continue;
      const RowOf ro = row_of(a, kvh, row0 + r);
      const bool present = !idle && masks.sees(ro.node, ro.node);
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

}  // namespace tfx
