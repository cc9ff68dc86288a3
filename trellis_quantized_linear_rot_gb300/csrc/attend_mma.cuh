// Tree attention with mma.sync: up to 16 rows a kv head (kRowWarps = 1), and
// blocks of 64 rows where the tcgen05 kernel does not apply (kRowWarps = 4).
//
// What bounds it is reading the cache: one token of 5 heads a kv head does
// 20 operations a byte. So everything serves to keep loads in flight: four
// warps, two or more blocks an SM, a ring of kStages tiles of keys and values
// filled by 16-byte asynchronous copies (any page size and any stride: each
// key's offset is looked up one tile ahead), and a ring that runs on across
// items. With 16 rows the warps take different keys of a tile, each with its
// own running maximum and sum, joined once an item; with 64 rows they take
// different rows.
//
// 32 tokens of 8 x 5 heads of 128 over up to 8,192 slots: 115 us for 684 MB,
// 5.9 TB/s, 0.87 of a copy's rate. One token over 300 slots: 8.7 us, all of it
// latency (lengths, page numbers, keys, the join, one after the other).
//
// Softmax in units of log 2: p = 2^(s - m), s = (q . k) scale log2(e).
// Scores, maxima, sums and accumulators are fp32; the weights are rounded to
// the dtype for the second product (what the matrix instruction takes), the
// sum uses them unrounded.
#pragma once

#include <type_traits>

#include "attend_work.cuh"

namespace tfx {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(__half, float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Not finite: all exponent bits set (either half of the word).
template <typename T>
__device__ __forceinline__ bool bad16(uint16_t x) {
  constexpr uint16_t m = std::is_same<T, __half>::value ? 0x7C00 : 0x7F80;
  return (x & m) == m;
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Whether either half of a word is not finite.
template <typename T>
__device__ __forceinline__ uint32_t bad_pair(uint32_t x) {
  constexpr uint32_t m = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
  const uint32_t y = ~x & m;   // a half is bad when none of its exponent bits is clear
  return (y & 0xFFFFu) == 0 || (y >> 16) == 0;
}

template <int D, int kRowWarps>
struct MmaShape {
  static constexpr int kThreads = 128;
  static constexpr int kRows = 16 * kRowWarps;
  static constexpr int kKeyWarps = 4 / kRowWarps;
  static constexpr int kTile = D == 256 ? 32 : 64;
  static constexpr int kGap = 1;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kHalf = kTile * kRowBytes;   // keys or values of a tile
  static constexpr int kStages = kRowWarps == 1 ? (D == 64 ? 5 : 3) : (D == 64 ? 3 : 2);
  static constexpr int kQBytes = kRows * kRowBytes;
  // A row block has at least a row a node, and more than 16 rows may have any
  // number of nodes.
  static constexpr int kNodes = kRowWarps == 1 ? 16 : TF_MAX_NODES;
  // A row block's q and parents come with the copies of its first tile, into
  // the places of that tile's stage, and go to registers when the item begins;
  // with D = 256 q stays in shared memory, in a place of its own.
  static constexpr int kQPlaces = kStages + (D == 256 ? 1 : 0);
  static constexpr int kSmem = kStages * 2 * kHalf + kQPlaces * kQBytes + kStages * kNodes * 4;
  // The warps' sums are joined in a stage whose tile is done with, kJoinCols
  // columns at a time.
  static constexpr int kJoinCols = 2 * kHalf / (kKeyWarps * kRows * 4) < D ? 2 * kHalf / (kKeyWarps * kRows * 4) : D;
};

template <typename T, int D, int kRowWarps>
__global__ void __launch_bounds__(128, D == 256 ? 1 : 2)
tree_attention_mma_kernel(const __grid_constant__ AttendArgs a) {
  using S = MmaShape<D, kRowWarps>;
  constexpr int kThreads = S::kThreads, kRows = S::kRows, kTile = S::kTile, kStages = S::kStages;
  constexpr int kKeys = kTile / S::kKeyWarps;   // keys of a tile a warp takes
  constexpr int kN = kKeys / 8;                 // its 8-key blocks
  constexpr int kChunks = D / 8;
  constexpr int kRing = kStages + 1;            // tiles whose offsets are known
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ TreeMasks<S::kNodes> masks;
  __shared__ int scratch[2 * (kThreads / 32) + 6];
  __shared__ int64_t at[kRing][kTile];
  __shared__ float wm[4][16], wl[4][16];
  __shared__ uint32_t bad[kTile / 32];          // keys of this tile with values that are not finite
  __shared__ uint32_t gone[kRing][kTile / 32];  // keys whose page is outside the pool
  __shared__ int last_here;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int row_warp = warp % kRowWarps, key_warp = warp / kRowWarps;
  const int rows_all = a.nodes * a.group;
  const int row_blocks = (rows_all + kRows - 1) / kRows, team = blockIdx.x / row_blocks;
  const Rows mine{static_cast<int>(blockIdx.x) - team * row_blocks, row_blocks};

  chain();
  Line line;
  Cursor look;   // next tile whose offsets are looked up
  const int n_tiles = find_run<kTile, S::kGap, kThreads>(a, gridDim.x / row_blocks, team, scratch, &line, &look);
  if (n_tiles == 0) return;
  Cursor cur = look, load = look;   // tiles computed and copied next
  const uint32_t ring = smem_u32(smem);
  const uint32_t q_ring = ring + kStages * 2 * S::kHalf;
  const uint32_t p_ring = q_ring + S::kQPlaces * S::kQBytes;
  const int* parents_ring = reinterpret_cast<const int*>(smem + kStages * 2 * S::kHalf + S::kQPlaces * S::kQBytes);
  const T* kp = static_cast<const T*>(a.k);
  const T* vp = static_cast<const T*>(a.v);

  // The page of this thread's key of the tile at cursor c is asked for early
  // (look_up), and its offset put in the ring for tile i later (settle; whole
  // warps call it): -1 for a slot that is not there.
  struct Pending {
    int page, row, kvh;
    bool exists;
  };
  auto look_up = [&](const Cursor& c) -> Pending {
    const int slot = c.t * kTile + tid, p = a.c.by_page(slot);
    const bool exists = slot < c.span.slots;
    return {exists ? a.c.page_table[c.b * a.c.stride_table + p] : 0, slot - p * a.c.page_size, c.item, exists};
  };
  auto settle = [&](const Pending& x, int i) {
    const bool outside = x.exists && static_cast<unsigned>(x.page) >= static_cast<unsigned>(a.c.pages);
    const uint32_t none = __ballot_sync(~0u, outside);
    if (lane == 0) gone[i % kRing][warp] = none;
    if (none && outside) record_index_error(a.c.err);
    at[i % kRing][tid] = x.exists && !outside ? x.page * a.c.stride_page + x.row * a.c.stride_token +
                                                    x.kvh * a.c.stride_head
                                              : -1;
  };
  // Copies of q and of the parents for the item of tile i (at cursor c).
  auto issue_rows = [&](const Cursor& c, int i) {
    const int h = c.item, first_row = mine.rb * kRows;
    const uint32_t dst = q_ring + (i % kStages) * S::kQBytes;
    for (int id = tid; id < kRows * kChunks; id += kThreads) {
      const int r = id / kChunks, ch = id % kChunks;
      const bool real = first_row + r < rows_all;
      const RowOf ro = row_of(a, h, real ? first_row + r : 0);
      copy16(dst + r * S::kRowBytes + ((ch ^ (r & 7)) << 4),
             static_cast<const T*>(a.q) + c.b * a.q_seq + ro.node * a.q_node + ro.head * a.q_head + ch * 8, real);
    }
    if (tid < a.nodes) copy4(p_ring + ((i % kStages) * S::kNodes + tid) * 4, a.parents + c.b * a.stride_parents + tid);
  };
  // Copies of tile i of the run.
  auto issue = [&](int i) {
    const uint32_t dst = ring + (i % kStages) * 2 * S::kHalf;
#pragma unroll
    for (int n = 0; n < kTile * kChunks / kThreads; ++n) {
      const int id = n * kThreads + tid, key = id / kChunks, ch = id % kChunks;
      const int64_t o = at[i % kRing][key];
      const uint32_t d = dst + key * S::kRowBytes + ((ch ^ (key & 7)) << 4);
      copy16(d, kp + (o < 0 ? 0 : o + ch * 8), o >= 0);
      copy16(d + S::kHalf, vp + (o < 0 ? 0 : o + ch * 8), o >= 0);
    }
  };

  // Fill the ring: q of the first item, the offsets of the first kStages
  // tiles, the copies of all but the last of them.
  issue_rows(cur, 0);
  Pending first[kStages];
#pragma unroll
  for (int i = 0; i < kStages; ++i)
    if (i < n_tiles) {
      if (tid < kTile) first[i] = look_up(look);
      advance<kTile, S::kGap>(a, &look);
    }
#pragma unroll
  for (int i = 0; i < kStages; ++i)
    if (i < n_tiles && tid < kTile) settle(first[i], i);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < n_tiles) {
      if (i > 0 && load.t == 0) issue_rows(load, i);
      issue(i);
      advance<kTile, S::kGap>(a, &load);
    }
    copies_commit();
  }

  uint32_t qf[D == 256 ? 1 : D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];
  const int row0 = mine.rb * kRows;
  int kvh = 0;
  int node[2];
  const uint32_t q_at = q_ring + kStages * S::kQBytes;   // D = 256 only
  bool fresh = true;
  const float sc = a.scale * kLog2e;

#pragma unroll 1
  for (int i = 0; i < n_tiles; ++i) {
    copies_wait<kStages - 2>();
    __syncthreads();   // tile i has landed; everyone is done with tile i - 1
    if (i + kStages - 1 < n_tiles) {
      if (load.t == 0) issue_rows(load, i + kStages - 1);
      issue(i + kStages - 1);
      advance<kTile, S::kGap>(a, &load);
    }
    copies_commit();
    const bool more = i + kStages < n_tiles;
    Pending next = {};
    if (more && tid < kTile) next = look_up(look);   // settled after this tile
    if (more) advance<kTile, S::kGap>(a, &look);

    if (fresh) {   // a new item: its rows of q, its masks
      kvh = cur.item;
      const uint32_t q_new = q_ring + (i % kStages) * S::kQBytes;
      if constexpr (D == 256) {
        unsigned char* q8 = smem + kStages * 2 * S::kHalf;
        for (int id = tid; id < S::kQBytes / 16; id += kThreads)
          reinterpret_cast<uint4*>(q8 + kStages * S::kQBytes)[id] =
              reinterpret_cast<const uint4*>(q8 + (i % kStages) * S::kQBytes)[id];
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int r = row_warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
          ldsm4(qf[ks], q_new + r * S::kRowBytes + (((ks * 2 + (lane >> 4)) ^ (r & 7)) << 4));
        }
      }
      masks.build(parents_ring + (i % kStages) * S::kNodes, a.nodes, a.c.err);
#pragma unroll
      for (int e = 0; e < D / 8; ++e)
        for (int x = 0; x < 4; ++x) o[e][x] = 0.f;
      for (int x = 0; x < 2; ++x) {
        const int r = row0 + row_warp * 16 + lane / 4 + x * 8;
        m[x] = -INFINITY, l[x] = 0.f;
        node[x] = r < rows_all ? r / a.group : -1;
      }
      fresh = false;
    }

    const uint32_t kt = ring + (i % kStages) * 2 * S::kHalf, vt = kt + S::kHalf;
    const int slot0 = cur.t * kTile;
    uint32_t missing = 0;
    for (int x = 0; x < kTile / 32; ++x) missing |= gone[i % kRing][x];
    const bool tail = slot0 + kTile > cur.span.context || missing;
    bool any_bad = false;
    // Values of tree nodes that are not finite must not reach the rows that do
    // not see them (0 times infinity): they are set to 0 here and added after
    // the product to the rows that do. The only node is seen by every row.
    if (tail && a.nodes > 1) {
      if (tid < kTile / 32) bad[tid] = 0;
      __syncthreads();
      unsigned char* v8 = smem + (i % kStages) * 2 * S::kHalf + S::kHalf;
      const int j0 = max(0, cur.span.context - slot0), j1 = min(kTile, cur.span.slots - slot0);
      for (int id = j0 * kChunks + tid; id < j1 * kChunks; id += kThreads) {
        const int key = id / kChunks, ch = id % kChunks;
        uint4* w = reinterpret_cast<uint4*>(v8 + key * S::kRowBytes + ((ch ^ (key & 7)) << 4));
        const uint4 x = *w;
        if (bad_pair<T>(x.x) | bad_pair<T>(x.y) | bad_pair<T>(x.z) | bad_pair<T>(x.w)) {
          uint16_t* h = reinterpret_cast<uint16_t*>(w);
          for (int y = 0; y < 8; ++y)
            if (bad16<T>(h[y])) h[y] = 0;
          atomicOr(&bad[key / 32], 1u << (key % 32));
        }
      }
      __syncthreads();
      for (int x = 0; x < kTile / 32; ++x) any_bad |= bad[x] != 0;
    }

    float s[kN][4];
#pragma unroll
    for (int n = 0; n < kN; ++n)
      for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t qa[4];
      if constexpr (D == 256) {
        const int r = row_warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
        ldsm4(qa, q_at + r * S::kRowBytes + (((ks * 2 + (lane >> 4)) ^ (r & 7)) << 4));
      } else {
        for (int x = 0; x < 4; ++x) qa[x] = qf[ks][x];
      }
#pragma unroll
      for (int n = 0; n < kN; n += 2) {
        uint32_t b[4];
        const int key = key_warp * kKeys + n * 8 + (lane >> 4) * 8 * (kN > 1) + (lane & 7);
        ldsm4(b, kt + key * S::kRowBytes + (((ks * 2 + ((lane >> 3) & 1)) ^ (key & 7)) << 4));
        mma16816<T>(s[n], qa, b[0], b[1]);
        if (kN > 1) mma16816<T>(s[n + (kN > 1)], qa, b[2], b[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s[n][x] *= sc;
        if (tail) {
          const int key = key_warp * kKeys + n * 8 + (lane % 4) * 2 + (x & 1), slot = slot0 + key;
          const int i_row = node[x >> 1], j = slot - cur.span.context;
          bool sees = slot < cur.span.slots && i_row >= 0;
          if (sees && j >= 0) sees = masks.sees(i_row, j);
          if (!sees || (gone[i % kRing][key / 32] >> (key % 32) & 1)) s[n][x] = -INFINITY;
        }
      }
    uint32_t p[kN][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float top = m[x];
#pragma unroll
      for (int n = 0; n < kN; ++n) top = fmaxf(top, fmaxf(s[n][2 * x], s[n][2 * x + 1]));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      const float base = top == -INFINITY ? 0.f : top;
      const float keep = exp2_approx(m[x] - base);
      m[x] = top;
      l[x] *= keep;
#pragma unroll
      for (int e = 0; e < D / 8; ++e) o[e][2 * x] *= keep, o[e][2 * x + 1] *= keep;
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const float p0 = exp2_approx(s[n][2 * x] - base), p1 = exp2_approx(s[n][2 * x + 1] - base);
        l[x] += p0 + p1;
        p[n][x] = pack2(T(), p0, p1);
      }
    }
#pragma unroll
    for (int n = 0; n < kN; n += 2) {
      const uint32_t pa[4] = {p[n][0], p[n][1], kN > 1 ? p[n + (kN > 1)][0] : 0u, kN > 1 ? p[n + (kN > 1)][1] : 0u};
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        uint32_t b[4];
        const int key = key_warp * kKeys + n * 8 + ((lane >> 3) & 1) * 8 * (kN > 1) + (lane & 7);
        ldsm4_t(b, vt + key * S::kRowBytes + (((e * 2 + (lane >> 4)) ^ (key & 7)) << 4));
        mma16816<T>(o[2 * e], pa, b[0], kN > 1 ? b[1] : 0u);
        mma16816<T>(o[2 * e + 1], pa, b[2], kN > 1 ? b[3] : 0u);
      }
    }
    if (any_bad) {
      for (int key = key_warp * kKeys; key < (key_warp + 1) * kKeys; ++key) {
        if (!(bad[key / 32] >> (key % 32) & 1)) continue;
        const int j = slot0 + key - cur.span.context;
        const int64_t off = slot_offset(a.c, cur.b, slot0 + key);
        if (off < 0) continue;
        const T* row = vp + off + static_cast<int64_t>(kvh) * a.c.stride_head;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (node[x] < 0 || !masks.sees(node[x], j)) continue;
#pragma unroll
          for (int e = 0; e < D / 8; ++e)
            for (int y = 0; y < 2; ++y) {
              const T w = row[e * 8 + (lane % 4) * 2 + y];
              if (bad16<T>(*reinterpret_cast<const uint16_t*>(&w))) o[e][2 * x + y] += to_f32(w);
            }
        }
      }
    }

    const bool item_ends = cur.t + 1 == cur.nt;
    if (item_ends || i + 1 == n_tiles) {
      const bool whole = item_ends && cur.first >= line.begin;
      const int rows = min(kRows, rows_all - row0);
      const bool idle = cur.span.context < 0;
      float* part = a.partials + part_index(line, mine, team, cur.first) * kPartFloats<kRows, D>;
      // Sums over the four lanes of a row, then over the warps with other keys.
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(~0u, l[x], 1);
        l[x] += __shfl_xor_sync(~0u, l[x], 2);
      }
      // Where a row's result goes: out and lse, or this block's part.
      auto finish = [&](int rl, float top, float sum, bool first, float* inv, T** out) {
        const RowOf ro = row_of(a, kvh, row0 + rl);
        const bool present = !idle && masks.sees(ro.node, ro.node);
        const bool empty = !present || sum == 0.f;
        *inv = empty ? 0.f : 1.f / sum;
        const size_t out_at = (static_cast<size_t>(cur.b) * a.nodes + ro.node) * a.heads + ro.head;
        *out = static_cast<T*>(a.out) + out_at * D;
        if (first) a.lse[out_at] = empty ? -INFINITY : (top + log2f(sum)) * kLn2;
      };
      if constexpr (S::kKeyWarps > 1) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (lane % 4 == 0) wm[warp][lane / 4 + x * 8] = m[x], wl[warp][lane / 4 + x * 8] = l[x];
        __syncthreads();   // and everyone is done with tile i
        float* sums = reinterpret_cast<float*>(smem + (i % kStages) * 2 * S::kHalf);
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = lane / 4 + x * 8;
          const float top = fmaxf(fmaxf(wm[0][r], wm[1][r]), fmaxf(wm[2][r], wm[3][r]));
          f[x] = exp2_approx(m[x] - (top == -INFINITY ? 0.f : top));
        }
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += S::kJoinCols) {
          if (c0) __syncthreads();
#pragma unroll
          for (int e = c0 / 8; e < (c0 + S::kJoinCols) / 8; ++e)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int r = lane / 4 + x * 8;
              // columns rotated by the row, so that a warp's rows lie in different banks
              const int col = (e * 8 - c0 + (lane % 4) * 2 + r * 8) % S::kJoinCols;
              *reinterpret_cast<float2*>(sums + (warp * 16 + r) * S::kJoinCols + col) =
                  float2{f[x] * o[e][2 * x], f[x] * o[e][2 * x + 1]};
            }
          __syncthreads();
          for (int id = tid; id < rows * (S::kJoinCols / 4); id += kThreads) {
            const int r = id / (S::kJoinCols / 4), e = (id - r * (S::kJoinCols / 4)) * 4;
            float4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float4 z = *reinterpret_cast<const float4*>(sums + (w * 16 + r) * S::kJoinCols +
                                                                (e + r * 8) % S::kJoinCols);
              y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
            }
            const float top = fmaxf(fmaxf(wm[0][r], wm[1][r]), fmaxf(wm[2][r], wm[3][r]));
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) sum += wl[w][r] * exp2_approx(wm[w][r] - base);
            if (whole) {
              float inv;
              T* out;
              finish(r, top, sum, c0 + e == 0, &inv, &out);
              const bool empty = inv == 0.f;
              const uint2 z = {empty ? 0u : pack2(T(), y.x * inv, y.y * inv),
                               empty ? 0u : pack2(T(), y.z * inv, y.w * inv)};
              *reinterpret_cast<uint2*>(out + c0 + e) = z;
            } else {
              *reinterpret_cast<float4*>(part + r * D + c0 + e) = y;
              if (c0 + e == 0) part[kRows * D + r] = top, part[kRows * D + kRows + r] = sum;
            }
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int rl = row_warp * 16 + lane / 4 + x * 8;
          if (rl >= rows) continue;
          float inv = 1.f;
          T* out = nullptr;
          if (whole) finish(rl, m[x], l[x], lane % 4 == 0, &inv, &out);
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            const int col = e * 8 + (lane % 4) * 2;
            if (whole)
              *reinterpret_cast<uint32_t*>(out + col) =
                  inv == 0.f ? 0u : pack2(T(), o[e][2 * x] * inv, o[e][2 * x + 1] * inv);
            else
              *reinterpret_cast<float2*>(part + rl * D + col) = float2{o[e][2 * x], o[e][2 * x + 1]};
          }
          if (!whole && lane % 4 == 0) part[kRows * D + rl] = m[x], part[kRows * D + kRows + rl] = l[x];
        }
      }
      if (!whole && !a.join_later) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          last_here = arrives_last(a, line, mine, cur.first, cur.nt);
          __threadfence();
        }
        __syncthreads();
        if (last_here)
          join_parts<T, kRows, D, kThreads>(a, line, mine, cur.b, kvh, row0, rows, cur.first, cur.nt, idle, tid);
      }
      fresh = true;
      __syncthreads();   // the masks and the stage may be written again
    }
    if (more && tid < kTile) settle(next, i + kStages);
    advance<kTile, S::kGap>(a, &cur);
  }
}

}  // namespace tfx
