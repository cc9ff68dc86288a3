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

template <int D, int kRowWarps>
struct MmaShape {
  static constexpr int kThreads = 128;
  static constexpr int kRows = 16 * kRowWarps;
  static constexpr int kKeyWarps = 4 / kRowWarps;
  static constexpr int kTile = D == 256 ? 32 : 64;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kHalf = kTile * kRowBytes;                       // keys or values of a tile
  static constexpr int kStages = kRowWarps == 1 ? (D == 64 ? 5 : 3) : (D == 64 ? 3 : 2);
  static constexpr int kJoinBytes = kKeyWarps > 1 ? kRows * D * 4 : 0;  // shared with the rows of q
  static constexpr int kQBytes = kRows * kRowBytes > kJoinBytes ? kRows * kRowBytes : kJoinBytes;
  static constexpr int kSmem = kStages * 2 * kHalf + kQBytes;
};

template <typename T, int D, int kRowWarps>
__global__ void __launch_bounds__(128, D == 256 ? 1 : 2) tree_attention_mma_kernel(const __grid_constant__ AttendArgs a) {
  using S = MmaShape<D, kRowWarps>;
  constexpr int kThreads = S::kThreads, kRows = S::kRows, kTile = S::kTile, kStages = S::kStages;
  constexpr int kKeys = kTile / S::kKeyWarps;   // keys of a tile a warp takes
  constexpr int kN = kKeys / 8;                 // its 8-key blocks
  constexpr int kChunks = D / 8;
  static_assert(kKeys % 16 == 0 || kN == 1, "a warp takes whole 16-key steps");
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ TreeMasks masks;
  __shared__ long long scratch[kThreads / 32 + 3];
  __shared__ int64_t at[2][kTile];
  __shared__ float wm[4][16], wl[4][16];
  __shared__ uint32_t bad[kTile / 32];               // keys of this tile with values that are not finite
  __shared__ uint32_t gone[kStages + 1][kTile / 32];  // keys whose page is outside the pool
  __shared__ int last_here;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int row_warp = warp % kRowWarps, key_warp = warp / kRowWarps;
  const int rows_all = a.nodes * a.group;
  const int row_blocks = (rows_all + kRows - 1) / kRows;
  const int items = a.c.kv_heads * row_blocks;

  Line line;
  Cursor look;   // next tile whose offsets are looked up
  if (!find_run<kTile, kThreads>(a, items, gridDim.x, scratch, &line, &look)) return;
  Cursor cur = look;
  const uint32_t ring = smem_u32(smem);
  unsigned char* qs = smem + kStages * 2 * S::kHalf;
  const uint32_t q_at = ring + kStages * 2 * S::kHalf;
  const int n_tiles = static_cast<int>(line.end - line.begin);

  // Offset of this thread's key of tile i of the run (the cursor's), -1 for a
  // slot that is not there. Whole warps call it.
  auto offset_of = [&](const Cursor& c, int i) -> int64_t {
    const int slot = c.t * kTile + tid;
    const bool exists = slot < c.span.slots;
    const int64_t o = exists ? slot_offset(a.c, c.b, slot) : -1;
    const uint32_t none = __ballot_sync(~0u, exists && o < 0);
    if (lane == 0) gone[i % (kStages + 1)][warp] = none;
    return o < 0 ? -1 : o + static_cast<int64_t>(c.item / row_blocks) * a.c.stride_head;
  };
  const T* kp = static_cast<const T*>(a.k);
  const T* vp = static_cast<const T*>(a.v);
  auto issue = [&](int i) {   // copies of tile i of the run
    const uint32_t dst = ring + (i % kStages) * 2 * S::kHalf;
    for (int id = tid; id < kTile * kChunks; id += kThreads) {
      const int key = id / kChunks, ch = id % kChunks;
      const int64_t o = at[i & 1][key];
      const uint32_t d = dst + key * S::kRowBytes + ((ch ^ (key & 7)) << 4);
      copy16(d, kp + (o < 0 ? 0 : o + ch * 8), o >= 0);
      copy16(d + S::kHalf, vp + (o < 0 ? 0 : o + ch * 8), o >= 0);
    }
  };

  // Fill the ring: offsets of a tile, then its copies.
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < n_tiles) {
      if (tid < kTile) at[i & 1][tid] = offset_of(look, i);
      __syncthreads();
      issue(i);
      advance<kTile>(a, items, &look);
    }
    copies_commit();
  }
  if (kStages - 1 < n_tiles) {
    __syncthreads();
    if (tid < kTile) at[(kStages - 1) & 1][tid] = offset_of(look, kStages - 1);
    advance<kTile>(a, items, &look);
  }

  uint32_t qf[D == 256 ? 1 : D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];
  int kvh = 0, row0 = 0;
  int node[2];
  bool fresh = true;
  const float sc = a.scale * kLog2e;

#pragma unroll 1
  for (int i = 0; i < n_tiles; ++i) {
    if (fresh) {   // a new item: its rows of q, its masks
      kvh = cur.item / row_blocks;
      row0 = (cur.item - kvh * row_blocks) * kRows;
      __syncthreads();
      for (int id = tid; id < kRows * kChunks; id += kThreads) {
        const int r = id / kChunks, ch = id % kChunks;
        uint4 x = {0, 0, 0, 0};
        if (row0 + r < rows_all) {
          const RowOf ro = row_of(a, kvh, row0 + r);
          x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + cur.b * a.q_seq + ro.node * a.q_node +
                                              ro.head * a.q_head + ch * 8);
        }
        *reinterpret_cast<uint4*>(qs + r * S::kRowBytes + ((ch ^ (r & 7)) << 4)) = x;
      }
      build_tree_masks(masks, a.parents + cur.b * a.stride_parents, a.nodes, a.c.err);
      if constexpr (D != 256) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const int r = row_warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
          ldsm4(qf[ks], q_at + r * S::kRowBytes + (((ks * 2 + (lane >> 4)) ^ (r & 7)) << 4));
        }
      }
      for (int e = 0; e < D / 8; ++e)
        for (int x = 0; x < 4; ++x) o[e][x] = 0.f;
      for (int x = 0; x < 2; ++x) {
        const int r = row0 + row_warp * 16 + lane / 4 + x * 8;
        m[x] = -INFINITY, l[x] = 0.f;
        node[x] = r < rows_all ? r / a.group : -1;
      }
      fresh = false;
    }
    copies_wait<kStages - 2>();
    __syncthreads();   // tile i has landed; everyone is done with tile i - 1
    if (i + kStages - 1 < n_tiles) issue(i + kStages - 1);
    copies_commit();
    const bool more = i + kStages < n_tiles;
    int64_t next_at = -1;
    if (more && tid < kTile) next_at = offset_of(look, i + kStages);   // stored after this tile

    const uint32_t kt = ring + (i % kStages) * 2 * S::kHalf, vt = kt + S::kHalf;
    const int slot0 = cur.t * kTile;
    uint32_t missing = 0;
    for (int x = 0; x < kTile / 32; ++x) missing |= gone[i % (kStages + 1)][x];
    const bool tail = slot0 + kTile > cur.span.context || missing;
    bool any_bad = false;
    if (tail) {
      // Values of tree nodes that are not finite must not reach the rows that
      // do not see them (0 times infinity): they are set to 0 here and added
      // after the product to the rows that do.
      if (tid < kTile / 32) bad[tid] = 0;
      __syncthreads();
      unsigned char* v8 = smem + (i % kStages) * 2 * S::kHalf + S::kHalf;
      const int j0 = max(0, cur.span.context - slot0);
      for (int id = tid; id < (kTile - j0) * kChunks; id += kThreads) {
        const int key = j0 + id / kChunks, ch = id % kChunks;
        uint16_t* w = reinterpret_cast<uint16_t*>(v8 + key * S::kRowBytes + ((ch ^ (key & 7)) << 4));
        for (int x = 0; x < 8; ++x)
          if (bad16<T>(w[x])) {
            w[x] = 0;
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
          if (sees && j >= 0) sees = masks.anc[i_row][j >> 5] >> (j & 31) & 1;
          if (!sees || (gone[i % (kStages + 1)][key / 32] >> (key % 32) & 1)) s[n][x] = -INFINITY;
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
          if (node[x] < 0 || !(masks.anc[node[x]][j >> 5] >> (j & 31) & 1)) continue;
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
      // Sums over the four lanes of a row, then over the warps with other keys.
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(~0u, l[x], 1);
        l[x] += __shfl_xor_sync(~0u, l[x], 2);
      }
      float* sum = reinterpret_cast<float*>(qs);
      if constexpr (S::kKeyWarps > 1) {
        for (int x = 0; x < 2; ++x)
          if (lane % 4 == 0) wm[warp][lane / 4 + x * 8] = m[x], wl[warp][lane / 4 + x * 8] = l[x];
        __syncthreads();
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = lane / 4 + x * 8;
          float top = -INFINITY;
          for (int w = 0; w < 4; ++w) top = fmaxf(top, wm[w][r]);
          const float base = top == -INFINITY ? 0.f : top;
          f[x] = exp2_approx(m[x] - base);
          l[x] = 0.f;
          for (int w = 0; w < 4; ++w) l[x] += wl[w][r] * exp2_approx(wm[w][r] - base);
          m[x] = top;
        }
        for (int w = 0; w < 4; ++w) {
          if (warp == w)
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float2* to = reinterpret_cast<float2*>(sum + (lane / 4 + x * 8) * D + e * 8 + (lane % 4) * 2);
                float2 y = w ? *to : float2{0.f, 0.f};
                y.x += f[x] * o[e][2 * x];
                y.y += f[x] * o[e][2 * x + 1];
                *to = y;
              }
          __syncthreads();
        }
      }
      const bool whole = item_ends && cur.first >= line.begin;
      const int rows = min(kRows, rows_all - row0);
      const bool idle = cur.span.context < 0;
      if (whole) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int rl = row_warp * 16 + lane / 4 + x * 8;
          if (node[x] < 0) continue;
          const RowOf ro = row_of(a, kvh, row0 + rl);
          const bool present = !idle && (masks.anc[ro.node][ro.node >> 5] >> (ro.node & 31) & 1);
          const bool empty = !present || l[x] == 0.f;
          const float inv = empty ? 0.f : 1.f / l[x];
          const size_t out_at = (static_cast<size_t>(cur.b) * a.nodes + ro.node) * a.heads + ro.head;
          T* out = static_cast<T*>(a.out) + out_at * D;
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            if (S::kKeyWarps > 1 && e % S::kKeyWarps != key_warp) continue;
            const int col = e * 8 + (lane % 4) * 2;
            float y0 = o[e][2 * x], y1 = o[e][2 * x + 1];
            if (S::kKeyWarps > 1) y0 = sum[rl * D + col], y1 = sum[rl * D + col + 1];
            *reinterpret_cast<uint32_t*>(out + col) = empty ? 0u : pack2(T(), y0 * inv, y1 * inv);
          }
          if (lane % 4 == 0 && key_warp == 0) a.lse[out_at] = empty ? -INFINITY : (m[x] + log2f(l[x])) * kLn2;
        }
      } else {
        float* part = Part<kRows, D>::at(a, line, blockIdx.x, cur.first);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int rl = row_warp * 16 + lane / 4 + x * 8;
          if (rl >= rows) continue;
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            if (S::kKeyWarps > 1 && e % S::kKeyWarps != key_warp) continue;
            const int col = e * 8 + (lane % 4) * 2;
            float2 y = {o[e][2 * x], o[e][2 * x + 1]};
            if (S::kKeyWarps > 1) y = *reinterpret_cast<const float2*>(sum + rl * D + col);
            *reinterpret_cast<float2*>(part + rl * D + col) = y;
          }
          if (lane % 4 == 0 && key_warp == 0) part[kRows * D + rl] = m[x], part[kRows * D + kRows + rl] = l[x];
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          last_here = arrives_last(a, line, cur.first, cur.nt);
          __threadfence();
        }
        __syncthreads();
        if (last_here)
          join_parts<T, kRows, D, kThreads>(a, line, masks, cur.b, kvh, row0, rows, cur.first, cur.nt, idle);
      }
      fresh = true;
    }
    if (more && tid < kTile) at[(i + kStages) & 1][tid] = next_at;
    if (more) advance<kTile>(a, items, &look);
    advance<kTile>(a, items, &cur);
  }
}

}  // namespace tfx
