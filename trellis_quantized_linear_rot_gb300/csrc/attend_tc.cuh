// Tree attention with tcgen05: more than 16 rows a kv head.
//
// With R rows a kv head the call does R operations a byte of the cache. A tile
// of 128 rows costs the tensor cores about 1,000 cycles for 128 keys (two
// products of 128 x 128 x 128) whether its rows are used or not, and memory
// about 2,800 cycles (64 KB at this SM's share), so up to one full tile of
// rows the cache's bytes bound it, and with several the tensor cores (the
// exponentials, 128 x 128 a tile and 32 a cycle, take half as long).
//
// One block an SM, a run of tiles for each team of blocks, one block for each
// block of rows: whole nodes with at most 128 rows (attend_work.cuh). An
// item's key tiles go alternately to two streams, each with its own scores,
// weights, sums and running maximum in Tensor Memory and registers, so that
// one stream's products run while the other's exponentials do:
//   warp 0        copies of keys and values, a box for each page or part of
//                 one, three tiles in flight
//   warps 1, 2    products of stream 0 and 1: S = Q K^T into Tensor Memory;
//                 O += P V with P from Tensor Memory
//   warp 3        copies of q, one an item
//   warps 4-7, 8-11  weights of stream 0 and 1, one thread a row: maximum,
//                 exponentials, P over S in Tensor Memory. A row's sums are
//                 rescaled only when its maximum has risen by more than 2^8
//                 (weights of up to 2^8 lose nothing in either dtype), which
//                 after the first tiles is rare
// At an item's end the two streams are joined, each group of warps taking
// half of the columns; items cut between blocks are joined by a launch of its
// own (the block that comes last joining them measured slower even for two
// parts: 53.7 us for 52.2). All waits are bounded.
//
// Measured, 8 kv heads of 128: 16 trees of 16 nodes x 6 heads over up to 4,096
// slots 44.2 us (179 MB, 4.0 TB/s); one tree of 64 x 5 over 50,001 slots 74.4
// us (65.6 GFLOP, 0.88 PFLOP/s, tensor pipe 50% active). A stream's tile goes
// round in 4,000 cycles: 1,750 of weights (380 the maximum, 1,030 exponentials
// and packing), the rest the products and what they wait for the other
// stream's. Two groups of 128 threads for a stream, half a row each, took
// longer (93 us).
#pragma once

#include "attend_mma.cuh"

namespace tfx {

// D[tmem] (+)= A B: A and B in shared memory, or A in Tensor Memory. One
// issuing thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
// Instruction descriptor: idesc_f16_f32 with the operands' type and, for the
// second product, a B whose rows (keys) run along the other axis.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_of(int n, bool b_by_keys) {
  const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
  return idesc_f16_f32(128, n) | (type << 7) | (type << 10) | (b_by_keys ? 1u << 16 : 0u);
}
// Shared-memory descriptor of values as B: 128-byte rows (64 columns) a key
// with the 128-byte swizzle, groups of 8 keys 1,024 bytes apart, the next 64
// columns `next` bytes on.
__device__ __forceinline__ uint64_t desc_by_keys(uint32_t at, uint32_t next) {
  return (smem_desc_sw128(at, 1024) & ~(0xFFFFull << 16)) | (static_cast<uint64_t>(next >> 4) << 16);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// Whether the phase of that parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Columns of this thread's Tensor Memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t column, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(column)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// One row of a tile, by its thread: from the scores (128 columns at `scores`)
// to the weights over them, with the running maximum m and sum l. The sums
// (D columns at `sums`) are rescaled where the maximum has risen by more than
// 2^8 since they were begun. kCut: only the keys in vis are seen. sc >= 0. The
// barriers `half` and `three` hear of the first 64 and the next 32 weights, so
// that their products can begin (a tree of 64 nodes over 50,001 slots 77.1 us
// without the second, 75.8 with it).
template <typename T, int D, bool kCut>
__device__ __forceinline__ void weigh(uint32_t scores, uint32_t sums, float sc, const uint32_t (&vis)[4], bool begun,
                                      uint32_t half, uint32_t three, float* m_row, float* l_row) {
  // The scores are read twice, in parts: all 128 of them and what is made of
  // them do not fit a thread's registers. The loops are not unrolled further:
  // the four roles' instructions together pass the cache for them (with all
  // four parts unrolled a tree of 64 nodes over 50,001 slots took 76.1 us for
  // 74.4, 16 trees of 16 over 4,096 45.7 for 44.6; with none 76.8 and 44.4).
  float hi[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  auto word_of = [&](int c) { return c < 2 ? (c == 0 ? vis[0] : vis[1]) : (c == 2 ? vis[2] : vis[3]); };
#pragma unroll(kCut ? 1 : 2)
  for (int c = 0; c < 4; ++c) {
    float v[32];
    tmem_ld32(scores + c * 32, v);
    const uint32_t word = kCut ? word_of(c) : 0;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      if (kCut) {
        if (!(word >> i & 1)) v[i] = -INFINITY;
        if (!(word >> (i + 1) & 1)) v[i + 1] = -INFINITY;
      }
      hi[i / 2 % 4] = fmaxf(hi[i / 2 % 4], fmaxf(v[i], v[i + 1]));
    }
  }
  float top = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
  top = top == -INFINITY ? -INFINITY : top * sc;
  float m = *m_row, l = *l_row;
  const bool rise = top > m + 8.f || m == -INFINITY;
  if (__any_sync(~0u, rise && begun && m > -INFINITY)) {
    const float f = rise && m > -INFINITY ? exp2_approx(m - fmaxf(m, top)) : 1.f;
    l *= f;
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      float o[16];
      uint32_t w[16];
      tmem_ld16(sums + c * 16, o);
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * f);
      tmem_st16(sums + c * 16, w);
    }
  }
  if (rise) m = fmaxf(m, top);
  const float low = m == -INFINITY ? 0.f : -m;
  float2 sum[4] = {};
#pragma unroll(kCut ? 1 : 2)
  for (int c = 0; c < 4; ++c) {
    float v[32];
    tmem_ld32(scores + c * 32, v);
    const uint32_t word = kCut ? word_of(c) : 0;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float2 x = fma2(float2{v[2 * i], v[2 * i + 1]}, float2{sc, sc}, float2{low, low});
      x.x = exp2_approx(x.x);
      x.y = exp2_approx(x.y);
      if (kCut) {
        if (!(word >> (2 * i) & 1)) x.x = 0.f;
        if (!(word >> (2 * i + 1) & 1)) x.y = 0.f;
      }
      sum[i % 4] = add2(sum[i % 4], x);
      w[i] = pack2(T(), x.x, x.y);
    }
    tmem_st16(scores + c * 16, w);   // over scores already read
    if (c == 1 || c == 2) {
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(c == 1 ? half : three);
    }
  }
  const float2 both = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
  *m_row = m;
  *l_row = l + (both.x + both.y);
}

// A tile j lies in stage j % 3 and belongs to stream j % 2. Its barriers are
// number j % 6, so that whoever waits on one waits for each of its phases in
// turn (a barrier of a stage would be waited for by the streams by turns, and
// a wait that passes over a phase cannot tell it from the next but one).
constexpr int kTcSlots = 6;
enum TcBarrier { kQFull, kQEmpty, kKFull, kKEmpty = kKFull + kTcSlots, kVFull = kKEmpty + kTcSlots,
                 kVEmpty = kVFull + kTcSlots, kSFull = kVEmpty + kTcSlots, kPFull = kSFull + 2,
                 kPHalf = kPFull + 2, kPThree = kPHalf + 2, kPvDone = kPThree + 2,
                 kBarriers = kPvDone + 2 };

struct TcShared {
  unsigned long long bars[kBarriers];
  float row_max[2][128], row_sum[2][128];   // of the streams, at an item's end
  uint32_t gone[3][4];                      // keys of a stage whose page is outside the pool (they are 0)
  uint32_t bad[2][4];                       // tree nodes with values that are not finite, of this item and another
  int any_gone;
  int16_t up[TF_MAX_NODES];                 // parents: -1 for none, -2 for an absent node
  int scratch[2 * (384 / 32) + 6];
  uint32_t tmem;
  int abort;
};

template <int D>
struct TcShape {
  static constexpr int kThreads = 384;
  static constexpr int kTile = 128, kGap = 4;
  static constexpr int kParts = D / 64;                  // 64-column parts of a tile
  static constexpr int kPartBytes = kTile * 128;         // one part of q, keys or values
  static constexpr int kTileBytes = kParts * kPartBytes;
  static constexpr int kStages = 3;
  static constexpr int kShared = (1 + 2 * kStages) * kTileBytes;   // where TcShared begins
  static constexpr int kSmem = kShared + static_cast<int>(sizeof(TcShared));
  static_assert(kSmem <= 232448, "a block has 227 KB");
  // Tensor Memory columns: scores of the streams (weights over them), sums.
  static constexpr int kScores = 0, kSums = 256, kColumns = 512;
};

// Node i's row of the tree: the nodes it sees, walked up from the parents.
struct Seen {
  uint32_t w[4];
};
__device__ __forceinline__ Seen seen_by(const int16_t* up, int node) {
  Seen s = {{0, 0, 0, 0}};
  for (int i = node; i >= 0 && up[i] >= -1; i = up[i])
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i >> 5 == x) s.w[x] |= 1u << (i & 31);
  return s;
}
__device__ __forceinline__ uint32_t seen_word(const Seen& s, int i) {
  return i == 0 ? s.w[0] : i == 1 ? s.w[1] : i == 2 ? s.w[2] : i == 3 ? s.w[3] : 0u;
}
struct TcMaps {
  CUtensorMap q, k, v;
};
struct TcArgs {
  AttendArgs a;
  int block_nodes;   // whole nodes of a row block
  int box;           // rows of a copy of keys or values: divides the tile and the page
};

template <typename T, int D>
__global__ void __launch_bounds__(384, 1)
tree_attention_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs args) {
  using S = TcShape<D>;
  constexpr int kTile = S::kTile, kStages = S::kStages;
  const AttendArgs& a = args.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  TcShared& sh = *reinterpret_cast<TcShared*>(smem + S::kShared);
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int row_blocks = (a.nodes + args.block_nodes - 1) / args.block_nodes;
  const int team = blockIdx.x / row_blocks;
  const Rows own{static_cast<int>(blockIdx.x) - team * row_blocks, row_blocks};
  const int node0 = own.rb * args.block_nodes;
  const uint32_t base = smem_u32(smem);
  const uint32_t q_at = base, k_at = base + S::kTileBytes, v_at = k_at + kStages * S::kTileBytes;
  auto bar = [&](int i) { return smem_u32(&sh.bars[i]); };
  if (base & 1023) {   // the swizzled tiles need it; there is no static shared memory before them
    if (tid == 0) atomicOr(a.c.err, kErrWait);
    chain();
    return;
  }

  if (tid == 0) {
    sh.abort = 0;
    sh.any_gone = 0;
    for (int i = 0; i < 4; ++i) sh.bad[0][i] = 0;
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQEmpty), 2);
    for (int i = 0; i < kTcSlots; ++i) {
      mbar_init(bar(kKFull + i), 1);
      mbar_init(bar(kKEmpty + i), 1);
      mbar_init(bar(kVFull + i), 1);
      mbar_init(bar(kVEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kPFull + i), 128);
      mbar_init(bar(kPHalf + i), 128);
      mbar_init(bar(kPThree + i), 128);
      mbar_init(bar(kPvDone + i), 1);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), S::kColumns);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  // What does not depend on the kernel before is done while that still runs.
  chain();
  Line line;
  Cursor cur;
  const int n_tiles = find_run<kTile, S::kGap, S::kThreads>(a, gridDim.x / row_blocks, team, sh.scratch, &line, &cur);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (n_tiles == 0) {
    // nothing to do
  } else if (warp == 0) {
    // ---------------------------------------------------------------- copies
    const int box = args.box, boxes = kTile / box;   // at most 16
    const uint32_t box_bytes = static_cast<uint32_t>(box) * 128;
    // Keys and values go at their own pace, whichever has a free stage: keys
    // are done with earlier. Each side asks for its pages a tile ahead.
    struct Side {
      Cursor cur, next;
      int page, j;
    };
    auto look_up = [&](const Cursor& c) {
      const int slot = c.t * kTile + lane * box;
      return lane < boxes && slot < c.span.slots ? a.c.page_table[c.b * a.c.stride_table + a.c.by_page(slot)] : -1;
    };
    Side ks = {cur, cur, look_up(cur), 0}, vs = ks;
    auto free_stage = [&](const Side& x, int empty) {
      const int b = x.j - kStages;   // the tile before in its stage
      return x.j < n_tiles && (b < 0 || mbar_test(bar(empty + b % kTcSlots), (b / kTcSlots) & 1));
    };
    auto issue = [&](Side* x, const CUtensorMap* map, uint32_t ring, int full, bool values) {
      const int st = x->j % kStages, slot = x->cur.t * kTile + lane * box;
      const bool exists = lane < boxes && slot < x->cur.span.slots;
      const bool outside = exists && static_cast<unsigned>(x->page) >= static_cast<unsigned>(a.c.pages);
      // What does not exist is read past the last page: the copy writes zeros,
      // so that nothing of an earlier tile is left to be multiplied.
      const int page = exists && !outside ? x->page : a.c.pages;
      const int kvh = x->cur.item, row = exists ? slot - a.c.by_page(slot) * a.c.page_size : 0;
      if (x->j + 1 < n_tiles) {
        advance<kTile, S::kGap>(a, &x->next);
        x->page = look_up(x->next);
      }
      const uint32_t missing = __ballot_sync(~0u, outside);
      if (values) {
        if (outside) record_index_error(a.c.err);
        if (lane < 4) {
          uint32_t word = 0;
          if (missing)
            for (int i = 0; i < 32; ++i) word |= (missing >> ((lane * 32 + i) / box) & 1u) << i;
          sh.gone[st][lane] = word;
          if (missing) sh.any_gone = 1;
        }
        __syncwarp();
      }
      const uint32_t b = bar(full + x->j % kTcSlots);
      if (lane == 0) mbar_arrive_expect_tx(b, S::kTileBytes);
      __syncwarp();
      if (lane < boxes)
        for (int h = 0; h < S::kParts; ++h)
          tma_load_4d(ring + st * S::kTileBytes + h * S::kPartBytes + lane * box_bytes, map, h * 64, row, kvh, page, b);
      __syncwarp();
      x->cur = x->next;
      ++x->j;
    };
    unsigned long long since = global_ns();
#pragma unroll 1
    for (uint32_t it = 1; vs.j < n_tiles; ++it) {
      const bool k_now = __all_sync(~0u, free_stage(ks, kKEmpty));
      if (k_now) issue(&ks, &maps.k, k_at, kKFull, false);
      const bool v_now = vs.j < ks.j && __all_sync(~0u, free_stage(vs, kVEmpty));
      if (v_now) issue(&vs, &maps.v, v_at, kVFull, true);
      if (k_now || v_now) {
        since = global_ns();
      } else {
        __nanosleep(20);
        if ((it & 63) == 0) {
          if (global_ns() - since > kWaitLimitNs) *abort_flag = 1;
          if (__any_sync(~0u, *abort_flag)) break;
        }
      }
    }
    if (vs.j < n_tiles) {   // given up: the copies in flight still have to land
      volatile int never = 0;
      for (int j = max(0, ks.j - kStages); j < ks.j; ++j)
        mbar_wait(bar(kKFull + j % kTcSlots), (j / kTcSlots) & 1, &never);
      for (int j = max(0, vs.j - kStages); j < vs.j; ++j)
        mbar_wait(bar(kVFull + j % kTcSlots), (j / kTcSlots) & 1, &never);
    }
  } else if (warp == 3) {
    // ----------------------------------------------------------- copies of q
    int n_items = 0;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n_tiles && ok; ++j) {
      if (j == 0 || cur.t == 0) {
        if (n_items > 0) ok = __all_sync(~0u, mbar_wait_sleepy(bar(kQEmpty), (n_items - 1) & 1, abort_flag, 100));
        if (!ok) break;
        const int kvh = cur.item;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kQFull), static_cast<uint32_t>(args.block_nodes * a.group) * 128 * S::kParts);
          for (int h = 0; h < S::kParts; ++h)
            tma_load_4d(q_at + h * S::kPartBytes, &maps.q, h * 64, kvh * a.group,
                        node0, cur.b, bar(kQFull));
        }
        __syncwarp();
        ++n_items;
      }
      advance<kTile, S::kGap>(a, &cur);
    }
    if (!ok) {
      volatile int never = 0;
      mbar_wait(bar(kQFull), (n_items - 1) & 1, &never);
    }
  } else if (warp == 1 || warp == 2) {
    // -------------------------------------------------------------- products
    const int s = warp - 1;
    const uint32_t scores = tmem + S::kScores + s * 128, sums = tmem + S::kSums + s * D;
    constexpr uint32_t kScoreDesc = idesc_of<T>(128, false), kSumDesc = idesc_of<T>(D, true);
    int n = 0;
    bool ok = true;
#pragma unroll 1
    for (int ja = 0, n_items = 0; ja < n_tiles && ok; ++n_items) {   // the items of the run, tiles ja .. jb - 1
      const int jb = ja + min(n_tiles - ja, cur.nt - cur.t), j0 = ja + ((ja ^ s) & 1);
      ok = __all_sync(~0u, mbar_wait(bar(kQFull), n_items & 1, abort_flag));
      // a stream without a tile of the item does not hold q up
      if (ok && j0 >= jb && jb < n_tiles && elect_one()) mbar_arrive(bar(kQEmpty));
      __syncwarp();
#pragma unroll 1
      for (int j = j0; j < jb && ok; j += 2) {
        const int st = j % kStages, slot_j = j % kTcSlots, phase = (j / kTcSlots) & 1;
        ok = mbar_wait(bar(kKFull + slot_j), phase, abort_flag);
        // the weights lie over the scores until their product is done
        if (ok && n > 0) ok = mbar_wait(bar(kPvDone + s), (n - 1) & 1, abort_flag);
        if (!__all_sync(~0u, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * S::kPartBytes + (k % 4) * 32;
            mma_ss(scores, smem_desc_sw128(q_at + off, 1024),
                   smem_desc_sw128(k_at + st * S::kTileBytes + off, 1024), kScoreDesc, k > 0);
          }
          mma_commit(bar(kSFull + s));
          // only what someone will wait for, so that nothing arrives after the end
          if (j + kStages < n_tiles) mma_commit(bar(kKEmpty + slot_j));
          if (j + 2 >= jb && jb < n_tiles) mma_commit(bar(kQEmpty));
        }
        __syncwarp();
        ok = mbar_wait(bar(kVFull + slot_j), phase, abort_flag) && mbar_wait(bar(kPHalf + s), n & 1, abort_flag);
        if (!__all_sync(~0u, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        auto add_up = [&](int k) {
          mma_ts(sums, scores + k * 8, desc_by_keys(v_at + st * S::kTileBytes + k * 2048, S::kPartBytes), kSumDesc,
                 j > j0 || k > 0);
        };
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k) add_up(k);
        }
        __syncwarp();
        ok = __all_sync(~0u, mbar_wait(bar(kPThree + s), n & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = kTile / 32; k < kTile / 64 * 3; ++k) add_up(k);
        }
        __syncwarp();
        ok = __all_sync(~0u, mbar_wait(bar(kPFull + s), n & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = kTile / 64 * 3; k < kTile / 16; ++k) add_up(k);
          mma_commit(bar(kPvDone + s));
          if (j + kStages < n_tiles) mma_commit(bar(kVEmpty + slot_j));
        }
        __syncwarp();
        ++n;
      }
      cur.t += jb - ja - 1;
      advance<kTile, S::kGap>(a, &cur);
      ja = jb;
    }
    if (!ok && n > 0) {   // given up: the products in flight still have to end
      volatile int never = 0;
      mbar_wait(bar(kPvDone + s), (n - 1) & 1, &never);
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------------- weights
    const int s = (warp - 4) / 4, row = (warp % 4) * 32 + lane, both = tid - 128;
    const uint32_t mine = static_cast<uint32_t>((warp % 4) * 32) << 16;   // this warp's Tensor Memory lanes
    const uint32_t scores = tmem + mine + S::kScores + s * 128, sums = tmem + mine + S::kSums + s * D;
    const float sc = a.scale * kLog2e;
    const int row_node = row / a.group;
    const T* values = static_cast<const T*>(a.v);
    const int node = row_node < args.block_nodes && node0 + row_node < a.nodes ? node0 + row_node : -1;
    int n = 0, n_items = 0, seen_b = -1;
    Seen seen = {};
#pragma unroll 1
    for (int ja = 0; ja < n_tiles;) {   // the items of the run, tiles ja .. jb - 1 of it
      const int jb = ja + min(n_tiles - ja, cur.nt - cur.t);
      const int kvh = cur.item;
      if (cur.b != seen_b) {   // the tree is its sequence's: another item of it has it still
        seen_b = cur.b;
        if (both < a.nodes) {
          int p = a.parents[cur.b * a.stride_parents + both];
          if (p >= both) {
            record_index_error(a.c.err);
            p = -2;
          }
          sh.up[both] = p < -2 ? -2 : p;
        }
        if (!group_all(3, 256, !*abort_flag)) break;
        seen = node >= 0 ? seen_by(sh.up, node) : Seen{};
      }
      // The other item's list of bad values is cleared: nobody reads it any more.
      uint32_t* bad = sh.bad[n_items & 1];
      if (both < 4) sh.bad[(n_items + 1) & 1][both] = 0;
      ++n_items;
      float m = -INFINITY, l = 0.f;
      bool used = false;
#pragma unroll 1
      for (int j = ja + ((ja ^ s) & 1); j < jb; j += 2) {
        const int st = j % kStages;
        const int slot0 = (cur.t + j - ja) * kTile;
        mbar_wait(bar(kSFull + s), n & 1, abort_flag);
        // (held until this tile's product; makes gone[] visible)
        mbar_wait(bar(kVFull + j % kTcSlots), (j / kTcSlots) & 1, abort_flag);
        __syncwarp();
        tc_fence_after();
        uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};   // keys this row sees
        if (slot0 + kTile <= cur.span.context && !*static_cast<volatile int*>(&sh.any_gone)) {
          weigh<T, D, false>(scores, sums, sc, vis, used, bar(kPHalf + s), bar(kPThree + s), &m, &l);
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int off = slot0 + w * 32 - cur.span.context;   // tree node of the word's first key
            uint32_t word = ~0u;
            if (off > -32) {
              word = off >= 0 ? __funnelshift_r(seen_word(seen, off >> 5), seen_word(seen, (off >> 5) + 1), off & 31)
                              : (seen.w[0] << -off) | ((1u << -off) - 1);
            }
            const int left = cur.span.slots - slot0 - w * 32;
            if (left < 32) word &= left > 0 ? (1u << left) - 1 : 0u;
            vis[w] = node >= 0 ? word & ~sh.gone[st][w] : 0u;
          }
          // Values that must not be multiplied, even by 0, become 0: those of
          // rows past the last slot, and of tree nodes where they are not
          // finite (added at the item's end to the rows that see them).
          const int end = min(kTile, (cur.span.slots - slot0 + args.box - 1) / args.box * args.box);
          const int j0 = max(0, cur.span.context - slot0), j1 = cur.span.slots - slot0;
          for (int id0 = j0 * (D / 8) + row; id0 < end * (D / 8); id0 += 4 * 128) {
            uint4 x[4];
            auto place = [&](int id) {
              const int key = id / (D / 8), ch = id % (D / 8);
              return reinterpret_cast<uint4*>(smem + (v_at - base) + st * S::kTileBytes + (ch / 8) * S::kPartBytes +
                                              key * 128 + (((ch % 8) ^ (key & 7)) << 4));
            };
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (id0 + u * 128 < end * (D / 8)) x[u] = *place(id0 + u * 128);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int id = id0 + u * 128, key = id / (D / 8);
              if (id >= end * (D / 8)) continue;
              if (key >= j1) {
                *place(id) = uint4{0, 0, 0, 0};
              } else if (a.nodes > 1 && (bad_pair<T>(x[u].x) | bad_pair<T>(x[u].y) | bad_pair<T>(x[u].z) |
                                         bad_pair<T>(x[u].w))) {
                uint16_t* h = reinterpret_cast<uint16_t*>(place(id));
                const int nd = slot0 + key - cur.span.context;
#pragma unroll 1
                for (int y = 0; y < 8; ++y)
                  if (bad16<T>(h[y])) h[y] = 0;
                atomicOr(&bad[nd / 32], 1u << (nd % 32));
              }
            }
          }
          fence_proxy_async_shared();
          weigh<T, D, true>(scores, sums, sc, vis, used, bar(kPHalf + s), bar(kPThree + s), &m, &l);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kPFull + s));
        used = true;
        ++n;
      }
      {
        // The streams' sums together; each group takes half of the columns.
        if (used) mbar_wait(bar(kPvDone + s), (n - 1) & 1, abort_flag);
        __syncwarp();
        sh.row_max[s][row] = used ? m : -INFINITY;
        sh.row_sum[s][row] = used ? l : 0.f;
        tc_fence_before();
        if (!group_all(3, 256, !*abort_flag)) break;
        tc_fence_after();
        const float m0 = sh.row_max[0][row], m1 = sh.row_max[1][row], top = fmaxf(m0, m1);
        const float low = top == -INFINITY ? 0.f : top;
        const float f0 = exp2_approx(m0 - low), f1 = exp2_approx(m1 - low);
        const float sum = f0 * sh.row_sum[0][row] + f1 * sh.row_sum[1][row];
        // A stream without a tile of this item has nothing in its columns (its
        // maximum is -inf, but so is that of one that saw nothing).
        const bool has0 = jb - ja > 1 || (ja & 1) == 0, has1 = jb - ja > 1 || (ja & 1) == 1;
        const bool whole = cur.t == 0 && cur.nt == jb - ja;
        const bool idle = cur.span.context < 0;
        const bool any_bad = (bad[0] | bad[1] | bad[2] | bad[3]) != 0;
        const int rows = min(args.block_nodes, a.nodes - node0) * a.group;
        const bool present = node >= 0 && !idle && sh.up[node] >= -1;
        const bool empty = !present || sum == 0.f;
        const float inv = whole ? (empty ? 0.f : 1.f / sum) : 1.f;
        const size_t out_at = node >= 0 ? (static_cast<size_t>(cur.b) * a.nodes + node) * a.heads + kvh * a.group +
                                              row - row_node * a.group : 0;
        T* out = static_cast<T*>(a.out) + out_at * D;
        float* part = a.partials + part_index(line, own, team, cur.first) * kPartFloats<128, D>;
#pragma unroll 1
        for (int c = s * (D / 2); c < (s + 1) * (D / 2); c += 16) {
          float x[16] = {}, y[16] = {};
          if (has0) tmem_ld16(tmem + mine + S::kSums + c, x);
          if (has1) tmem_ld16(tmem + mine + S::kSums + D + c, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = (f0 * x[i] + f1 * y[i]) * inv;
          if (node < 0) continue;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              *reinterpret_cast<uint4*>(out + c + i) =
                  empty ? uint4{0, 0, 0, 0}
                        : uint4{pack2(T(), x[i], x[i + 1]), pack2(T(), x[i + 2], x[i + 3]),
                                pack2(T(), x[i + 4], x[i + 5]), pack2(T(), x[i + 6], x[i + 7])};
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) __stcg(part + (c + i) * 128 + row, x[i]);
          }
        }
        // Values that are not finite, where they are seen: whatever is finite
        // adds nothing to them, so what is written already serves.
        if (any_bad && node >= 0 && !empty)
#pragma unroll 1
          for (int nd = 0; nd <= node; ++nd) {
            if (!(bad[nd / 32] >> (nd % 32) & 1) || !(seen_word(seen, nd / 32) >> (nd % 32) & 1)) continue;
            const int64_t off = slot_offset(a.c, cur.b, cur.span.context + nd);
            if (off < 0) continue;
            const T* from = values + off + kvh * a.c.stride_head;
#pragma unroll 1
            for (int c = s * (D / 2); c < (s + 1) * (D / 2); ++c) {
              if (!bad16<T>(reinterpret_cast<const uint16_t*>(from)[c])) continue;
              if (whole) {
                out[c] = from_f32<T>(to_f32(out[c]) + to_f32(from[c]));
              } else {
                __stcg(part + c * 128 + row, __ldcg(part + c * 128 + row) + to_f32(from[c]));
              }
            }
          }
        tc_fence_before();
        if (node >= 0 && s == 0) {
          if (whole) {
            a.lse[out_at] = empty ? -INFINITY : (top + log2f(sum)) * kLn2;
          } else {
            part[128 * D + row] = top;
            part[128 * D + 128 + row] = sum;
          }
        }
        // Sums, parents and maxima have been read.
        if (!group_all(3, 256, true)) break;
      }
      cur.t += jb - ja - 1;
      advance<kTile, S::kGap>(a, &cur);
      ja = jb;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, S::kColumns);
  if (tid == 0 && sh.abort) atomicOr(a.c.err, kErrWait);
}

}  // namespace tfx
