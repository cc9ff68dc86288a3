// Attention over a cache in 4 bits with tcgen05: more than 16 rows a kv head.
//
// The tiles, streams, rows and joins are those of attend_tc.cuh: blocks of up
// to 128 rows, tiles of 128 keys that go alternately to two streams, scores
// and weights in Tensor Memory. What is different is how a tile gets there:
//   warp 0        copies of codes and factors, three tiles in flight
//   warps 1, 2    products of stream 0 and 1
//   warps 4-7, 8-11  weights of stream 0 and 1, one thread a row
//   warps 12-15, 16-19  codes of stream 0 and 1 to fp16 in the products' layout,
//                 keys and values, one thread a key, and q at an item's begin
//
// A code has 3 bits and a sign and a factor 8 bits, so c s is exact in fp16's
// 11, as long as it stays in range: factors go in relative to the largest of
// their 32 keys, whose exponents ek and ev the weights' threads put back. That
// is right where every row sees the 32 alike, and they are of similar sizes.
// Where they reach past the context (rows see different nodes, and what an
// absent node's slot holds is anything), or their factors differ by more than
// kKeySpread or kValueSpread, codes go in without factors, and a score and a
// weight are multiplied by their key's own, in fp32: what a row does not see has
// no part in its scores, maximum or exponent, and what it sees is not rounded
// for its neighbours' sake. q is scaled into fp16's range by a power of two a
// row. Elements are in the order in which they come out of a word
// (0, 4, 1, 5, 2, 6, 3, 7), in q too, and in the sums until they are written.
//
// Weights are p 2^(ev - E), E of a row rising like its maximum, so that
// values of any size weigh what they should; sums of weights are of p itself.
// The largest weight of a row is bounded (largest p times largest factor of 32
// keys, 2^6 too much at most; where keys are treated one by one their own); the
// bound is 2^8 when E is set, so that fp16's last bit is 2^-26 of the largest
// weight or less.
//
// Weights are rounded to fp16 for the second product, as values are in it: see
// attend_q.cuh.
//
// Measured: 16 trees of 16 nodes x 6 heads of 128 x 8 over up to 4,096 slots
// 56.1 us (289 TFLOP/s; 45.8 with heads of 64), of 64 nodes 156 (424), one tree
// of 64 x 5 over 50,001 slots 117 (560). With values whose sizes differ by up to
// 2^4 69, by up to 2^12, where every key is treated by itself, 75. Not memory
// (14% of its rate at 16 nodes) but the chain of a tile bounds it, codes,
// scores, weights, sums, and the instructions of five roles: issue slots 53%
// busy, tensor pipe 24%. Unrolled, the roles do not fit the instruction cache
// (61 us for 55).
#pragma once

#include "attend_q.cuh"
#include "attend_tc.cuh"

namespace tfx {

// Codes of tile j lie in stage j % 3 and are stream j % 2's; their barriers are
// number j % 6, so that whoever waits on one waits for each of its phases. So
// is the end of an item's q told to the group of warps that has the next item's
// first tile, and writes its q, on a barrier of that group's own.
constexpr int kQtcStages = 3, kQtcSlots = 6;
enum QtcBarrier { kCFull, kCEmpty = kCFull + kQtcSlots, kXQFull = kCEmpty + kQtcSlots, kXQEmpty,
                  kXKFull = kXQEmpty + 2, kXKEmpty = kXKFull + 2, kXVFull = kXKEmpty + 2, kXVEmpty = kXVFull + 2,
                  kXSFull = kXVEmpty + 2, kXPFull = kXSFull + 2, kXPHalf = kXPFull + 2, kXPThree = kXPHalf + 2,
                  kXPvDone = kXPThree + 2, kXWords = kXPvDone + 2, kXBarriers = kXWords + 4 };

struct QtcShared {
  unsigned long long bars[kXBarriers];
  float row_max[2][128], row_sum[2][128];   // of the streams, at an item's end
  int row_exp[2][128];
  // What the weights need to know of a stream's tile, in places by turns: the
  // place is written with the tile's keys, while the tile before is weighed.
  struct Words {
    float row_factor[128];                  // scale log2(e) over the power that q was scaled by
    // Of each key, where a tile's are not treated alike: what a score and a
    // weight are multiplied by, and the least power of two (its exponent) that
    // the latter is below.
    alignas(16) float key_by[128], value_by[128], value_log[128];
    int ek[4], ev[4];                       // exponents of each 32 keys
    int apart[4];                           // whether their factors are not in the operands
    uint32_t there[4];                      // keys that exist
  } words[2][2];
  int16_t up[TF_MAX_NODES];                 // parents: -1 for none, -2 for an absent node
  int scratch[2 * (640 / 32) + 6];
  uint32_t tmem;
  int abort;
};

template <int D>
struct QtcShape {
  static constexpr int kThreads = 640;
  static constexpr int kTile = 128, kGap = 4;
  static constexpr int kParts = D / 64;                  // 64-column parts of a tile
  static constexpr int kPartBytes = kTile * 128;
  static constexpr int kTileBytes = kParts * kPartBytes;
  static constexpr int kRowBytes = D / 2;                // of codes
  static constexpr int kHalf = kTile * kRowBytes;
  static constexpr int kStageBytes = 2 * kHalf + kTile * 4;   // codes of keys and values, factors
  static constexpr int kKeysAt = kTileBytes, kValuesAt = kKeysAt + 2 * kTileBytes, kCodesAt = kValuesAt + 2 * kTileBytes;
  static constexpr int kShared = kCodesAt + kQtcStages * kStageBytes;
  static constexpr int kSmem = kShared + static_cast<int>(sizeof(QtcShared));
  static_assert(kSmem <= 232448, "a block has 227 KB");
  static constexpr int kScores = 0, kSums = 256, kColumns = 512;
};

struct QtcArgs {
  QAttendArgs q;
  int block_nodes;   // whole nodes of a row block
  float zero;        // 0: a product and this are rounded, where the compiler would fuse it with what is added next
};

// Factors of 32 keys go into the operands where they differ by no more powers of
// two than these. Of keys: c s 2^8 is a normal fp16 number down to 2^-18 of the
// largest, and exact. Of values: what the weights' bound is too large by, which
// their rounding to fp16 pays for.
constexpr int kKeySpread = 18, kValueSpread = 6;
// The least exponent E, of a factor that goes into an operand, and the largest of
// a value that does: 2^(ev - E) is a number in fp32 then. Others are treated one
// by one, where a weight is (p v) 2^-E.
constexpr int kLeastExp = -100, kMostKeyExp = 100, kMostValueExp = 26;
// In the place of the exponent of 0.
constexpr int kNoExp = 1000;

// One row of a tile, by its thread, as weigh() of attend_tc.cuh, with a factor
// for the scores and one for the weights of each 32 keys, or (kEach) of each
// key, with the keys that the row sees in vis. sc: the row's factor, not below 0.
// Each key's scores are rounded before m, a rounded one, is subtracted, so that p
// is 2^8 at most, and the weights' bound is kept relative to the scores'. Where a
// warp's scores are large all tiles are treated so (not kEach: false then, and
// nothing is done): at 2^30 an exact product passes m by up to 64, and its weight
// fp16's range, and a value's exponent is lost beside a score. (All tiles always:
// trees of 64 nodes 158.7 us for 156.)
constexpr float kLargeScore = 0x1p20f;
template <int D, bool kEach>
__device__ __forceinline__ bool weigh_q(uint32_t scores, uint32_t sums, const QtcShared::Words& words, float sc,
                                        float zero, const uint32_t (&vis)[4], bool begun, uint32_t half,
                                        uint32_t three, float* m_row, float* l_row, int* e_row) {
  auto word_of = [&](int c) { return c < 2 ? (c == 0 ? vis[0] : vis[1]) : (c == 2 ? vis[2] : vis[3]); };
  auto score_by = [&](int c) { return sc * power2(words.ek[c] - 8); };
  auto pairs_at = [&](const float* of, int key, float2 (&x)[2]) {   // of four keys
    const float4 y = *reinterpret_cast<const float4*>(of + key);
    x[0] = float2{y.x, y.y}, x[1] = float2{y.z, y.w};
  };
  auto product = [&](float x, float y, float2 by) { return fma2(float2{x, y}, by, float2{zero, zero}); };
  // Parts of 32 keys, up to the last that has some.
  const int parts = !kEach || words.there[3] ? 4 : words.there[2] ? 3 : words.there[1] ? 2 : 1;
  // The largest score, and the largest weight with its values' size (kEach: were
  // the largest score 0).
  float top = -INFINITY, need = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < parts; ++c) {
    float v[32];
    tmem_ld32(scores + c * 32, v);
    float hi[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if constexpr (kEach) {
      const uint32_t word = word_of(c);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float2 by[2];
        pairs_at(words.key_by, c * 32 + i, by);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int n = i + 2 * k;
          const float2 x = product(v[n], v[n + 1], mul2(by[k], float2{sc, sc}));
          v[n] = word >> n & 1 ? x.x : -INFINITY;
          v[n + 1] = word >> (n + 1) & 1 ? x.y : -INFINITY;
          hi[n / 2 % 4] = fmaxf(hi[n / 2 % 4], fmaxf(v[n], v[n + 1]));
        }
      }
      const float high = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
      const float base = high == -INFINITY ? 0.f : high;
      float2 large = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float2 log[2];
        pairs_at(words.value_log, c * 32 + i, log);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 weight = add2(add2(float2{v[i + 2 * k], v[i + 2 * k + 1]}, float2{-base, -base}), log[k]);
          large = float2{fmaxf(large.x, weight.x), fmaxf(large.y, weight.y)};
        }
      }
      const float size = fmaxf(large.x, large.y);
      need = high > top ? fmaxf(need + (top - high), size) : fmaxf(need, high - top + size);
      top = fmaxf(top, high);
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2) hi[i / 2 % 4] = fmaxf(hi[i / 2 % 4], fmaxf(v[i], v[i + 1]));
      const float high = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3])) * score_by(c);
      top = fmaxf(top, high);
      need = fmaxf(need, high + static_cast<float>(words.ev[c]));
    }
  }
  float m = *m_row, l = *l_row;
  int e = *e_row;
  const bool rise = top > m + 8.f;
  const float to = rise ? top : m;
  if (!kEach && __any_sync(~0u, !(fabsf(to) < kLargeScore))) return false;
  need = kEach ? need + (top - to) : need - to;
  const bool grow = need > static_cast<float>(e) + 15.f;   // a weight might pass fp16's range
  if (__any_sync(~0u, rise || grow)) {
    const float down = m - to;   // 0, or below
    int to_e = e;
    if (rise) to_e = max(kLeastExp, e + static_cast<int>(floorf(fmaxf(down, -400.f))));
    if (rise || grow) to_e = min(126, max(to_e, static_cast<int>(ceilf(fmaxf(need, -190.f))) - 8));
    l *= exp2_approx(down);
    if (begun) {
      const float f = exp2_approx(down + static_cast<float>(e - to_e));
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
    m = to;
    e = to_e;
  }
  auto stored = [&](int c) {   // weights over scores already read
    if (c == 1 || c == 2) {
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(c == 1 ? half : three);
    }
  };
  float2 sum[4] = {};
  const float to16 = power2(-e);
#pragma unroll 1
  for (int c = 0; c < parts; ++c) {
    float v[32];
    tmem_ld32(scores + c * 32, v);
    uint32_t w[16];
    if constexpr (kEach) {
      const uint32_t word = word_of(c);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float2 by[2], values[2];
        pairs_at(words.key_by, c * 32 + i, by);
        pairs_at(words.value_by, c * 32 + i, values);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool sees_x = word >> (i + 2 * k) & 1, sees_y = word >> (i + 2 * k + 1) & 1;
          float2 x = add2(product(v[i + 2 * k], v[i + 2 * k + 1], mul2(by[k], float2{sc, sc})), float2{-m, -m});
          x.x = sees_x ? exp2_approx(x.x) : 0.f;
          x.y = sees_y ? exp2_approx(x.y) : 0.f;
          sum[i / 4 % 2 * 2 + k] = add2(sum[i / 4 % 2 * 2 + k], x);
          x = mul2(mul2(x, values[k]), float2{to16, to16});   // (this order: the product is in range)
          w[i / 2 + k] = pack2(__half(), sees_x ? x.x : 0.f, sees_y ? x.y : 0.f);   // whatever the factor
        }
      }
    } else {
      const float by = score_by(c), size = power2(max(-126, words.ev[c] - e));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float2 x = fma2(float2{v[2 * i], v[2 * i + 1]}, float2{by, by}, float2{-m, -m});
        x.x = exp2_approx(x.x);
        x.y = exp2_approx(x.y);
        sum[i % 4] = add2(sum[i % 4], x);
        x = mul2(x, float2{size, size});
        w[i] = pack2(__half(), x.x, x.y);
      }
    }
    tmem_st16(scores + c * 16, w);
    stored(c);
  }
#pragma unroll 1
  for (int c = parts; c < 4; ++c) {
    const uint32_t none[16] = {};
    tmem_st16(scores + c * 16, none);
    stored(c);
  }
  const float2 both = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
  *m_row = m;
  *l_row = l + (both.x + both.y);
  *e_row = e;
  return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(640, 1) kvq_attention_tc_kernel(const __grid_constant__ QtcArgs args) {
  using S = QtcShape<D>;
  constexpr int kTile = S::kTile, kRB = S::kRowBytes;
  const AttendArgs& a = args.q.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  QtcShared& sh = *reinterpret_cast<QtcShared*>(smem + S::kShared);
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int row_blocks = (a.nodes + args.block_nodes - 1) / args.block_nodes;
  const int team = blockIdx.x / row_blocks;
  const Rows own{static_cast<int>(blockIdx.x) - team * row_blocks, row_blocks};
  const int node0 = own.rb * args.block_nodes;
  const int rows = min(args.block_nodes, a.nodes - node0) * a.group;
  const uint32_t base = smem_u32(smem);
  const uint32_t q_at = base, k_at = base + S::kKeysAt, v_at = base + S::kValuesAt;
  auto bar = [&](int i) { return smem_u32(&sh.bars[i]); };
  if (base & 1023) {   // the swizzled tiles need it; there is no static shared memory before them
    if (tid == 0) atomicOr(a.c.err, kErrWait);
    chain();
    return;
  }
  if (tid == 0) {
    sh.abort = 0;
    for (int i = 0; i < kQtcSlots; ++i) {
      mbar_init(bar(kCFull + i), args.q.box ? 1 : 32);
      mbar_init(bar(kCEmpty + i), 4);
    }
    mbar_init(bar(kXQFull), 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kXQEmpty + i), 2);
      mbar_init(bar(kXKFull + i), 4);
      mbar_init(bar(kXKEmpty + i), 1);
      mbar_init(bar(kXVFull + i), 4);
      mbar_init(bar(kXVEmpty + i), 1);
      mbar_init(bar(kXSFull + i), 1);
      mbar_init(bar(kXPFull + i), 128);
      mbar_init(bar(kXPHalf + i), 128);
      mbar_init(bar(kXPThree + i), 128);
      mbar_init(bar(kXPvDone + i), 1);
      mbar_init(bar(kXWords + i), 4);
      mbar_init(bar(kXWords + 2 + i), 4);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), S::kColumns);
    tmem_relinquish();
  }
  chain();
  Line line;
  Cursor cur;
  const int n_tiles = find_run<kTile, S::kGap, S::kThreads>(a, gridDim.x / row_blocks, team, sh.scratch, &line, &cur);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  // The registers of 640 threads, 96 each, are shared out anew: the first four
  // warps keep theirs, 32 go from a thread of the last eight to one of weights.
  if (warp < 4) {
    if (n_tiles == 0 || warp == 3) {
      // nothing to do
    } else if (warp == 0) {
      // -------------------------------------------------------------- copies
      // (a page outside the pool is recorded and left out by the threads of its keys)
      const uint8_t* kp = static_cast<const uint8_t*>(a.k);
      const uint8_t* vp = static_cast<const uint8_t*>(a.v);
      auto stage_free = [&](int j) {
        const int before = j - kQtcStages;   // the tile before in its stage
        return before < 0 ||
               __all_sync(~0u, mbar_wait(bar(kCEmpty + before % kQtcSlots), (before / kQtcSlots) & 1, abort_flag));
      };
      auto codes_of = [&](int j) { return base + S::kCodesAt + j % kQtcStages * S::kStageBytes; };
      if (args.q.box) {   // 4 slots at least: a lane has a run
        const int box = args.q.box;
        const bool has_run = lane < kTile / box;
        const uint32_t bytes = box * kRB;
        const int32_t* pages = a.c.page_table + cur.b * a.c.stride_table;
        const uint8_t* k_head = kp + cur.item * a.c.stride_head;
        const uint32_t* s_head = args.q.scales + cur.item * args.q.scale_head;
        int page = -1, row = 0;
        auto look_up = [&]() {
          const int slot = cur.t * kTile + lane * box;
          page = -1;
          if (has_run && slot < cur.span.slots) {
            const int p = a.c.by_page(slot);
            page = pages[p];
            row = slot - p * a.c.page_size;
          }
        };
        look_up();
#pragma unroll 1
        for (int j = 0; j < n_tiles; ++j) {
          const bool real = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.c.pages);
          const uint8_t* k_at = k_head + static_cast<uint64_t>(static_cast<uint32_t>(page)) * a.c.stride_page + row * kRB;
          const uint32_t* s_at = s_head + static_cast<uint64_t>(static_cast<uint32_t>(page)) * args.q.scale_page + row;
          const uint32_t there = __ballot_sync(~0u, real);
          if (j + 1 < n_tiles) {
            if (++cur.t == cur.nt) {   // the next item
              cur.t = cur.nt - 1;
              advance<kTile, S::kGap>(a, &cur);
              pages = a.c.page_table + cur.b * a.c.stride_table;
              k_head = kp + cur.item * a.c.stride_head;
              s_head = args.q.scales + cur.item * args.q.scale_head;
            }
            look_up();
          }
          if (!stage_free(j)) break;
          const uint32_t full = bar(kCFull + j % kQtcSlots), codes = codes_of(j);
          if (lane == 0) mbar_arrive_expect_tx(full, __popc(there) * (2 * bytes + box * 4));
          __syncwarp();
#pragma unroll 1
          for (uint32_t left = there; left; left &= left - 1) {
            const int run = __ffs(left) - 1;
            const uint64_t from = __shfl_sync(~0u, reinterpret_cast<uint64_t>(k_at), run);
            const uint64_t with = __shfl_sync(~0u, reinterpret_cast<uint64_t>(s_at), run);
            if (elect_one()) {
              copy_run(codes + run * bytes, reinterpret_cast<const void*>(from), bytes, full);
              copy_run(codes + S::kHalf + run * bytes, reinterpret_cast<const void*>(from + (vp - kp)), bytes, full);
              copy_run(codes + 2 * S::kHalf + run * box * 4, reinterpret_cast<const void*>(with), box * 4, full);
            }
            __syncwarp();
          }
        }
      } else {   // a lane has a key of each 32
        constexpr int kChunks = kRB / 16;
#pragma unroll 1
        for (int j = 0; j < n_tiles; ++j) {
          const int32_t* pages = a.c.page_table + cur.b * a.c.stride_table;
          auto look = [&](int k, int* row) {
            const int slot = cur.t * kTile + k * 32 + lane, p = a.c.by_page(slot);
            *row = slot - p * a.c.page_size;
            return slot < cur.span.slots ? pages[p] : -1;
          };
          int next_row, next_page = look(0, &next_row);
          if (!stage_free(j)) break;
          const uint32_t full = bar(kCFull + j % kQtcSlots), codes = codes_of(j);
#pragma unroll 1
          for (int k = 0; k < kTile / 32; ++k) {
            const int page = next_page, row = next_row;
            if (k + 1 < kTile / 32) next_page = look(k + 1, &next_row);
            const bool real = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.c.pages);
            const int64_t at = real ? page * a.c.stride_page + row * a.c.stride_token + cur.item * a.c.stride_head : -1;
            const uint32_t into = codes + (k * 32 * kChunks + lane) * 16;
#pragma unroll
            for (int n = 0; n < kChunks; ++n) {
              const int id = n * 32 + lane;
              const int64_t from = __shfl_sync(~0u, at, id / kChunks);
              if (from >= 0) {
                copy16(into + n * 512, kp + from + id % kChunks * 16, true);
                copy16(into + n * 512 + S::kHalf, vp + from + id % kChunks * 16, true);
              }
            }
            if (real)
              copy4(codes + 2 * S::kHalf + (k * 32 + lane) * 4,
                    args.q.scales + page * args.q.scale_page + row * args.q.scale_token + cur.item * args.q.scale_head);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
          advance<kTile, S::kGap>(a, &cur);
        }
      }
    } else {
      // ------------------------------------------------------------ products
      const int s = warp - 1;
      const uint32_t scores = tmem + S::kScores + s * 128, sums = tmem + S::kSums + s * D;
      constexpr uint32_t kScoreDesc = idesc_of<__half>(128, false), kSumDesc = idesc_of<__half>(D, true);
      const uint32_t k_tile = k_at + s * S::kTileBytes, v_tile = v_at + s * S::kTileBytes;
      int n = 0;
      bool ok = true;
#pragma unroll 1
      for (int ja = 0, n_items = 0; ja < n_tiles && ok; ++n_items) {   // the items of the run, tiles ja .. jb - 1
        const int jb = ja + min(n_tiles - ja, cur.nt - cur.t), j0 = ja + ((ja ^ s) & 1);
        ok = __all_sync(~0u, mbar_wait(bar(kXQFull), n_items & 1, abort_flag));
        // a stream without a tile of the item does not hold q up
        if (ok && j0 >= jb && jb < n_tiles && elect_one()) mbar_arrive(bar(kXQEmpty + (jb & 1)));
        __syncwarp();
#pragma unroll 1
        for (int j = j0; j < jb && ok; j += 2) {
          ok = mbar_wait(bar(kXKFull + s), n & 1, abort_flag);
          // the weights lie over the scores until their product is done
          if (ok && n > 0) ok = mbar_wait(bar(kXPvDone + s), (n - 1) & 1, abort_flag);
          if (!__all_sync(~0u, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k / 4) * S::kPartBytes + (k % 4) * 32;
              mma_ss(scores, smem_desc_sw128(q_at + off, 1024), smem_desc_sw128(k_tile + off, 1024), kScoreDesc, k > 0);
            }
            mma_commit(bar(kXSFull + s));
            // only what someone will wait for, so that nothing arrives after the end
            if (j + 2 < n_tiles) mma_commit(bar(kXKEmpty + s));
            if (j + 2 >= jb && jb < n_tiles) mma_commit(bar(kXQEmpty + (jb & 1)));
          }
          __syncwarp();
          ok = mbar_wait(bar(kXVFull + s), n & 1, abort_flag) && mbar_wait(bar(kXPHalf + s), n & 1, abort_flag);
          if (!__all_sync(~0u, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          auto add_up = [&](int k) {
            mma_ts(sums, scores + k * 8, desc_by_keys(v_tile + k * 2048, S::kPartBytes), kSumDesc, j > j0 || k > 0);
          };
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k) add_up(k);
          }
          __syncwarp();
          ok = __all_sync(~0u, mbar_wait(bar(kXPThree + s), n & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = kTile / 32; k < kTile / 64 * 3; ++k) add_up(k);
          }
          __syncwarp();
          ok = __all_sync(~0u, mbar_wait(bar(kXPFull + s), n & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = kTile / 64 * 3; k < kTile / 16; ++k) add_up(k);
            mma_commit(bar(kXPvDone + s));
            if (j + 2 < n_tiles) mma_commit(bar(kXVEmpty + s));
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
        mbar_wait(bar(kXPvDone + s), (n - 1) & 1, &never);
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // ------------------------------------------------------- codes to fp16
    // key: a thread's key of a tile, and row of q
    const int s = (warp - 12) / 4, key = (tid - 384) % 128, quarter = (warp - 12) % 4;
    // 16-byte chunk c of row r of a tile in the products' layout.
    auto place = [&](int at, int r, int c) {
      return reinterpret_cast<uint4*>(smem + at + (c / 8) * S::kPartBytes + r * 128 + (((c % 8) ^ (r & 7)) << 4));
    };
    // Codes of this thread's row times the factor s16, which is exact.
    auto unpack_row = [&](const unsigned char* codes, int to, __half s16) {
      const __half2 by = __half2half2(s16), by16 = __hmul2(by, __float2half2_rn(0.0625f));
#pragma unroll 1
      for (int it = 0; it < kRB / 16; ++it) {
        // (this order keeps eight threads on different banks, reading and writing)
        const int chunk = kRB == 64 ? (it + (key >> 1)) & 3 : (it + (key >> 2)) & 1;
        const uint4 w4 = *reinterpret_cast<const uint4*>(codes + key * kRB + chunk * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = w[i] >> 8;
          const uint32_t c[4] = {whole2<4, false>(w[i]), whole2<4, true>(w[i]), whole2<4, false>(x), whole2<4, true>(x)};
          uint32_t y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&c[z]), z & 1 ? by16 : by);
            y[z] = *reinterpret_cast<const uint32_t*>(&p);
          }
          *place(to, key, chunk * 4 + i) = uint4{y[0], y[1], y[2], y[3]};
        }
      }
    };
    int n_ends = 0;   // of q that this group has waited for
    bool ok = true;
    float row_factor = 0.f;   // of row `key` of the item
    // The page of this thread's key, asked for a tile ahead: -1 where there is
    // no such key (a -1 in the table becomes -2).
    auto outside_is = [](int page) { return page == -1 ? -2 : page; };
    auto page_of = [&](const Cursor& c) {
      const int slot = c.t * kTile + key;
      return slot < c.span.slots ? outside_is(a.c.page_table[c.b * a.c.stride_table + a.c.by_page(slot)]) : -1;
    };
    // q of an item: its rows' factors for both streams, q itself by the one
    // that has the item's first tile.
    auto new_item = [&](const Cursor& c, bool first, int cur_j) {
      if (first && cur_j > 0) {
        ok = __all_sync(~0u, mbar_wait(bar(kXQEmpty + s), n_ends & 1, abort_flag));
        ++n_ends;
      }
      if (!ok) return;
      const int node = key / a.group;
      const uint4* from =
          reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + c.b * a.q_seq + (node0 + node) * a.q_node +
                                         (c.item * a.group + key - node * a.group) * a.q_head);
      uint32_t top = 0;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        float x[8];
        unpack8<T>(key < rows ? from[i] : uint4{0, 0, 0, 0}, x);
#pragma unroll
        for (int y = 0; y < 8; ++y) top = max(top, __float_as_uint(x[y]) & 0x7FFFFFFFu);
      }
      const int shift = top == 0 || top >= 0x7F800000u ? 0 : min(14 - exponent_of(__uint_as_float(top)), 126);
      const float by = power2(shift);
      row_factor = a.scale * kLog2e * power2(-shift);
      if (!first) return;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        float x[8];
        unpack8<T>(key < rows ? from[i] : uint4{0, 0, 0, 0}, x);
        *place(0, key, i) = uint4{pack2(__half(), x[0] * by, x[4] * by), pack2(__half(), x[1] * by, x[5] * by),
                                  pack2(__half(), x[2] * by, x[6] * by), pack2(__half(), x[3] * by, x[7] * by)};
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kXQFull));
    };
    int next_page = -1;
#pragma unroll 1
    for (int j = 0; j < n_tiles && ok; ++j) {
      const bool first = j == 0 || cur.t == 0;
      if ((j & 1) != s) {   // the other stream's
        if (first) new_item(cur, false, j);
        advance<kTile, S::kGap>(a, &cur);
        if (j == 0 && n_tiles > 1) next_page = page_of(cur);
        continue;
      }
      if (j == 0) next_page = page_of(cur);
      const int use = j >> 1;   // the stream's tiles before
      if (first) new_item(cur, true, j);
      if (!ok) break;
      const int page = next_page;
      Cursor after = cur;
      if (j + 2 < n_tiles) {
        advance<kTile, S::kGap>(a, &after);
        advance<kTile, S::kGap>(a, &after);
        next_page = page_of(after);
      }
      const int st = j % kQtcStages, slot_j = j % kQtcSlots;
      ok = __all_sync(~0u, mbar_wait(bar(kCFull + slot_j), (j / kQtcSlots) & 1, abort_flag));
      if (ok && use > 0) ok = __all_sync(~0u, mbar_wait(bar(kXKEmpty + s), (use - 1) & 1, abort_flag));
      if (!ok) break;
      const unsigned char* codes = smem + S::kCodesAt + st * S::kStageBytes;
      const bool real = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.c.pages);
      if (page != -1 && !real) record_index_error(a.c.err);
      const uint32_t factors = real ? reinterpret_cast<const uint32_t*>(codes + 2 * S::kHalf)[key] : 0;
      const float ks = key_scale(factors), vs = value_scale(factors);
      const uint32_t there = __ballot_sync(~0u, real);
      // Largest and least exponents of the warp's 32 keys (128 of what is not
      // finite). A key of 0 is exact beside any other; a value of 0 is not
      // beside others, whose weights may be less than its own by any power.
      const int own_k = exponent_of(fabsf(ks)), own_v = vs != 0.f ? exponent_of(fabsf(vs)) : -kNoExp;
      const int high_k = __reduce_max_sync(~0u, ks != 0.f ? own_k : -kNoExp);
      const int low_k = __reduce_min_sync(~0u, ks != 0.f ? own_k : kNoExp);
      const int high_v = __reduce_max_sync(~0u, own_v), low_v = __reduce_min_sync(~0u, own_v);
      const int ek = max(high_k, kLeastExp), ev = max(high_v, kLeastExp);
      const bool apart = cur.t * kTile + quarter * 32 + 32 > cur.span.context || high_k - low_k > kKeySpread ||
                         low_k < kLeastExp || high_k > kMostKeyExp || high_v - low_v > kValueSpread ||
                         (low_v < kLeastExp && high_v > -kNoExp) || high_v > kMostValueExp;
      // (the scores of the stream's tile before are made, which came after the
      // weights of the one before that: nobody reads this place any more)
      QtcShared::Words& words = sh.words[s][use & 1];
      words.row_factor[key] = row_factor;
      // (operands are 2^8 times as large as values: codes of 7 at most are exact either way)
      words.key_by[key] = apart ? ks * 0x1p-8f : power2(ek - 8);
      words.value_by[key] = apart ? vs : power2(ev);
      words.value_log[key] = apart ? own_v + 1 : ev;
      if (lane == 0) {
        words.ek[quarter] = ek, words.ev[quarter] = ev;
        words.there[quarter] = there, words.apart[quarter] = apart;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kXWords + 2 * s + (use & 1)));
      unpack_row(codes, S::kKeysAt + s * S::kTileBytes, __float2half_rn(apart ? 256.f : ks * power2(8 - ek)));
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kXKFull + s));
      if (use > 0) ok = __all_sync(~0u, mbar_wait(bar(kXVEmpty + s), (use - 1) & 1, abort_flag));
      if (!ok) break;
      unpack_row(codes + S::kHalf, S::kValuesAt + s * S::kTileBytes,
                 __float2half_rn(apart ? 256.f : vs * power2(8 - ev)));
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kXVFull + s));
        if (j + kQtcStages < n_tiles) mbar_arrive(bar(kCEmpty + slot_j));
      }
      advance<kTile, S::kGap>(a, &cur);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // --------------------------------------------------------------- weights
    const int s = (warp - 4) / 4, row = (warp % 4) * 32 + lane, both = tid - 128;
    const uint32_t mine = static_cast<uint32_t>((warp % 4) * 32) << 16;   // this warp's Tensor Memory lanes
    const uint32_t scores = tmem + mine + S::kScores + s * 128, sums = tmem + mine + S::kSums + s * D;
    const int row_node = row / a.group;
    const int node = row < rows ? node0 + row_node : -1;
    int n = 0, seen_b = -1;
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
      float m = kNoMax, l = 0.f;
      int e = kLeastExp;
      bool used = false;
#pragma unroll 1
      for (int j = ja + ((ja ^ s) & 1); j < jb; j += 2) {
        const int slot0 = (cur.t + j - ja) * kTile;
        mbar_wait(bar(kXSFull + s), n & 1, abort_flag);
        mbar_wait(bar(kXWords + 2 * s + (n & 1)), (n >> 1) & 1, abort_flag);
        __syncwarp();
        tc_fence_after();
        const QtcShared::Words& words = sh.words[s][n & 1];
        const float sc = words.row_factor[row];
        uint32_t vis[4], all = ~0u;
        int apart = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          vis[w] = words.there[w];
          all &= vis[w];
          apart |= words.apart[w];
        }
        bool done = false;
        if (all == ~0u && !apart)   // a whole tile of the context
          done = weigh_q<D, false>(scores, sums, words, sc, args.zero, vis, used, bar(kXPHalf + s), bar(kXPThree + s),
                                   &m, &l, &e);
        if (!done) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int off = slot0 + w * 32 - cur.span.context;   // tree node of the word's first key
            uint32_t word = ~0u;
            if (off > -32) {
              word = off >= 0 ? __funnelshift_r(seen_word(seen, off >> 5), seen_word(seen, (off >> 5) + 1), off & 31)
                              : (seen.w[0] << -off) | ((1u << -off) - 1);
            }
            vis[w] = node >= 0 ? word & vis[w] : 0u;
          }
          weigh_q<D, true>(scores, sums, words, sc, args.zero, vis, used, bar(kXPHalf + s), bar(kXPThree + s), &m, &l,
                           &e);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kXPFull + s));
        used = true;
        ++n;
      }
      {
        // The streams' sums together; each group takes half of the columns.
        if (used) mbar_wait(bar(kXPvDone + s), (n - 1) & 1, abort_flag);
        __syncwarp();
        sh.row_max[s][row] = used && m > kNoMax ? m : -INFINITY;
        sh.row_sum[s][row] = used ? l : 0.f;
        sh.row_exp[s][row] = e;
        tc_fence_before();
        if (!group_all(3, 256, !*abort_flag)) break;
        tc_fence_after();
        const float m0 = sh.row_max[0][row], m1 = sh.row_max[1][row], top = fmaxf(m0, m1);
        const float low = top == -INFINITY ? 0.f : top;
        const float sum = exp2_approx(m0 - low) * sh.row_sum[0][row] + exp2_approx(m1 - low) * sh.row_sum[1][row];
        const float f0 = exp2_approx(m0 - low + static_cast<float>(sh.row_exp[0][row] - 8));
        const float f1 = exp2_approx(m1 - low + static_cast<float>(sh.row_exp[1][row] - 8));
        // A stream without a tile of this item has nothing in its columns.
        const bool has0 = jb - ja > 1 || (ja & 1) == 0, has1 = jb - ja > 1 || (ja & 1) == 1;
        const bool whole = cur.t == 0 && cur.nt == jb - ja;
        const bool idle = cur.span.context < 0;
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
          float z[16];   // in the order of the head again
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int from = (i & 8) + (i & 4 ? 2 * (i & 3) + 1 : 2 * (i & 3));
            z[i] = (f0 * x[from] + f1 * y[from]) * inv;
          }
          if (node < 0) continue;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              *reinterpret_cast<uint4*>(out + c + i) =
                  empty ? uint4{0, 0, 0, 0}
                        : uint4{pack2(T(), z[i], z[i + 1]), pack2(T(), z[i + 2], z[i + 3]), pack2(T(), z[i + 4], z[i + 5]),
                                pack2(T(), z[i + 6], z[i + 7])};
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) __stcg(part + (c + i) * 128 + row, z[i]);
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
  if (tid == 0 && *abort_flag) {   // given up somewhere: the copies in flight still have to land
    mbar_drain(bar(kCFull), kQtcSlots);
    atomicOr(a.c.err, kErrWait);
  }
}

}  // namespace tfx
