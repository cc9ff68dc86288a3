// Attention over a quantised cache with mma.sync, up to 8 or 16 rows a block.
//
// Reading the cache bounds it, at a quarter of the bytes of a 16-bit cache,
// so that an element has about three instructions of a lane in the time its
// bytes take. Everything is arranged to make an element cheap:
//
// * A code c + bias masked out of a word, below the exponent of 1024, is the
//   fp16 number 1024 + c + bias (or 1024 + 16 (c + bias), for the upper of two
//   nibbles): one logical instruction for two codes and one subtraction give
//   exact whole numbers, with half a shift. (Without the exponent they are
//   exact subnormals, and the subtraction could be left to the sums' start,
//   but the matrix instruction aligns products by their exponents as written,
//   and scores were off by 2^-19.)
// * Keys are the rows of A in S^T = K Q^T, values (transposed) those of A in
//   O^T = V^T P^T, and the few rows of q are columns: 16 x 16 codes an
//   instruction where A = Q would take 8 x 16.
// * The factor of a key multiplies its scores, the factor of a value its
//   weights, in fp32.
// * The order of dimensions in a product is free, if q is in the same one, so
//   each lane takes the words as they lie in a row, and the order of the keys
//   is that of the lanes that need them for the second product.
// * The four warps take different keys of a tile, each with a running maximum,
//   sum and ring of asynchronous copies of its own: they meet at an item's
//   ends only.
//
// Weights. p = 2^(s - m), s = (q . c) ks scale log2(e); O = sum of w c with w
// = p vs 2^-E rounded to fp16. m is raised when a score passes it by 8, the
// row's E when a weight would pass 2^15, so that most tiles need no exchange
// between lanes; E is about the largest p vs so far, so that factors of any
// size and range lose nothing. q is scaled by a power of two into fp16's range
// (exact but for elements 2^-39 below the row's largest).
#pragma once

#include "attend_mma.cuh"
#include "qcache.cuh"

namespace tfx {

template <int kBits, int D, int kCols>   // kCols: groups of 8 rows of a block
struct QShape {
  static constexpr int kThreads = 128;
  static constexpr int kRows = 8 * kCols;
  static constexpr int kRowBytes = D * kBits / 8;
  static constexpr int kTile = kRowBytes <= 64 ? 128 : 64;
  static constexpr int kGap = 1;
  static constexpr int kKeys = kTile / 4;             // of a warp
  static constexpr int kBlocks = D == 256 ? 2 : 3;   // an SM
  static constexpr int kStages = kRowBytes <= 32 ? 4 : 3;
  static constexpr int kHalf = kKeys * kRowBytes;     // a warp's keys or values of a tile
  static constexpr int kWarpBytes = 2 * kHalf;
  static constexpr int kStageBytes = 4 * kWarpBytes;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kNodes = TF_MAX_NODES;
  // Codes, rows of q, factors, parents; then the tree's masks.
  static constexpr int kQAt = kStages * kStageBytes;
  static constexpr int kScalesAt = kQAt + kStages * kQBytes;
  static constexpr int kParentsAt = kScalesAt + kStages * kTile * 4;
  static constexpr int kSmem = kParentsAt + kStages * kNodes * 4;
  // The warps' sums are joined in a stage that is done with, kJoinCols columns at a time.
  static constexpr int kJoinFit = kStageBytes / (4 * kRows * 4);
  static constexpr int kJoinCols = kJoinFit < D ? kJoinFit : D;
};

// A row's 16-byte chunk c of key k (of a warp's) in shared memory, so that the
// lanes that read at once meet different banks: in the first product lanes (g,
// t) read a quarter of key (g / 2) 4 + g % 2, in the second an eighth of key 4t.
template <int kRowBytes>
__device__ __forceinline__ int key_chunk(int k, int c) {
  constexpr int kChunks = kRowBytes / 16;
  const int at = k * kChunks + c;
  if (kRowBytes == 32) return at ^ (k & 4);
  if (kRowBytes >= 128) return at ^ ((k & 1) * 4);
  return at;
}
template <int kRowBytes>
__device__ __forceinline__ int value_chunk(int k, int c) {
  constexpr int kChunks = kRowBytes / 16;
  const int at = k * kChunks + c, t = k / 4 & 3;
  if (kRowBytes == 256) return at ^ ((t & 1) | (t & 2) * 2);
  return at ^ (t * 2);
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two whole numbers of a word: the lower nibbles or bytes of its halves
// (kUpper false), or the upper nibbles, 16 times as large.
template <int kBits, bool kUpper>
__device__ __forceinline__ uint32_t whole2(uint32_t w) {
  constexpr uint32_t kMask = kBits == 8 ? 0x00FF00FFu : kUpper ? 0x00F000F0u : 0x000F000Fu;
  constexpr uint32_t kFrom = kBits == 8 || kUpper ? 0x64806480u : 0x64086408u;   // 1024 + 128, 1024 + 8
  const uint32_t x = (w & kMask) | 0x64006400u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&kFrom));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void load_words(uint32_t (&w)[1], const unsigned char* p) { w[0] = *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ void load_words(uint32_t (&w)[2], const unsigned char* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  w[0] = x.x, w[1] = x.y;
}
__device__ __forceinline__ void load_words(uint32_t (&w)[4], const unsigned char* p) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
}

// 2^e for a whole e from -126 to 127.
__device__ __forceinline__ float power2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The exponent of a positive finite number, -127 for subnormal ones and 0.
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>(__float_as_uint(x) >> 23 & 255) - 127; }

template <typename T, int kBits, int D, int kCols>
__global__ void __launch_bounds__(128, QShape<kBits, D, kCols>::kBlocks)
kvq_attention_kernel(const __grid_constant__ QAttendArgs args) {
  using S = QShape<kBits, D, kCols>;
  constexpr int kTile = S::kTile, kStages = S::kStages, kKeys = S::kKeys, kRB = S::kRowBytes, kRows = S::kRows;
  constexpr int kTiles16 = kKeys / 16;        // 16-key parts of a warp's keys
  constexpr int kSteps = D / 16;              // of the first product; 16-row parts of the second
  constexpr int kWordSteps = kBits == 4 ? 2 : 1;   // steps a word of codes is good for
  const AttendArgs& a = args.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ TreeMasks<S::kNodes> masks;
  __shared__ int scratch[2 * 4 + 6];
  __shared__ uint32_t gone[4][kStages + 1];   // a warp's keys of a tile whose page is outside the pool
  __shared__ float wm[4][kRows], wl[4][kRows];
  __shared__ int last_here;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
  const int rows_all = a.nodes * a.group;
  const int row_blocks = (rows_all + kRows - 1) / kRows, team = blockIdx.x / row_blocks;
  const Rows mine{static_cast<int>(blockIdx.x) - team * row_blocks, row_blocks};
  const int row0 = mine.rb * kRows;

  chain();
  Line line;
  Cursor look;   // next tile whose pages are looked up
  const int n_tiles = find_run<kTile, S::kGap, S::kThreads>(a, gridDim.x / row_blocks, team, scratch, &line, &look);
  if (n_tiles == 0) return;
  Cursor cur = look, load = look;   // tiles computed and copied next
  const uint8_t* kp = static_cast<const uint8_t*>(a.k);
  const uint8_t* vp = static_cast<const uint8_t*>(a.v);

  // A lane has a key of its warp's: its page is asked for one tile before its
  // places are made of it (-1: not there), those one tile before the copies.
  struct Pending {
    int page, row, kvh;
    bool exists;
  };
  struct Places {
    int64_t codes, factors;
  };
  auto look_up = [&](const Cursor& c) -> Pending {
    const int slot = c.t * kTile + warp * kKeys + lane, p = a.c.by_page(slot);
    const bool exists = lane < kKeys && slot < c.span.slots;
    return {exists ? a.c.page_table[c.b * a.c.stride_table + p] : 0, slot - p * a.c.page_size, c.item, exists};
  };
  auto settle = [&](const Pending& x, int i) -> Places {
    const bool outside = x.exists && static_cast<unsigned>(x.page) >= static_cast<unsigned>(a.c.pages);
    const uint32_t none = __ballot_sync(~0u, outside);
    if (lane == 0) gone[warp][i % (kStages + 1)] = none;
    if (none && outside) record_index_error(a.c.err);
    if (!x.exists || outside) return {-1, 0};
    return {x.page * a.c.stride_page + x.row * a.c.stride_token + x.kvh * a.c.stride_head,
            x.page * args.scale_page + x.row * args.scale_token + x.kvh * args.scale_head};
  };
  // Copies of q and of the parents for the item of tile i, by all warps.
  auto issue_rows = [&](const Cursor& c, int i) {
    const uint32_t dst = smem_u32(smem + S::kQAt) + (i % kStages) * S::kQBytes;
    constexpr int kChunks = D / 8;
    for (int id = tid; id < kRows * kChunks; id += 128) {
      const int r = id / kChunks, ch = id % kChunks;
      const bool real = row0 + r < rows_all;
      const RowOf ro = row_of(a, c.item, real ? row0 + r : 0);
      copy16(dst + r * D * 2 + ((ch ^ (r & 7)) << 4),
             static_cast<const T*>(a.q) + c.b * a.q_seq + ro.node * a.q_node + ro.head * a.q_head + ch * 8, real);
    }
    if (tid < a.nodes)
      copy4(smem_u32(smem + S::kParentsAt) + ((i % kStages) * S::kNodes + tid) * 4, a.parents + c.b * a.stride_parents + tid);
  };
  // Copies of this warp's keys of tile i of the run.
  auto issue = [&](const Places& at, int i) {
    const int st = i % kStages;
    const uint32_t dst = smem_u32(smem) + st * S::kStageBytes + warp * S::kWarpBytes;
    constexpr int kChunks = kRB / 16;
#pragma unroll
    for (int n = 0; n < kKeys * kChunks / 32; ++n) {
      const int id = n * 32 + lane, key = id / kChunks, ch = id % kChunks;
      const int64_t o = __shfl_sync(~0u, at.codes, key);
      const int64_t from = o < 0 ? 0 : o + ch * 16;
      copy16(dst + key_chunk<kRB>(key, ch) * 16, kp + from, o >= 0);
      copy16(dst + S::kHalf + value_chunk<kRB>(key, ch) * 16, vp + from, o >= 0);
    }
    if (lane < kKeys)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(smem + S::kScalesAt) +
                                                                        (st * kTile + warp * kKeys + lane) * 4),
                   "l"(args.scales + at.factors), "r"(at.codes < 0 ? 0 : 4)
                   : "memory");
  };

  // The first kStages - 1 tiles, the places of the one after them.
  Places next;
  Pending ahead;
  {
    Pending first[kStages];
    issue_rows(cur, 0);
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      if (i < n_tiles) {
        first[i] = look_up(look);
        advance<kTile, S::kGap>(a, &look);
      }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (i < n_tiles) {
        if (i > 0 && load.t == 0) issue_rows(load, i);
        issue(settle(first[i], i), i);
        advance<kTile, S::kGap>(a, &load);
      }
      copies_commit();
    }
    next = {-1, 0};
    if (kStages - 1 < n_tiles) next = settle(first[kStages - 1], kStages - 1);
    ahead = {0, 0, 0, false};
    if (kStages < n_tiles) {
      ahead = look_up(look);
      advance<kTile, S::kGap>(a, &look);
    }
  }

  uint32_t qf[kCols][kSteps][2];
  float f[kCols][2];                          // of rows 2t, 2t + 1: the scores' factor
  float o[kSteps][kCols][4];
  float m[kCols][2], l[kCols][2];
  int e[kCols][2];
  int node[kCols][2];
  bool fresh = true;
  int masks_of = -1;

#pragma unroll 1
  for (int i = 0; i < n_tiles; ++i) {
    copies_wait<kStages - 2>();
    __syncwarp();
    if (i + kStages - 1 < n_tiles) {
      if (load.t == 0) issue_rows(load, i + kStages - 1);
      issue(next, i + kStages - 1);
      advance<kTile, S::kGap>(a, &load);
    }
    copies_commit();
    if (i + kStages < n_tiles) next = settle(ahead, i + kStages);
    if (i + kStages + 1 < n_tiles) {
      ahead = look_up(look);
      advance<kTile, S::kGap>(a, &look);
    }
    const int st = i % kStages;

    if (fresh) {   // a new item: its rows of q, its masks
      __syncthreads();   // all warps' copies of q have landed
      const unsigned char* q8 = smem + S::kQAt + st * S::kQBytes;
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        const int r = n * 8 + g;
        // Four (8 bits) or eight elements of row r that a word of codes has.
        auto elements = [&](int word, float (&x)[8]) {
          constexpr int kPer = 32 / kBits;
          const int first = word * kPer, ch = first / 8;
          const T* p = reinterpret_cast<const T*>(q8 + r * D * 2 + ((ch ^ (r & 7)) << 4)) + first % 8;
#pragma unroll
          for (int y = 0; y < kPer; ++y) x[y] = to_f32(p[y]);
        };
        auto word_of = [&](int w) { return kRB == 32 ? 2 * t + w : 4 * (t + w / 4 * 4) + w % 4; };
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < kSteps / kWordSteps; ++w) {
          float x[8];
          elements(word_of(w), x);
#pragma unroll
          for (int y = 0; y < 32 / kBits; ++y) top = max(top, __float_as_uint(x[y]) & 0x7FFFFFFFu);
        }
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        // q 2^shift is below 2^15
        const int shift = top == 0 || top >= 0x7F800000u ? 0 : min(14 - exponent_of(__uint_as_float(top)), 126);
        const float by = power2(shift);
        auto pair = [&](float x, float y, float upper) { return pack2(__half(), x * by * upper, y * by * upper); };
#pragma unroll
        for (int w = 0; w < kSteps / kWordSteps; ++w) {
          float x[8];
          elements(word_of(w), x);
          if constexpr (kBits == 4) {
            qf[n][2 * w][0] = pair(x[0], x[4], 1.f);
            qf[n][2 * w][1] = pair(x[2], x[6], 1.f);
            qf[n][2 * w + 1][0] = pair(x[1], x[5], 0.0625f);   // codes in the upper nibble are 16 times as large
            qf[n][2 * w + 1][1] = pair(x[3], x[7], 0.0625f);
          } else {
            qf[n][w][0] = pair(x[0], x[2], 1.f);
            qf[n][w][1] = pair(x[1], x[3], 1.f);
          }
        }
        const float back = a.scale * kLog2e * power2(-shift);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          f[n][x] = __shfl_sync(~0u, back, (2 * t + x) * 4);
          const int row = row0 + n * 8 + 2 * t + x;
          node[n][x] = row < rows_all ? row / a.group : -1;
          m[n][x] = -INFINITY, l[n][x] = 0.f, e[n][x] = -120;
        }
      }
#pragma unroll
      for (int d = 0; d < kSteps; ++d)
        for (int n = 0; n < kCols; ++n)
          for (int x = 0; x < 4; ++x) o[d][n][x] = 0.f;
      if (cur.b != masks_of) {
        masks_of = cur.b;
        masks.build(reinterpret_cast<const int*>(smem + S::kParentsAt) + st * S::kNodes, a.nodes, a.c.err);
      }
      __syncthreads();   // q's place and the parents' may be written again
      fresh = false;
    }

    const int slot0 = cur.t * kTile + warp * kKeys;
    if (slot0 < cur.span.slots) {
      const unsigned char* kt = smem + st * S::kStageBytes + warp * S::kWarpBytes;
      const unsigned char* vt = kt + S::kHalf;
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(smem + S::kScalesAt) + st * kTile + warp * kKeys;
      const uint32_t missing = gone[warp][i % (kStages + 1)];
      const bool tail = slot0 + kKeys > cur.span.context || missing;
      // This lane's keys of a part: key0 and key0 + 2 (rows g and g + 8 of A).
      const int key0 = g / 2 * 4 + g % 2;
      float s[kTiles16][kCols][4];
      uint32_t factors[kTiles16][2];
#pragma unroll
      for (int u = 0; u < kTiles16; ++u) {
        factors[u][0] = sc[u * 16 + key0], factors[u][1] = sc[u * 16 + key0 + 2];
#pragma unroll
        for (int n = 0; n < kCols; ++n)
          for (int x = 0; x < 4; ++x) s[u][n][x] = 0.f;
        constexpr int kLoad = kRB == 32 ? 2 : 4;   // words of a load
#pragma unroll
        for (int w0 = 0; w0 < kSteps / kWordSteps; w0 += kLoad) {
          uint32_t ka[kLoad], kb[kLoad];
          if (kRB == 32) {   // half a chunk
            load_words(ka, kt + key_chunk<kRB>(u * 16 + key0, t / 2) * 16 + t % 2 * 8);
            load_words(kb, kt + key_chunk<kRB>(u * 16 + key0 + 2, t / 2) * 16 + t % 2 * 8);
          } else {
            load_words(ka, kt + key_chunk<kRB>(u * 16 + key0, t + w0) * 16);
            load_words(kb, kt + key_chunk<kRB>(u * 16 + key0 + 2, t + w0) * 16);
          }
#pragma unroll
          for (int w = 0; w < kLoad; ++w) {
            const uint32_t xa = ka[w] >> 8, xb = kb[w] >> 8;
            const int step = (w0 + w) * kWordSteps;
            const uint32_t lo[4] = {whole2<kBits, false>(ka[w]), whole2<kBits, false>(kb[w]), whole2<kBits, false>(xa),
                                    whole2<kBits, false>(xb)};
#pragma unroll
            for (int n = 0; n < kCols; ++n) mma16816<__half>(s[u][n], lo, qf[n][step][0], qf[n][step][1]);
            if constexpr (kBits == 4) {
              const uint32_t hi[4] = {whole2<4, true>(ka[w]), whole2<4, true>(kb[w]), whole2<4, true>(xa), whole2<4, true>(xb)};
#pragma unroll
              for (int n = 0; n < kCols; ++n) mma16816<__half>(s[u][n], hi, qf[n][step + 1][0], qf[n][step + 1][1]);
            }
          }
        }
      }
      bool rise = false;
      float high[kCols][2];
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) high[n][x] = -INFINITY;
#pragma unroll
      for (int u = 0; u < kTiles16; ++u)
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            s[u][n][x] = s[u][n][x] * f[n][x & 1] * key_scale(factors[u][x >> 1]);
            if (tail) {
              const int key = u * 16 + key0 + (x >> 1) * 2, slot = slot0 + key, j = slot - cur.span.context;
              const int i_row = node[n][x & 1];
              bool sees = slot < cur.span.slots && i_row >= 0 && !(missing >> key & 1);
              if (sees && j >= 0) sees = masks.sees(i_row, j);
              if (!sees) s[u][n][x] = -INFINITY;
            }
            high[n][x & 1] = fmaxf(high[n][x & 1], s[u][n][x]);
          }
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) rise |= high[n][x] > m[n][x] + 8.f || (m[n][x] == -INFINITY && high[n][x] > -INFINITY);
      rise = __any_sync(~0u, rise);
      // What a risen maximum takes from the sums: 2^down; the least E may be then.
      float down[kCols][2];
      int least[kCols][2];
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) down[n][x] = 0.f, least[n][x] = e[n][x];
      if (rise) {
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float top = high[n][x];
            for (int z = 4; z < 32; z *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, z));
            if (!(top > m[n][x])) continue;   // a maximum of the whole warp: the lanes of a row agree
            down[n][x] = m[n][x] - top;
            least[n][x] = max(-120, e[n][x] + static_cast<int>(floorf(fmaxf(down[n][x], -250.f))));
            l[n][x] *= exp2_approx(down[n][x]);
            m[n][x] = top;
          }
      }
      // p, then the weights p vs over the scores.
      float most[kCols][2] = {}, base[kCols][2];
#pragma unroll
      for (int n = 0; n < kCols; ++n)
        for (int x = 0; x < 2; ++x) base[n][x] = m[n][x] == -INFINITY ? 0.f : m[n][x];
#pragma unroll
      for (int u = 0; u < kTiles16; ++u)
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float p = exp2_approx(s[u][n][x] - base[n][x & 1]);
            float w = p * value_scale(factors[u][x >> 1]);
            if (tail && s[u][n][x] == -INFINITY) w = 0.f;   // a key that is not seen, whatever its factor
            l[n][x & 1] += p;
            s[u][n][x] = w;
            most[n][x & 1] = fmaxf(most[n][x & 1], w);
          }
      bool over = rise;
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) over |= most[n][x] * power2(-e[n][x]) > 0x1p15f;
      if (__any_sync(~0u, over)) {
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float top = most[n][x];
            for (int z = 4; z < 32; z *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, z));
            const int to = min(126, max(least[n][x], exponent_of(top) + 1));
            const float by = exp2_approx(down[n][x] + static_cast<float>(e[n][x] - to));
            e[n][x] = to;
#pragma unroll
            for (int d = 0; d < kSteps; ++d) o[d][n][x] *= by, o[d][n][x + 2] *= by;
          }
      }
      float to16[kCols][2];
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) to16[n][x] = power2(-e[n][x]);
#pragma unroll
      for (int u = 0; u < kTiles16; ++u) {
        uint32_t b[kCols][2];
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            b[n][x] = transpose8(pack2(__half(), s[u][n][2 * x] * to16[n][0], s[u][n][2 * x + 1] * to16[n][1]));
        // An eighth of the rows of keys 4t .. 4t + 3.
        constexpr int kBytes = kRB / 8, kLoad = kBytes >= 16 ? 4 : kBytes / 4;
#pragma unroll
        for (int w0 = 0; w0 < kBytes / 4; w0 += kLoad) {
          uint32_t v[4][kLoad];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int at = g * kBytes + w0 * 4;
            load_words(v[z], vt + value_chunk<kRB>(u * 16 + 4 * t + z, at / 16) * 16 + at % 16);
          }
#pragma unroll
          for (int w = 0; w < kLoad; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t pick = half ? 0x7632u : 0x5410u;
              const uint32_t x = __byte_perm(v[0][w], v[1][w], pick), y = __byte_perm(v[2][w], v[3][w], pick);
              if constexpr (kBits == 4) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const uint32_t xs = z ? x >> 8 : x, ys = z ? y >> 8 : y;
                  const uint32_t c[4] = {whole2<4, false>(xs), whole2<4, true>(xs), whole2<4, false>(ys), whole2<4, true>(ys)};
#pragma unroll
                  for (int n = 0; n < kCols; ++n)
                    mma16816<__half>(o[(w0 + w) * 4 + half * 2 + z][n], c, b[n][0], b[n][1]);
                }
              } else {
                const uint32_t c[4] = {whole2<8, false>(x), whole2<8, false>(x >> 8), whole2<8, false>(y),
                                       whole2<8, false>(y >> 8)};
#pragma unroll
                for (int n = 0; n < kCols; ++n) mma16816<__half>(o[(w0 + w) * 2 + half][n], c, b[n][0], b[n][1]);
              }
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
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          for (int z = 4; z < 32; z *= 2) l[n][x] += __shfl_xor_sync(~0u, l[n][x], z);
          if (g == 0) wm[warp][n * 8 + 2 * t + x] = m[n][x], wl[warp][n * 8 + 2 * t + x] = l[n][x];
        }
      __syncthreads();   // and everyone is done with tile i
      float* sums = reinterpret_cast<float*>(smem + st * S::kStageBytes);
      float by[kCols][2];   // from this warp's units to the item's
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = n * 8 + 2 * t + x;
          const float top = fmaxf(fmaxf(wm[0][r], wm[1][r]), fmaxf(wm[2][r], wm[3][r]));
          by[n][x] = exp2_approx(m[n][x] - (top == -INFINITY ? 0.f : top) + static_cast<float>(e[n][x]));
        }
      // A lane's columns are D / 8 in a row; groups of four are rotated by the
      // row, so that the lanes that write at once meet different banks.
      constexpr int kFours = S::kJoinCols / 4;
      constexpr float kOdd = kBits == 4 ? 0.0625f : 1.f;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += S::kJoinCols) {
        if (c0) __syncthreads();
#pragma unroll
        for (int d = 0; d < kSteps; d += 2) {
          const int col = g * (D / 8) + d * 2 - c0;
          if (S::kJoinCols < D && (col < 0 || col >= S::kJoinCols)) continue;
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int r = n * 8 + 2 * t + x;
              const float z = by[n][x], zo = z * kOdd;
              *reinterpret_cast<float4*>(sums + (warp * kRows + r) * S::kJoinCols + (col / 4 + r / 2) % kFours * 4) =
                  float4{o[d][n][x] * z, o[d][n][x + 2] * zo, o[d + 1][n][x] * z, o[d + 1][n][x + 2] * zo};
            }
        }
        __syncthreads();
        for (int id = tid; id < rows * kFours; id += 128) {
          const int r = id / kFours, four = id - r * kFours, col = c0 + four * 4;
          float4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float4 z = *reinterpret_cast<const float4*>(sums + (w * kRows + r) * S::kJoinCols +
                                                              (four + r / 2) % kFours * 4);
            y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
          }
          const float top = fmaxf(fmaxf(wm[0][r], wm[1][r]), fmaxf(wm[2][r], wm[3][r]));
          const float low = top == -INFINITY ? 0.f : top;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) sum += wl[w][r] * exp2_approx(wm[w][r] - low);
          if (whole) {
            const RowOf ro = row_of(a, cur.item, row0 + r);
            const bool present = !idle && masks.sees(ro.node, ro.node);
            const bool empty = !present || sum == 0.f;
            const float inv = empty ? 0.f : 1.f / sum;
            const size_t at = (static_cast<size_t>(cur.b) * a.nodes + ro.node) * a.heads + ro.head;
            if (col == 0) a.lse[at] = empty ? -INFINITY : (top + log2f(sum)) * kLn2;
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + col) =
                empty ? uint2{0, 0} : uint2{pack2(T(), y.x * inv, y.y * inv), pack2(T(), y.z * inv, y.w * inv)};
          } else {
            *reinterpret_cast<float4*>(part + r * D + col) = y;
            if (col == 0) part[kRows * D + r] = top, part[kRows * D + kRows + r] = sum;
          }
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
          join_parts<T, kRows, D, 128>(a, line, mine, cur.b, cur.item, row0, rows, cur.first, cur.nt, idle, tid);
      }
      fresh = true;
      __syncthreads();   // the masks and the stage may be written again
    }
    advance<kTile, S::kGap>(a, &cur);
  }
}

}  // namespace tfx
