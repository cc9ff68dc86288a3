// Attention over a quantised cache with mma.sync, 8 to 32 rows a block.
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
// * Four warps take different keys of a tile, each with a running maximum and
//   sum of its own: they meet at an item's ends only. A fifth warp looks pages
//   up and copies: what a tile costs besides its arithmetic (with the four
//   warps' own copies a quarter of all instructions) is spent once for them.
//
// Weights. p = 2^(s - m), s = (q . c) ks scale log2(e); O = sum of w c with w
// = p vs 2^-E rounded to fp16. m is raised when a lane's p add up to more than
// 2^9, the row's E when a weight would pass 2^15, so that most tiles need no
// exchange between lanes; 2^E is about 2^-8 of the largest p vs so far, so that
// factors of any size and range lose nothing. Weights are rounded because the
// matrix instruction takes 16 bits beside the codes' fp16 (two parts would be
// twice the products): 2^-12 of a weight, and outputs are as far from the 64-bit
// ones as the plain form's in bf16, 1.0 to 1.2 times as far in fp16. q is scaled
// by a power of two into fp16's range: an element is off by 2^-39 of its row's
// largest at most (2^-35 where it meets upper nibbles, for which it is divided
// by 16), by nothing if it has bf16's 8 bits and is 2^-31 of it or more (2^-27).
//
// Measured, heads of 128: 32 tokens x 5 heads a kv head x 8 over up to 8,192
// slots in 4 bits 55.7 us (174 MB, 3.1 TB/s), in 8 bits 74.5 (342 MB, 4.6
// TB/s), in 4 bits over up to 32,768 160 (693 MB, 4.3 TB/s). Issue slots are
// 53% busy, the ALU 42%: half of a warp's 611 instructions for 32 keys are the
// codes' conversion. Start and end are most of the 15.2 us over up to 256
// slots. Pages of 16 slots 63.9, of 7 (no bulk copies) 75.5. With 16 rows a kv
// head 91.5: five warps a block leave 168 registers a thread, and 204 bytes are
// spilled. The wide form: 16 trees of 16 x 6 heads over up to 4,096 slots in 8
// bits 172 us, issue slots 37% busy with two arithmetic warps a scheduler.
#pragma once

#include "attend_mma.cuh"
#include "qcache.cuh"

namespace tfx {

// kCols: groups of 8 rows of a block. The narrow form has four warps of
// arithmetic and q in registers, two or three blocks an SM; the wide one, for
// more rows, eight warps (one block an SM, of which they take the registers),
// q in shared memory in the order of its fragments, and 16 keys at a time.
template <int kBits, int D, int kCols>
struct QShape {
  static constexpr bool kWide = D == 256 ? kCols == 2 : kCols == 4;
  static constexpr int kWarps = kWide ? 8 : 4;          // of arithmetic
  static constexpr int kArith = 32 * kWarps;
  static constexpr int kThreads = kWide ? 384 : 160;    // and a warp (wide: a group of four, for its registers) of copies
  static constexpr int kRows = 8 * kCols;
  static constexpr int kRowBytes = D * kBits / 8;
  static constexpr int kKeys = kRowBytes <= 64 ? 32 : 16;   // of a warp
  static constexpr int kTile = kKeys * kWarps;
  static constexpr int kGap = 1;
  static constexpr int kBlocks = kWide ? 1 : D == 256 || (D == 128 && kCols == 2) ? 2 : 3;   // an SM
  static constexpr int kStages = kRowBytes <= 32 ? 4 : kWide && kRowBytes == 256 ? 2 : 3;
  static constexpr int kHalf = kTile * kRowBytes;     // keys or values of a tile
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kNodes = TF_MAX_NODES;
  // Codes, keys before values; rows of q; factors; q's fragments.
  static constexpr int kQAt = kStages * kStageBytes;
  static constexpr int kScalesAt = kQAt + kStages * kQBytes;
  static constexpr int kFragsAt = kScalesAt + kStages * kTile * 4;
  static constexpr int kSmem = kFragsAt + (kWide ? kQBytes : 0);
  // The warps' sums are joined in a stage that is done with, kJoinCols columns at a time.
  static constexpr int kJoinFit = kStageBytes / (kWarps * kRows * 4);
  static constexpr int kJoinCols = kJoinFit < D ? kJoinFit : D;
};

// The keys of a 16-key part that lane (g, t) has. In the first product rows g
// and g + 8 of A are keys of_row(g) and of_row(g) ^ 2, in the second the pairs
// of k 2t and 2t + 8 are keys of_pair(t, 0 .. 3). Rows lie one after the other
// in shared memory, and this order keeps the lanes that read at once on
// different banks: parts of 8 and 16 bytes of rows of 64 bytes twofold in the
// second product, of longer rows fourfold, none otherwise.
__device__ __forceinline__ int of_pair(int t, int z) { return 4 * t + (z ^ (t >> 1 | (t & 1) << 1)); }
__device__ __forceinline__ int of_row(int g) { return of_pair(g >> 1, g & 1); }

// A run of bytes, by one lane: both addresses and the size multiples of 16.
__device__ __forceinline__ void copy_run(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "n"(kMask), "r"(0x64006400u));   // (w & mask) | 1024
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&kFrom));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void load_words(uint32_t (&w)[1], const unsigned char* p) {
  w[0] = *reinterpret_cast<const uint32_t*>(p);
}
__device__ __forceinline__ void load_words(uint32_t (&w)[2], const unsigned char* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  w[0] = x.x, w[1] = x.y;
}
__device__ __forceinline__ void load_words(uint32_t (&w)[4], const unsigned char* p) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
}

// A maximum before any score: every finite one is far above it, so that the
// first weights do not fit and the maximum rises, and -inf is far below it.
constexpr float kNoMax = -3.0e38f;

// 2^e for a whole e from -126 to 127.
__device__ __forceinline__ float power2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The exponent of a positive finite number, -127 for subnormal ones and 0.
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>(__float_as_uint(x) >> 23 & 255) - 127; }

template <typename T, int kBits, int D, int kCols>
__global__ void __launch_bounds__(QShape<kBits, D, kCols>::kThreads, QShape<kBits, D, kCols>::kBlocks)
kvq_attention_kernel(const __grid_constant__ QAttendArgs args) {
  using S = QShape<kBits, D, kCols>;
  constexpr int kTile = S::kTile, kStages = S::kStages, kKeys = S::kKeys, kRB = S::kRowBytes, kRows = S::kRows;
  constexpr bool kWide = S::kWide;
  constexpr int kWarps = S::kWarps, kArith = S::kArith;
  constexpr int kTiles16 = kWide ? 1 : kKeys / 16;   // 16-key parts of a warp's keys, worked on together
  constexpr int kSteps = D / 16;              // of the first product; 16-row parts of the second
  constexpr int kWordSteps = kBits == 4 ? 2 : 1;   // steps a word of codes is good for
  const AttendArgs& a = args.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ TreeMasks<S::kNodes> masks;
  __shared__ int scratch[2 * (S::kThreads / 32) + 6];
  __shared__ uint32_t gone[kStages][kTile / 32];   // keys whose page is outside the pool
  __shared__ float wm[kWarps][kRows], wl[kWarps][kRows];
  __shared__ __align__(8) float row_factor[kWide ? kRows : 2];   // of the item's scores
  __shared__ int last_here[2], given_up;
  __shared__ unsigned long long full[kStages], empty[kStages];   // a tile has landed; all warps are done with it
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
  const int rows_all = a.nodes * a.group;
  const int row_blocks = (rows_all + kRows - 1) / kRows, team = blockIdx.x / row_blocks;
  const Rows mine{static_cast<int>(blockIdx.x) - team * row_blocks, row_blocks};
  const int row0 = mine.rb * kRows;

  if (tid == 0) {
    given_up = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&full[i]), args.box ? 1 : 33);
      mbar_init(smem_u32(&empty[i]), kWarps);
    }
    fence_barrier_init();
  }
  chain();
  Line line;
  Cursor cur;   // tile computed next
  const int n_tiles = find_run<kTile, S::kGap, S::kThreads>(a, gridDim.x / row_blocks, team, scratch, &line, &cur);
  if (n_tiles == 0) return;
  const uint8_t* kp = static_cast<const uint8_t*>(a.k);
  const uint8_t* vp = static_cast<const uint8_t*>(a.v);
  auto given_up_here = [&] { return *static_cast<volatile int*>(&given_up) != 0; };

  __syncthreads();   // the barriers are there
  // Wide: the registers of 384 threads, 168 each, are shared out anew: 56 for
  // copies, twice 224 for arithmetic.
  if (warp >= kWarps) {
    if constexpr (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp > kWarps) return;
    // A tile's keys are runs of args.box slots of a page, whose codes and
    // factors lie together: a lane has a run's place, and each run is copied in
    // three pieces. Where they don't lie together (box 0) a lane has a key in
    // each 32, and all lanes copy 16 bytes at a time. A tile's pages are asked
    // for while the tile before it is waited for.
    const int rows = min(kRows, rows_all - row0);
    bool any_gone = false;
    for (int i = lane; i < kStages * kTile / 32; i += 32) gone[0][i] = 0;
    __syncwarp();
    Cursor c = cur;
    int st = 0, phase = 1, i = 0;   // phase: of the stage's last use by the other warps
    // Runs (from first_run on) of a tile whose page is outside the pool: rare, but
    // from then on every tile says which of its keys are gone.
    auto note_gone = [&](uint32_t outside, int box, int first_run, bool mine_too) {
      any_gone = true;
      if (mine_too) record_index_error(a.c.err);
      for (int word = first_run * box / 32; word < min((first_run + 32) * box, kTile) / 32; ++word) {
        uint32_t bits = 0;
        for (int z = 0; z < 32; ++z) bits |= (outside >> ((word * 32 + z) / box - first_run) & 1u) << z;
        if (lane == 0) gone[st][word] = bits;
      }
      __syncwarp();
    };
    auto stage_free = [&]() {
      return i < kStages || __all_sync(~0u, mbar_wait(smem_u32(&empty[st]), phase, &given_up));
    };
    auto pages_of = [&](const Cursor& x) { return a.c.page_table + x.b * a.c.stride_table; };
    if (args.box) {
      const int box = args.box;
      const bool has_run = lane < kTile / box;
      const uint32_t bytes = box * kRB;
      const int32_t* pages = pages_of(c);
      const uint8_t* k_head = kp + c.item * a.c.stride_head;
      const uint32_t* s_head = args.scales + c.item * args.scale_head;
      const int64_t to_values = vp - kp;
      int page = 0, row = -1;   // of the lane's run of tile i; row -1: it is not there
      auto look_up = [&]() {
        const int slot = c.t * kTile + lane * box;
        row = -1;
        if (has_run && slot < c.span.slots) {
          const int p = a.c.by_page(slot);
          page = pages[p];
          row = slot - p * a.c.page_size;
        }
      };
      look_up();
#pragma unroll 1
      for (; i < n_tiles; ++i) {
        const bool with_rows = i == 0 || c.t == 0;
        const int b = c.b, item = c.item, my_page = page, my_row = row, tile_slot = c.t * kTile;
        const uint8_t* k_at = k_head;
        const uint32_t* s_at = s_head;
        if (i + 1 < n_tiles) {
          if (++c.t == c.nt) {   // the next item
            c.t = c.nt - 1;
            advance<kTile, S::kGap>(a, &c);
            pages = pages_of(c);
            k_head = kp + c.item * a.c.stride_head;
            s_head = args.scales + c.item * args.scale_head;
          }
          look_up();
        }
        const bool real = my_row >= 0 && static_cast<uint32_t>(my_page) < static_cast<uint32_t>(a.c.pages);
        const uint32_t there = __ballot_sync(~0u, real), outside = __ballot_sync(~0u, my_row >= 0 && !real);
        if (!stage_free()) break;   // (no copy of the tile is begun)
        if (any_gone || outside) note_gone(outside, box, 0, my_row >= 0 && !real);
        const uint32_t bar = smem_u32(&full[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(there) * (2 * bytes + box * 4) + (with_rows ? rows * D * 2 : 0));
        __syncwarp();
        // What does not exist keeps an earlier tile's bytes: whatever they are, it gets no weight.
#pragma unroll 1
        for (uint32_t left = there; left; left &= left - 1) {
          const int run = __ffs(left) - 1;
          // (only the page comes from its lane, so that the rest is the warp's arithmetic)
          const uint64_t of_run = static_cast<uint32_t>(__shfl_sync(~0u, my_page, run));
          const int slot = tile_slot + run * box, row_of_run = slot - a.c.by_page(slot) * a.c.page_size;
          const uint8_t* from = k_at + of_run * a.c.stride_page + row_of_run * kRB;
          const uint32_t* with = s_at + of_run * args.scale_page + row_of_run;
          if (elect_one()) {
            const uint32_t keys = smem_u32(smem) + st * S::kStageBytes + run * bytes;
            copy_run(keys, from, bytes, bar);
            copy_run(keys + S::kHalf, from + to_values, bytes, bar);
            copy_run(smem_u32(smem + S::kScalesAt) + (st * kTile + run * box) * 4, with, box * 4, bar);
          }
          __syncwarp();
        }
        if (with_rows && lane < rows) {   // 32 rows at most
          const RowOf ro = row_of(a, item, row0 + lane);
          copy_run(smem_u32(smem + S::kQAt) + st * S::kQBytes + lane * D * 2,
                   static_cast<const T*>(a.q) + b * a.q_seq + ro.node * a.q_node + ro.head * a.q_head, D * 2, bar);
        }
        if (++st == kStages) st = 0, phase ^= 1;
      }
    } else {
      constexpr int kChunks = kRB / 16, kRowChunks = D / 8;
#pragma unroll 1
      for (; i < n_tiles; ++i) {
        const int32_t* pages = pages_of(c);
        struct Look {
          int page, row;   // row -1: not there
        };
        auto look = [&](int k) -> Look {
          const int slot = c.t * kTile + k * 32 + lane, p = a.c.by_page(slot);
          return slot < c.span.slots ? Look{pages[p], slot - p * a.c.page_size} : Look{0, -1};
        };
        Look next = look(0);
        if (!stage_free()) break;
        const uint32_t bar = smem_u32(&full[st]), keys = smem_u32(smem) + st * S::kStageBytes;
        if (i == 0 || c.t == 0)
          for (int id = lane; id < rows * kRowChunks; id += 32) {
            const RowOf ro = row_of(a, c.item, row0 + id / kRowChunks);
            copy16(smem_u32(smem + S::kQAt) + st * S::kQBytes + id * 16,
                   static_cast<const T*>(a.q) + c.b * a.q_seq + ro.node * a.q_node + ro.head * a.q_head +
                       id % kRowChunks * 8,
                   true);
          }
#pragma unroll 1
        for (int k = 0; k < kTile / 32; ++k) {
          const Look x = next;
          if (k + 1 < kTile / 32) next = look(k + 1);
          const bool real = x.row >= 0 && static_cast<uint32_t>(x.page) < static_cast<uint32_t>(a.c.pages);
          const uint32_t outside = __ballot_sync(~0u, x.row >= 0 && !real);
          if (any_gone || outside) note_gone(outside, 1, k * 32, x.row >= 0 && !real);
          const int64_t at = real ? x.page * a.c.stride_page + x.row * a.c.stride_token + c.item * a.c.stride_head : -1;
          const uint32_t into = keys + (k * 32 * kChunks + lane) * 16;
#pragma unroll 4
          for (int n = 0; n < kChunks; ++n) {
            const int id = n * 32 + lane;
            const int64_t from = __shfl_sync(~0u, at, id / kChunks);
            if (from >= 0) {
              copy16(into + n * 512, kp + from + id % kChunks * 16, true);
              copy16(into + n * 512 + S::kHalf, vp + from + id % kChunks * 16, true);
            }
          }
          if (real)
            copy4(smem_u32(smem + S::kScalesAt) + (st * kTile + k * 32 + lane) * 4,
                  args.scales + x.page * args.scale_page + x.row * args.scale_token + c.item * args.scale_head);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        if (lane == 0) mbar_arrive(bar);   // for gone[], which no copy writes
        advance<kTile, S::kGap>(a, &c);
        if (++st == kStages) st = 0, phase ^= 1;
      }
    }
    // Every copy has landed before the others are through, unless a wait gave
    // up: then before this warp or the others leave, whichever see it.
    if (given_up_here()) {
      mbar_drain(smem_u32(&full[0]), kStages);
      if (lane == 0) atomicOr(a.c.err, kErrWait);
    }
    return;
  }
  if constexpr (kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
  // The warps of arithmetic meet here.
  auto meet = [] { asm volatile("barrier.sync 1, %0;" ::"n"(kArith) : "memory"); };

  uint32_t qf[kWide ? 1 : kCols][kWide ? 1 : kSteps][2];
  uint2* frags = reinterpret_cast<uint2*>(smem + S::kFragsAt) + lane;   // of group n and step k at (n kSteps + k) 32
  float f[kWide ? 1 : kCols][2];              // of rows 2t, 2t + 1: the scores' factor
  float o[kSteps][kCols][4];
  float m[kCols][2], l[kCols][2];
  int e[kCols][2];
  struct Part {   // an item that other runs have parts of
    int b, item, first, nt;
    bool idle;
  } parts[2];
  int n_parts = 0;
  bool fresh = true;
  int masks_of = cur.b;
  masks.build(a.parents + cur.b * a.stride_parents, a.nodes, a.c.err, meet);   // while the first tile is on its way

  int st = 0, phase = 0;
#pragma unroll 1
  for (int i = 0; i < n_tiles; ++i) {
    mbar_wait(smem_u32(&full[st]), phase, &given_up);
    __syncwarp();

    if (fresh) {   // a new item: its rows of q, its masks
      const unsigned char* q8 = smem + S::kQAt + st * S::kQBytes;
#pragma unroll
      for (int n0 = 0; n0 < (kWide ? 1 : kCols); ++n0) {
        const int n = kWide ? warp : n0;   // wide: a group a warp
        if (kWide && n >= kCols) break;
        const int r = n * 8 + g;
        // The elements of row r that this lane's words of codes have, eight or
        // (8 bits) four of them a word, in 16-byte pieces.
        constexpr int kPieces = D / 32;
        auto piece_of = [&](int i) {   // of the row's D / 8
          if (kBits == 8) return kRB == 64 ? t * 2 + i : t * 2 + i / 2 * 8 + i % 2;
          return kRB == 32 ? t * 2 + i : t * 4 + i / 4 * 16 + i % 4;
        };
        uint4 raw[kPieces];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          raw[i] = row0 + r < rows_all ? reinterpret_cast<const uint4*>(q8)[r * (D / 8) + piece_of(i)] : uint4{0, 0, 0, 0};
          float x[8];
          unpack8<T>(raw[i], x);
#pragma unroll
          for (int y = 0; y < 8; ++y) top = max(top, __float_as_uint(x[y]) & 0x7FFFFFFFu);
        }
        top = max(top, __shfl_xor_sync(~0u, top, 1));
        top = max(top, __shfl_xor_sync(~0u, top, 2));
        // q 2^shift is below 2^15
        const int shift = top == 0 || top >= 0x7F800000u ? 0 : min(14 - exponent_of(__uint_as_float(top)), 126);
        const float by = power2(shift);
        auto pair = [&](float x, float y, float upper) { return pack2(__half(), x * by * upper, y * by * upper); };
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          float x[8];
          unpack8<T>(raw[i], x);
          auto keep = [&](int step, uint32_t b0, uint32_t b1) {
            if (kWide) frags[(n * kSteps + step) * 32] = uint2{b0, b1};
            else qf[kWide ? 0 : n0][kWide ? 0 : step][0] = b0, qf[kWide ? 0 : n0][kWide ? 0 : step][1] = b1;
          };
          if constexpr (kBits == 4) {
            keep(2 * i, pair(x[0], x[4], 1.f), pair(x[2], x[6], 1.f));
            keep(2 * i + 1, pair(x[1], x[5], 0.0625f), pair(x[3], x[7], 0.0625f));   // upper codes are 16 times as large
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y)
              keep(2 * i + y, pair(x[4 * y], x[4 * y + 2], 1.f), pair(x[4 * y + 1], x[4 * y + 3], 1.f));
          }
        }
        const float back = a.scale * kLog2e * power2(-shift);
        if (kWide) {
          if (t == 0) row_factor[r] = back;
        } else {
#pragma unroll
          for (int x = 0; x < 2; ++x) f[kWide ? 0 : n0][x] = __shfl_sync(~0u, back, (2 * t + x) * 4);
        }
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) m[n][x] = kNoMax, l[n][x] = 0.f, e[n][x] = -120;
#pragma unroll
      for (int d = 0; d < kSteps; ++d)
        for (int n = 0; n < kCols; ++n)
          for (int x = 0; x < 4; ++x) o[d][n][x] = 0.f;
      if (cur.b != masks_of) {   // (everybody is through with the item before: they met at its end)
        masks_of = cur.b;
        masks.build(a.parents + cur.b * a.stride_parents, a.nodes, a.c.err, meet);
      }
      if (kWide) meet();   // q is there
      fresh = false;
    }

    const int slot0 = cur.t * kTile + warp * kKeys;
    if (slot0 < cur.span.slots) {
      const unsigned char* kt = smem + st * S::kStageBytes + warp * kKeys * kRB;
      const unsigned char* vt = kt + S::kHalf;
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(smem + S::kScalesAt) + st * kTile + warp * kKeys;
      const uint32_t missing = kKeys == 32 ? gone[st][warp] : gone[st][warp / 2] >> (warp % 2 * 16) & 0xFFFFu;
      const bool tail = slot0 + kKeys > cur.span.context || missing;
      // This lane's keys of a part: key0 and key0 ^ 2 (rows g and g + 8 of A).
      const int key0 = of_row(g);
#pragma unroll 1
      for (int part0 = 0; part0 < kKeys; part0 += 16 * kTiles16, kt += 16 * kTiles16 * kRB, vt += 16 * kTiles16 * kRB) {
      if (kWide && slot0 + part0 >= cur.span.slots) break;
      auto q_of = [&](int n, int step) {
        return kWide ? frags[(n * kSteps + step) * 32]
                     : uint2{qf[kWide ? 0 : n][kWide ? 0 : step][0], qf[kWide ? 0 : n][kWide ? 0 : step][1]};
      };
      float s[kTiles16][kCols][4];
      uint32_t factors[kTiles16][2];
#pragma unroll
      for (int u = 0; u < kTiles16; ++u) {
        factors[u][0] = sc[part0 + u * 16 + key0], factors[u][1] = sc[part0 + u * 16 + (key0 ^ 2)];
#pragma unroll
        for (int n = 0; n < kCols; ++n)
          for (int x = 0; x < 4; ++x) s[u][n][x] = 0.f;
        constexpr int kLoad = kRB == 32 ? 2 : 4;   // words of a load
#pragma unroll
        for (int w0 = 0; w0 < kSteps / kWordSteps; w0 += kLoad) {
          uint32_t ka[kLoad], kb[kLoad];
          const int quarter = kRB == 32 ? t * 8 : (t + w0) * 16;
          load_words(ka, kt + (u * 16 + key0) * kRB + quarter);
          load_words(kb, kt + (u * 16 + (key0 ^ 2)) * kRB + quarter);
#pragma unroll
          for (int w = 0; w < kLoad; ++w) {
            const uint32_t xa = ka[w] >> 8, xb = kb[w] >> 8;
            const int step = (w0 + w) * kWordSteps;
            const uint32_t lo[4] = {whole2<kBits, false>(ka[w]), whole2<kBits, false>(kb[w]), whole2<kBits, false>(xa),
                                    whole2<kBits, false>(xb)};
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
              const uint2 b = q_of(n, step);
              mma16816<__half>(s[u][n], lo, b.x, b.y);
            }
            if constexpr (kBits == 4) {
              const uint32_t hi[4] = {whole2<4, true>(ka[w]), whole2<4, true>(kb[w]), whole2<4, true>(xa),
                                      whole2<4, true>(xb)};
#pragma unroll
              for (int n = 0; n < kCols; ++n) {
                const uint2 b = q_of(n, step + 1);
                mma16816<__half>(s[u][n], hi, b.x, b.y);
              }
            }
          }
        }
      }
      // Scores in units of log 2; -inf for a key that is not seen.
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        const float2 by = kWide ? *reinterpret_cast<const float2*>(row_factor + (n * 8 + 2 * t) % (kWide ? kRows : 2))
                                : float2{f[kWide ? 0 : n][0], f[kWide ? 0 : n][1]};
#pragma unroll
        for (int u = 0; u < kTiles16; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x)   // (factors first: a score may pass fp32's range without the key's; rounded, as m is)
            s[u][n][x] = __fmul_rn(s[u][n][x], (x & 1 ? by.y : by.x) * key_scale(factors[u][x >> 1]));
      }
      if (tail) {
#pragma unroll
        for (int u = 0; u < kTiles16; ++u)
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = part0 + u * 16 + (key0 ^ (x & 2)), slot = slot0 + key, j = slot - cur.span.context;
              const int row = row0 + n * 8 + 2 * t + (x & 1), i_row = row < rows_all ? row / a.group : -1;
              bool sees = slot < cur.span.slots && i_row >= 0 && !(missing >> key & 1);
              if (sees && j >= 0) sees = masks.sees(i_row, j);
              if (!sees) s[u][n][x] = -INFINITY;
            }
      }
      // p = 2^(s - m) and the weights p vs 2^-E. Where a row's maximum or its
      // E has to rise they are worked out again: at an item's first tile, and
      // seldom after it.
      float w[kTiles16][kCols][4], sum[kCols][2];
      bool over = false;
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float to16 = power2(-e[n][x]);   // 2^-E
          float largest = sum[n][x] = 0.f;   // (a bad value that the row does not see, NaN here, is passed over)
#pragma unroll
          for (int u = 0; u < kTiles16; ++u)
#pragma unroll
            for (int y = x; y < 4; y += 2) {
              const float p = exp2_approx(s[u][n][y] - m[n][x]);
              sum[n][x] += p;
              w[u][n][y] = p * value_scale(factors[u][y >> 1]) * to16;   // (vs 2^-E alone may be infinite, p 0)
              largest = fmaxf(largest, fabsf(w[u][n][y]));
            }
          over |= sum[n][x] > 0x1p9f || largest > 0x1p15f;
        }
      if (__any_sync(~0u, over)) {
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float high = -INFINITY;
#pragma unroll
            for (int u = 0; u < kTiles16; ++u) high = fmaxf(high, fmaxf(s[u][n][x], s[u][n][x + 2]));
            for (int z = 4; z < 32; z *= 2) high = fmaxf(high, __shfl_xor_sync(~0u, high, z));
            // What the maximum takes from the sums, 2^down, and the least E may be then.
            float down = 0.f;
            int least = e[n][x];
            if (high > m[n][x]) {
              down = m[n][x] - high;
              least = max(-120, least + static_cast<int>(floorf(fmaxf(down, -250.f))));
              l[n][x] *= exp2_approx(down);
              m[n][x] = high;
            }
            float most = 0.f;
            sum[n][x] = 0.f;
#pragma unroll
            for (int u = 0; u < kTiles16; ++u)
#pragma unroll
              for (int y = x; y < 4; y += 2) {
                const float p = exp2_approx(s[u][n][y] - m[n][x]);
                sum[n][x] += p;
                w[u][n][y] = p * value_scale(factors[u][y >> 1]);
                most = fmaxf(most, fabsf(w[u][n][y]));
              }
            for (int z = 4; z < 32; z *= 2) most = fmaxf(most, __shfl_xor_sync(~0u, most, z));
            const int to = min(126, max(least, exponent_of(most) - 7));   // the largest weight is below 2^8
            const float by = exp2_approx(down + static_cast<float>(e[n][x] - to));
            e[n][x] = to;
            const float to16 = power2(-to);
#pragma unroll
            for (int u = 0; u < kTiles16; ++u) w[u][n][x] *= to16, w[u][n][x + 2] *= to16;
#pragma unroll
            for (int d = 0; d < kSteps; ++d) o[d][n][x] *= by, o[d][n][x + 2] *= by;
          }
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) l[n][x] += sum[n][x];
      if (tail) {   // no weight for a key that is not seen, whatever its factor
#pragma unroll
        for (int u = 0; u < kTiles16; ++u)
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (s[u][n][x] == -INFINITY) w[u][n][x] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < kTiles16; ++u) {
        uint32_t b[kCols][2];
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            b[n][x] = transpose8(pack2(__half(), w[u][n][2 * x], w[u][n][2 * x + 1]));
        // An eighth of the rows of the lane's four keys.
        constexpr int kBytes = kRB / 8, kLoad = kBytes >= 16 ? 4 : kBytes / 4;
#pragma unroll
        for (int w0 = 0; w0 < kBytes / 4; w0 += kLoad) {
          uint32_t v[4][kLoad];
#pragma unroll
          for (int z = 0; z < 4; ++z) load_words(v[z], vt + (u * 16 + of_pair(t, z)) * kRB + g * kBytes + w0 * 4);
#pragma unroll
          for (int i_w = 0; i_w < kLoad; ++i_w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t pick = half ? 0x7632u : 0x5410u;
              const uint32_t x = __byte_perm(v[0][i_w], v[1][i_w], pick), y = __byte_perm(v[2][i_w], v[3][i_w], pick);
              if constexpr (kBits == 4) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const uint32_t xs = z ? x >> 8 : x, ys = z ? y >> 8 : y;
                  const uint32_t c[4] = {whole2<4, false>(xs), whole2<4, true>(xs), whole2<4, false>(ys),
                                         whole2<4, true>(ys)};
#pragma unroll
                  for (int n = 0; n < kCols; ++n)
                    mma16816<__half>(o[(w0 + i_w) * 4 + half * 2 + z][n], c, b[n][0], b[n][1]);
                }
              } else {
                const uint32_t c[4] = {whole2<8, false>(x), whole2<8, false>(x >> 8), whole2<8, false>(y),
                                       whole2<8, false>(y >> 8)};
#pragma unroll
                for (int n = 0; n < kCols; ++n) mma16816<__half>(o[(w0 + i_w) * 2 + half][n], c, b[n][0], b[n][1]);
              }
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
          if (m[n][x] <= kNoMax) m[n][x] = -INFINITY;
          if (g == 0) wm[warp][n * 8 + 2 * t + x] = m[n][x], wl[warp][n * 8 + 2 * t + x] = l[n][x];
        }
      meet();   // and everyone is done with tile i
      float* sums = reinterpret_cast<float*>(smem + st * S::kStageBytes);
      float by[kCols][2];   // from this warp's units to the item's
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = n * 8 + 2 * t + x;
          float top = wm[0][r];
          for (int w = 1; w < kWarps; ++w) top = fmaxf(top, wm[w][r]);
          by[n][x] = exp2_approx(m[n][x] - (top == -INFINITY ? 0.f : top) + static_cast<float>(e[n][x]));
        }
      // A lane's columns are D / 8 in a row; groups of four are rotated by the
      // row, so that the lanes that write at once meet different banks.
      constexpr int kFours = S::kJoinCols / 4;
      constexpr float kOdd = kBits == 4 ? 0.0625f : 1.f;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += S::kJoinCols) {
        if (c0) meet();
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
        meet();
        for (int id = tid; id < rows * kFours; id += kArith) {
          const int r = id / kFours, four = id - r * kFours, col = c0 + four * 4;
          float4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 z = *reinterpret_cast<const float4*>(sums + (w * kRows + r) * S::kJoinCols +
                                                              (four + r / 2) % kFours * 4);
            y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
          }
          float top = wm[0][r];
          for (int w = 1; w < kWarps; ++w) top = fmaxf(top, wm[w][r]);
          const float low = top == -INFINITY ? 0.f : top;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sum += wl[w][r] * exp2_approx(wm[w][r] - low);
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
      if (!whole && !a.join_later) {   // at most twice: of the run's first and of its last item
        parts[n_parts].b = cur.b, parts[n_parts].item = cur.item;
        parts[n_parts].first = cur.first, parts[n_parts].nt = cur.nt;
        parts[n_parts].idle = idle;
        ++n_parts;
      }
      fresh = true;
      fence_proxy_async_shared();
      meet();   // the masks and the stage may be written again
    }
    __syncwarp();
    if (lane == 0 && i + kStages < n_tiles) mbar_arrive(smem_u32(&empty[st]));
    if (++st == kStages) st = 0, phase ^= 1;
    advance<kTile, S::kGap>(a, &cur);
  }
  // Parts are counted when the run is through: counting takes a fence and a
  // round trip to memory, 2 us that each of the two would hold the run up for.
  if (n_parts > 0) {
    meet();
    if (tid == 0) {
      __threadfence();
      for (int x = 0; x < 2; ++x) last_here[x] = x < n_parts && arrives_last(a, line, mine, parts[x].first, parts[x].nt);
      __threadfence();
    }
    meet();
    for (int x = 0; x < 2; ++x)
      if (last_here[x])
        join_parts<T, kRows, D, kArith>(a, line, mine, parts[x].b, parts[x].item, row0, min(kRows, rows_all - row0),
                                     parts[x].first, parts[x].nt, parts[x].idle, tid);
  }
  // (these warps have met since the last of their waits)
  if (threadIdx.x == 0 && given_up_here()) {
    mbar_drain(smem_u32(&full[0]), kStages);
    atomicOr(a.c.err, kErrWait);
  }
}

}  // namespace tfx
