// Launch of the attention of a drafted token tree over a quantised paged cache
// (tf_kvq_attention).
#include <algorithm>
#include <numeric>

#include "attend_qtc.cuh"

namespace tfx {
namespace {

constexpr int kMaxDevices = 64;

// Blocks of a launch with `blocks` places: whole teams of row_blocks, one at least.
int team_blocks(int blocks, int row_blocks) { return std::max(1, blocks / row_blocks) * row_blocks; }

// Slots that are copied at once: the most that divide both a page and a tile,
// where their rows lie one after the other, and their factors too, at multiples
// of 16 bytes; 0 where they don't.
int run_of_slots(const QAttendArgs& x, int tile, int row_bytes) {
  const CacheView& c = x.a.c;
  const int box = std::gcd(c.page_size, tile);
  const bool together = c.stride_token == row_bytes && x.scale_token == 1 && ((x.scale_page | x.scale_head) & 3) == 0 &&
                        (reinterpret_cast<uintptr_t>(x.scales) & 15) == 0;
  return together && box >= std::max(4, tile / 32) ? box : 0;   // a lane has a run
}

// Parts of an item above which a launch of its own joins them, where a run may
// have kLongRun tiles and where it can't. 16 tokens over up to 8,192 slots (3
// parts) 35.9 us with the launch, 37.5 with the block that comes last; 32 (1
// part) 56.4 and 55.1, over up to 256 17.8 and 14.4. With short runs a call
// outside a graph is bound by the host, for which a second launch is 2 us: one
// token over 300 slots (3 parts) 14.8 with it and 12.6 without, call after
// call, 6 chains of 5 over up to 1,500 (4 parts) 16.1 and 14.3 (in a graph 11.8
// and 13.8, 15.8 and 16.4).
constexpr int kManyParts = 2, kManyPartsOfShort = 6, kLongRun = 4;

template <typename T, int kBits, int D, int kCols>
cudaError_t launch(QAttendArgs x, int device, cudaStream_t s) {
  using S = QShape<kBits, D, kCols>;
  static_assert(S::kBlocks <= kMostBlocksPerSm, "the workspace has room for these");
  AttendArgs& a = x.a;
  static PerDeviceOnce<kMaxDevices> once;
  const int e = once.run(device, cudaErrorInvalidDevice, [] {
    return static_cast<int>(cudaFuncSetAttribute(kvq_attention_kernel<T, kBits, D, kCols>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
  });
  if (e != cudaSuccess) return static_cast<cudaError_t>(e);
  const int row_blocks = (a.nodes * a.group + S::kRows - 1) / S::kRows;
  const int blocks = team_blocks(S::kBlocks * a.num_sms, row_blocks);
  const int64_t runs = blocks / row_blocks;
  const int64_t tiles = (static_cast<int64_t>(a.c.table_width) * a.c.page_size + S::kTile - 1) / S::kTile;
  const bool long_runs = tiles * a.c.batch * a.c.kv_heads >= kLongRun * runs;
  a.join_later = parts_of(a, runs, S::kTile) > (long_runs ? kManyParts : kManyPartsOfShort);
  x.box = run_of_slots(x, S::kTile, S::kRowBytes);
  const cudaError_t launched =
      launch_chained(kvq_attention_kernel<T, kBits, D, kCols>, dim3(blocks), dim3(S::kThreads), S::kSmem, 1, s, x);
  if (launched != cudaSuccess || !a.join_later) return launched;
  return launch_join<T, S::kRows, D, S::kTile, S::kGap>(a, blocks / row_blocks, row_blocks, S::kRows, s);
}

// More than kManyRows rows of 4 bits a kv head.
template <typename T, int D>
cudaError_t launch_tc(QAttendArgs x, int device, cudaStream_t s) {
  using S = QtcShape<D>;
  AttendArgs& a = x.a;
  static PerDeviceOnce<kMaxDevices> once;
  const int e = once.run(device, cudaErrorInvalidDevice, [] {
    return static_cast<int>(
        cudaFuncSetAttribute(kvq_attention_tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
  });
  if (e != cudaSuccess) return static_cast<cudaError_t>(e);
  x.box = run_of_slots(x, S::kTile, S::kRowBytes);
  const QtcArgs args = {x, std::min(S::kTile / a.group, a.nodes), 0.f};
  const int row_blocks = (a.nodes + args.block_nodes - 1) / args.block_nodes;
  const int blocks = team_blocks(a.num_sms, row_blocks);
  const cudaError_t launched =
      launch_chained(kvq_attention_tc_kernel<T, D>, dim3(blocks), dim3(S::kThreads), S::kSmem, 1, s, args);
  // No item has a second tile to be cut off.
  if (launched != cudaSuccess || static_cast<int64_t>(a.c.table_width) * a.c.page_size <= S::kTile) return launched;
  return launch_join<T, 128, D, S::kTile, S::kGap>(a, blocks / row_blocks, row_blocks, args.block_nodes * a.group, s);
}

// 24 rows a kv head (trees) 52 us with tcgen05 and 65 with mma.sync's wide
// form, 20 (32 tokens over up to 8,192 slots) 131 and 151. Up to 16 mma.sync
// has all rows in one block: 16 of them take 93 us.
constexpr int kManyRows = 16;

template <typename T, int kBits>
cudaError_t by_dim(const QAttendArgs& x, int device, cudaStream_t s) {
  const int rows = x.a.nodes * x.a.group;
  if constexpr (kBits == 4)
    if (rows > kManyRows && x.a.group <= 128 && x.a.scale >= 0.f && x.a.c.head_dim != 256)
      return x.a.c.head_dim == 64 ? launch_tc<T, 64>(x, device, s) : launch_tc<T, 128>(x, device, s);
  switch (x.a.c.head_dim) {
    case 64:
      return rows <= 8 ? launch<T, kBits, 64, 1>(x, device, s)
             : rows <= 16 ? launch<T, kBits, 64, 2>(x, device, s) : launch<T, kBits, 64, 4>(x, device, s);
    case 128:
      return rows <= 8 ? launch<T, kBits, 128, 1>(x, device, s)
             : rows <= 16 ? launch<T, kBits, 128, 2>(x, device, s) : launch<T, kBits, 128, 4>(x, device, s);
    default: return rows <= 8 ? launch<T, kBits, 256, 1>(x, device, s) : launch<T, kBits, 256, 2>(x, device, s);
  }
}

}  // namespace

// A counter for each part (their number and place depend on the device alone;
// a launch with more blocks of rows than places has one run, and nothing to
// join), then two parts for each block of the launch: 16 rows, or 32
// where a block has an SM to itself.
AttendWorkspace kvq_attend_workspace(int nodes, int heads, int kv_heads, int head_dim, int num_sms) {
  const int64_t rows = static_cast<int64_t>(nodes) * (heads / kv_heads);
  const size_t places = static_cast<size_t>(kMostBlocksPerSm) * num_sms;
  AttendWorkspace w;
  w.partials_at = attend_counter_bytes(num_sms);
  size_t part_rows = std::max<size_t>(places, (rows + 7) / 8) * 16;
  // Blocks of rows of the tcgen05 kernel hold whole nodes, of 128 rows at most.
  if (rows > kManyRows) part_rows = std::max(part_rows, std::max<size_t>(num_sms, nodes) * 128);
  w.bytes = w.partials_at + 2 * part_rows * (head_dim + 2) * sizeof(float);
  return w;
}

cudaError_t launch_kvq_attention(const QAttendArgs& x, int dtype, int bits, int device, cudaStream_t s) {
  if (dtype == TF_F16) return bits == 4 ? by_dim<__half, 4>(x, device, s) : by_dim<__half, 8>(x, device, s);
  return bits == 4 ? by_dim<__nv_bfloat16, 4>(x, device, s) : by_dim<__nv_bfloat16, 8>(x, device, s);
}

}  // namespace tfx
