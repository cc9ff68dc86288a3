// Launch of the attention of a drafted token tree over a paged cache
// (tf_tree_attention).
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <numeric>

#include "attend_tc.cuh"

namespace tfx {
namespace {

constexpr int kMaxDevices = 64;

// Rows a kv head up to which the 16-row mma.sync kernel takes them in one
// block, with two blocks an SM; above, the tcgen05 kernel, whose tiles have
// 128 rows and whose one block an SM starts and ends slower. 8 sequences of
// 4,096 slots, 8 kv heads of 128: 16 rows 36.3 us on mma.sync, 39.3 on
// tcgen05; 17 rows 58.0 (blocks of 64 rows) and 39.4; 128 rows 104 and 45.
// 1 sequence of 2,000: 16 rows 11.5 and 14.4; 24 rows 14.6 and 14.4.
constexpr int kFewRows = 16;

// Blocks of a launch with `blocks` places: whole teams of row_blocks, one at least.
int team_blocks(int blocks, int row_blocks) { return std::max(1, blocks / row_blocks) * row_blocks; }

// Parts of an item above which a launch of its own joins them. 304 parts: 22
// us with the launch, 53 us with the last block; 38 parts 15.7 and 20.0; 9
// parts 21.2 and 22.5; 1 to 4 parts level.
constexpr int kManyParts = 6;

template <typename T, int D, int kRowWarps>
cudaError_t launch_mma(AttendArgs a, int device, cudaStream_t s) {
  using S = MmaShape<D, kRowWarps>;
  static PerDeviceOnce<kMaxDevices> once;
  const int e = once.run(device, cudaErrorInvalidDevice, [] {
    return static_cast<int>(cudaFuncSetAttribute(tree_attention_mma_kernel<T, D, kRowWarps>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
  });
  if (e != cudaSuccess) return static_cast<cudaError_t>(e);
  const int row_blocks = (a.nodes * a.group + S::kRows - 1) / S::kRows;
  const int blocks = team_blocks(kBlocksPerSm * a.num_sms, row_blocks);
  a.join_later = parts_of(a, blocks / row_blocks, S::kTile) > kManyParts;
  const cudaError_t launched = launch_chained(tree_attention_mma_kernel<T, D, kRowWarps>, dim3(blocks),
                                              dim3(S::kThreads), S::kSmem, 1, s, a);
  if (launched != cudaSuccess || !a.join_later) return launched;
  return launch_join<T, S::kRows, D, S::kTile, S::kGap>(a, blocks / row_blocks, row_blocks, S::kRows, s);
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A map of 16-bit elements over (n0, n1, n2, n3) with strides of the last
// three in elements, boxes of (64, b1, b2, 1) with the 128-byte swizzle.
bool make_map(CUtensorMap* map, bool half, const void* at, const int64_t (&n)[4], const int64_t (&stride)[3], int b1,
              int b2) {
  cuuint64_t dims[4], strides[3];
  for (int i = 0; i < 4; ++i) dims[i] = static_cast<cuuint64_t>(n[i]);
  // A dimension of one element has any stride.
  for (int i = 0; i < 3; ++i) strides[i] = n[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(stride[i]) * 2;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2), 1}, ones[4] = {1, 1, 1, 1};
  auto encode = map_encoder();
  return encode && encode(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                          const_cast<void*>(at), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B,
                          // a row of 64 elements has another head's row beside it
                          n[0] == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch_tc(const AttendArgs& a, int box, int device, cudaStream_t s) {
  using S = TcShape<D>;
  static PerDeviceOnce<kMaxDevices> once;
  const int e = once.run(device, cudaErrorInvalidDevice, [] {
    return static_cast<int>(cudaFuncSetAttribute(tree_attention_tc_kernel<T, D>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
  });
  if (e != cudaSuccess) return static_cast<cudaError_t>(e);
  const bool half = std::is_same<T, __half>::value;
  TcArgs args;
  args.a = a;
  args.block_nodes = std::min(S::kTile / a.group, a.nodes);
  args.box = box;
  TcMaps maps;
  const CacheView& c = a.c;
  if (!make_map(&maps.q, half, a.q, {D, a.heads, a.nodes, c.batch}, {a.q_head, a.q_node, a.q_seq}, a.group,
                args.block_nodes) ||
      !make_map(&maps.k, half, a.k, {D, c.page_size, c.kv_heads, c.pages},
                {c.stride_token, c.stride_head, c.stride_page}, box, 1) ||
      !make_map(&maps.v, half, a.v, {D, c.page_size, c.kv_heads, c.pages},
                {c.stride_token, c.stride_head, c.stride_page}, box, 1))
    return cudaErrorInvalidValue;
  const int row_blocks = (a.nodes + args.block_nodes - 1) / args.block_nodes;
  const int blocks = team_blocks(a.num_sms, row_blocks);
  const cudaError_t launched =
      launch_chained(tree_attention_tc_kernel<T, D>, dim3(blocks), dim3(S::kThreads), S::kSmem, 1, s, maps, args);
  // No item has a second tile to be cut off.
  if (launched != cudaSuccess || static_cast<int64_t>(c.table_width) * c.page_size <= S::kTile) return launched;
  return launch_join<T, 128, D, S::kTile, S::kGap>(a, blocks / row_blocks, row_blocks, args.block_nodes * a.group, s);
}

// Rows of a copy for the tcgen05 kernel: the largest that divides both the
// tile and the page, 0 where the call does not suit the kernel (heads of 256,
// pages that are no multiple of 8 rows, more heads a kv head than a tile has
// rows, a stride of 0 that repeats an element, a negative scale). mma.sync
// takes those in blocks of 64 rows: 16 trees of 16 x 6 over up to 4,096 slots,
// 8 kv heads of 128, take 132 us with pages of 20 slots and 44 with pages of
// 32; heads of 256 370.
int tc_box(const AttendArgs& a) {
  const CacheView& c = a.c;
  if (c.head_dim == 256 || a.group > 128 || a.scale < 0.f) return 0;
  const int box = std::gcd(c.page_size, 128);
  const bool repeats = (c.page_size > 1 && !c.stride_token) || (c.kv_heads > 1 && !c.stride_head) ||
                       (c.pages > 1 && !c.stride_page) || (a.heads > 1 && !a.q_head) || (a.nodes > 1 && !a.q_node) ||
                       (c.batch > 1 && !a.q_seq);
  return box >= 8 && !repeats ? box : 0;
}

template <typename T>
cudaError_t launch_typed(const AttendArgs& a, int device, cudaStream_t s) {
  const bool few = a.nodes * a.group <= kFewRows;
  const int box = few ? 0 : tc_box(a);
  switch (a.c.head_dim) {
    case 64:
      return few ? launch_mma<T, 64, 1>(a, device, s)
                 : box ? launch_tc<T, 64>(a, box, device, s) : launch_mma<T, 64, 4>(a, device, s);
    case 128:
      return few ? launch_mma<T, 128, 1>(a, device, s)
                 : box ? launch_tc<T, 128>(a, box, device, s) : launch_mma<T, 128, 4>(a, device, s);
    default: return few ? launch_mma<T, 256, 1>(a, device, s) : launch_mma<T, 256, 4>(a, device, s);
  }
}

}  // namespace

// A counter for each part (their number and place depend on the device alone;
// a launch with more blocks of rows than places has one run, and nothing to
// join), then two parts for each block of the launch: 16 rows, or 64 (the
// tcgen05 kernel has half the blocks and twice the rows).
AttendWorkspace attend_workspace(int nodes, int heads, int kv_heads, int head_dim, int num_sms) {
  const int64_t rows = static_cast<int64_t>(nodes) * (heads / kv_heads);
  const size_t places = static_cast<size_t>(kBlocksPerSm) * num_sms;
  const size_t blocks = std::max<size_t>(places, (rows + 63) / 64);
  // Blocks of rows of the tcgen05 kernel hold whole nodes, half of 128 rows at least.
  const size_t wide = std::max<size_t>(num_sms, nodes) * 2;
  AttendWorkspace w;
  w.partials_at = (2 * places * sizeof(int) + 255) & ~static_cast<size_t>(255);
  const size_t part_rows = rows <= kFewRows ? places * 16 : std::max(blocks, wide) * 64;
  w.bytes = w.partials_at + 2 * part_rows * (head_dim + 2) * sizeof(float);
  return w;
}

cudaError_t launch_tree_attention(const AttendArgs& a, int dtype, int device, cudaStream_t s) {
  return dtype == TF_F16 ? launch_typed<__half>(a, device, s) : launch_typed<__nv_bfloat16>(a, device, s);
}

}  // namespace tfx
