// Launch of the attention of a drafted token tree over a paged cache
// (tf_tree_attention).
#include "attend_mma.cuh"

namespace tfx {
namespace {

constexpr int kMaxDevices = 64;

// Rows a kv head up to which the 16-row kernel takes them in one block.
constexpr int kFewRows = 16;

template <typename T, int D, int kRowWarps>
cudaError_t launch_mma(const AttendArgs& a, int device, cudaStream_t s) {
  using S = MmaShape<D, kRowWarps>;
  static PerDeviceOnce<kMaxDevices> once;
  const int e = once.run(device, cudaErrorInvalidDevice, [] {
    return static_cast<int>(cudaFuncSetAttribute(tree_attention_mma_kernel<T, D, kRowWarps>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
  });
  if (e != cudaSuccess) return static_cast<cudaError_t>(e);
  tree_attention_mma_kernel<T, D, kRowWarps><<<kBlocksPerSm * a.num_sms, S::kThreads, S::kSmem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const AttendArgs& a, int device, cudaStream_t s) {
  const bool few = a.nodes * a.group <= kFewRows;
  switch (a.c.head_dim) {
    case 64: return few ? launch_mma<T, 64, 1>(a, device, s) : launch_mma<T, 64, 4>(a, device, s);
    case 128: return few ? launch_mma<T, 128, 1>(a, device, s) : launch_mma<T, 128, 4>(a, device, s);
    default: return few ? launch_mma<T, 256, 1>(a, device, s) : launch_mma<T, 256, 4>(a, device, s);
  }
}

}  // namespace

// A counter for each part (their number and place depend on the device
// alone), then two parts for each block of the launch: 16 rows, or 64 (the
// tcgen05 kernel has half the blocks and twice the rows).
AttendWorkspace attend_workspace(int nodes, int heads, int kv_heads, int head_dim, int num_sms) {
  const int64_t rows = static_cast<int64_t>(nodes) * (heads / kv_heads);
  const size_t parts = static_cast<size_t>(kBlocksPerSm) * num_sms * 2;
  AttendWorkspace w;
  w.partials_at = (parts * sizeof(int) + 255) & ~static_cast<size_t>(255);
  w.bytes = w.partials_at + parts * (rows <= kFewRows ? 16 : 64) * (head_dim + 2) * sizeof(float);
  return w;
}

cudaError_t launch_tree_attention(const AttendArgs& a, int dtype, int device, cudaStream_t s) {
  return dtype == TF_F16 ? launch_typed<__half>(a, device, s) : launch_typed<__nv_bfloat16>(a, device, s);
}

}  // namespace tfx
