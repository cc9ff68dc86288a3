// Internal types and launchers of the operators declared in tf_qcache.h.
#pragma once

#include "spec.h"
#include "tf_qcache.h"

namespace tfx {

// A quantised cache as its kernels see it: the strides of c are those of the
// codes, in bytes; a pair of factors is one 32-bit word (strides in words).
struct QView {
  CacheView c;
  int64_t scale_layer, scale_page, scale_token, scale_head;
  uint8_t* k;
  uint8_t* v;
  uint32_t* scales;
  int bits;
};

// Rows [batch][nodes][kv_heads][head_dim] to be written.
struct RowsIn {
  const void* at;
  int64_t seq, node, head;
};

struct NormRopeArgs {
  tf_head_rows q, k;       // k.heads is 0 where there are no keys
  const int32_t* positions;
  int64_t stride_positions;
  const double* inv_freq;
  int rotary, flags;
  float eps;
  int batch, nodes;
  int num_sms;
};

// a.c, a.k and a.v as in QView; a.num_sms, partials and counters as there.
struct QAttendArgs {
  AttendArgs a;
  int64_t scale_page, scale_token, scale_head;
  const uint32_t* scales;
  int box;   // slots of a page that lie together and are copied at once, 0 where none do
};

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int dtype, int weight_dtype, int head_dim, cudaStream_t s);
cudaError_t launch_kvq_write(const QView& c, const RowsIn& k_new, const RowsIn& v_new, int dtype,
                             const int32_t* counts, int nodes, cudaStream_t s);
cudaError_t launch_kvq_read(const QView& c, const int32_t* starts, void* k_out, void* v_out, int dtype, int64_t seq,
                            int64_t slot, int64_t head, int slots, cudaStream_t s);
cudaError_t launch_kvq_keep(const QView& c, const int32_t* path, const int32_t* counts, int nodes,
                            int32_t* new_lengths, cudaStream_t s);
cudaError_t launch_kvq_attention(const QAttendArgs& a, int dtype, int bits, int device, cudaStream_t s);
AttendWorkspace kvq_attend_workspace(int nodes, int heads, int kv_heads, int head_dim, int num_sms);

}  // namespace tfx
