// Verification of drafted tokens against the target's probabilities
// (tf_verify_draft).
//
// Probabilities are whole numbers: w = round(2^30 exp(z - max z)), and their
// sums are exact in 64 bits, so a token never depends on the order of a sum.
// One block takes one sequence and walks down its tree, reading the rows of
// the nodes it reaches.
#include "spec.cuh"

namespace tfx {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

__device__ __forceinline__ float clean(float x) { return isnan(x) ? -INFINITY : x; }

// One row of logits: z = x / T and the weights against the row's maximum.
template <typename T>
struct Row {
  const T* x;
  float inv, top;
  __device__ __forceinline__ float z(int i) const { return __fmul_rn(clean(to_f32(x[i])), inv); }
  __device__ __forceinline__ float e(float z) const {
    if (z == top) return z > -INFINITY ? 1.f : 0.f;
    return expf(__fsub_rn(z, top));
  }
};

__device__ __forceinline__ uint32_t whole(float x) { return __float2uint_rn(x); }

struct Shared {
  unsigned long long sums[kWarps + 1];
  float tops[kWarps];
  int at[kWarps];
  int token;
};

__device__ float block_max(Shared& s, float x, int i, int* where) {
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(~0u, x, o);
    const int j = __shfl_xor_sync(~0u, i, o);
    if (y > x || (y == x && j < i)) x = y, i = j;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) s.tops[threadIdx.x / 32] = x, s.at[threadIdx.x / 32] = i;
  __syncthreads();
  x = s.tops[0], i = s.at[0];
  for (int w = 1; w < kWarps; ++w)
    if (s.tops[w] > x || (s.tops[w] == x && s.at[w] < i)) x = s.tops[w], i = s.at[w];
  *where = i;
  return x;
}

// Sum over the block of each warp's sum; s.sums[w] keeps what lies before
// warp w and s.sums[kWarps] the total.
__device__ unsigned long long block_sum(Shared& s, unsigned long long x) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) s.sums[threadIdx.x / 32 + 1] = x;
  if (threadIdx.x == 0) s.sums[0] = 0;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w <= kWarps; ++w) s.sums[w] += s.sums[w - 1];
  __syncthreads();
  return s.sums[kWarps];
}

// The least i with weight(0) + .. + weight(i) > t, for a t below the total;
// the warps' parts are contiguous and s.sums is block_sum's.
template <typename F>
__device__ int block_pick(Shared& s, unsigned long long t, int lo, int hi, F weight) {
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (t >= s.sums[w] && t < s.sums[w + 1]) {
    unsigned long long before = s.sums[w];
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const unsigned long long x = i0 + lane < hi ? weight(i0 + lane) : 0;
      unsigned long long run = x;
      for (int o = 1; o < 32; o *= 2) {
        const unsigned long long y = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += y;
      }
      const unsigned hit = __ballot_sync(~0u, before + run > t);
      if (hit) {
        if (lane == 0) s.token = i0 + __ffs(hit) - 1;
        break;
      }
      before += __shfl_sync(~0u, run, 31);
    }
  }
  __syncthreads();
  return s.token;
}

__device__ __forceinline__ unsigned long long threshold(float u, unsigned long long total) {
  const double x = floor(static_cast<double>(u) * static_cast<double>(total));
  if (!(x > 0.0)) return 0;
  const unsigned long long t = x >= 18446744073709551615.0 ? ~0ull : static_cast<unsigned long long>(x);
  return t < total ? t : total - 1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_draft_kernel(VerifyArgs a) {
  __shared__ Shared s;
  __shared__ int par[TF_MAX_NODES], tok[TF_MAX_NODES];
  const int b = blockIdx.x, tid = threadIdx.x;
  for (int j = tid; j < a.nodes; j += kThreads) {
    int p = a.parents[b * a.stride_parents + j];
    if (p >= j) {
      record_index_error(a.err);
      p = -2;
    }
    par[j] = p;
    tok[j] = a.tokens[b * a.nodes + j];
  }
  const int part = (a.vocab + kWarps - 1) / kWarps;
  const int lo = min(a.vocab, tid / 32 * part), hi = min(a.vocab, lo + part), lane = tid % 32;
  __syncthreads();
  int count = 0, node = par[0] >= -1 ? 0 : -1;
  const int64_t row0 = static_cast<int64_t>(b) * a.nodes;
  while (node >= 0) {
    Row<T> p{static_cast<const T*>(a.logits) + b * a.seq + node * a.node, a.inv_temp, 0.f};
    Row<T> q{static_cast<const T*>(a.draft) + b * a.draft_seq + node * a.draft_node, a.inv_temp, 0.f};
    const bool draft = a.draft != nullptr && !a.greedy;
    float top = -INFINITY;
    int best = a.vocab;
    for (int i = lo + lane; i < hi; i += 32) {
      const float z = p.z(i);
      if (z > top) top = z, best = i;
    }
    p.top = block_max(s, top, best, &best);
    unsigned long long sum = 0;
    for (int i = lo + lane; i < hi; i += 32) sum += whole(p.e(p.z(i)) * 1073741824.f);
    const unsigned long long mass = block_sum(s, sum);
    int next = -1, token = -1;
    if (mass > 0 && draft) {
      float qtop = -INFINITY;
      int unused = 0;
      for (int i = lo + lane; i < hi; i += 32) qtop = fmaxf(qtop, q.z(i));
      q.top = block_max(s, qtop, 0, &unused);
      sum = 0;
      for (int i = lo + lane; i < hi; i += 32) sum += whole(q.e(q.z(i)) * 1073741824.f);
      const unsigned long long qmass = block_sum(s, sum);
      const float cp = static_cast<float>(2305843009213693952.0 / static_cast<double>(mass));
      const double q1 = qmass ? 2305843009213693952.0 / static_cast<double>(qmass) : 0.0;
      double level = 0.0, left = 2147483648.0;
      float cq = 0.f;
      auto rest = [&](int i) -> unsigned long long {
        const uint32_t x = whole(__fmul_rn(p.e(p.z(i)), cp)), y = whole(__fmul_rn(q.e(q.z(i)), cq));
        return x > y ? x - y : 0;
      };
      for (int c = node + 1; c < a.nodes && next < 0; ++c) {
        const int t = tok[c];
        if (par[c] != node || t < 0 || t >= a.vocab) continue;
        const float qt = __fmul_rn(q.e(q.z(t)), static_cast<float>(q1));
        const double rt = level > 0.0 ? static_cast<double>(rest(t)) : static_cast<double>(__fmul_rn(p.e(p.z(t)), cp));
        if (static_cast<double>(a.u_accept[row0 + c]) * static_cast<double>(qt) * left < rt * 2147483648.0) {
          next = c;
          break;
        }
        level += left / 2147483648.0;
        cq = static_cast<float>(level * q1);
        sum = 0;
        for (int i = lo + lane; i < hi; i += 32) sum += rest(i);
        const unsigned long long all = block_sum(s, sum);
        left = static_cast<double>(all);
        if (all == 0) {
          level = 0.0;
          break;
        }
      }
      if (next >= 0) {
        token = tok[next];
      } else if (level > 0.0) {
        token = block_pick(s, threshold(a.u_sample[row0 + node], s.sums[kWarps]), lo, hi, rest);
      } else {
        sum = 0;
        for (int i = lo + lane; i < hi; i += 32) sum += whole(p.e(p.z(i)) * 1073741824.f);
        block_sum(s, sum);
        token = block_pick(s, threshold(a.u_sample[row0 + node], mass), lo, hi,
                           [&](int i) -> unsigned long long { return whole(p.e(p.z(i)) * 1073741824.f); });
      }
    } else if (mass > 0) {
      token = a.greedy ? best
                       : block_pick(s, threshold(a.u_sample[row0 + node], mass), lo, hi,
                                    [&](int i) -> unsigned long long { return whole(p.e(p.z(i)) * 1073741824.f); });
      for (int c = a.nodes - 1; c > node; --c)
        if (par[c] == node && tok[c] == token) next = c;
    }
    if (tid == 0) {
      a.path[row0 + count] = node;
      a.out_tokens[row0 + count] = token;
      a.logprobs[row0 + count] =
          token < 0 ? 0.f
                    : __fsub_rn(p.z(token), p.top) - logf(static_cast<float>(mass) * 9.31322574615478515625e-10f);
    }
    ++count;
    node = next;
    __syncthreads();
  }
  if (tid == 0) a.counts[b] = count;
  for (int k = count + tid; k < a.nodes; k += kThreads) {
    a.path[row0 + k] = -1;
    a.out_tokens[row0 + k] = -1;
    a.logprobs[row0 + k] = 0.f;
  }
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, int dtype, cudaStream_t s) {
  if (dtype == TF_F32) verify_draft_kernel<float><<<a.batch, kThreads, 0, s>>>(a);
  if (dtype == TF_F16) verify_draft_kernel<__half><<<a.batch, kThreads, 0, s>>>(a);
  if (dtype == TF_BF16) verify_draft_kernel<__nv_bfloat16><<<a.batch, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace tfx
