// Verification of drafted tokens against the target's probabilities
// (tf_verify_draft).
//
// Probabilities are whole numbers: w = round(2^30 exp(z - max z)), and their
// sums are exact in 64 bits, so a token never depends on the order of a sum
// nor on how a row is split.
//
// What a node decides (the child it goes on to, or the token sampled) depends
// on its own rows of logits only. A cluster of blocks takes a node: each block
// a part of the vocabulary, with one exchange through distributed shared
// memory for the maximum, one for the sum and one for each refusal's rest; the
// row is read from memory once and again from the L1 cache or L2. What bounds
// a row is latency: passes and meetings of the cluster one after the other, in
// a block whose 16 warps issue 1.3 of 4 instructions a cycle.
//
// With no more rows than SMs, every row is taken at once by a cluster of its
// own, in the time of one row, and the block that completes a sequence's last
// row follows the decisions from node 0 and writes the outputs. With more, a
// cluster takes a sequence and walks down its tree, so that only the rows on
// the accepted path are read.
//
// 8 chains of 8 rows of 129,280 in bf16 with a draft: 42 us (2 blocks a row).
// 32 trees of 16 rows in fp32: 65 us, 78 MB of 265 read; at temperature 0,
// with its pass for the lowest index, 71 (one row 10.2 and 10.3).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "spec.cuh"

namespace cg = cooperative_groups;

namespace tfx {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCluster = 8;
constexpr float kOne = 1073741824.f;                 // 2^30: the largest weight
constexpr double kUnit = 2305843009213693952.0;      // 2^61
constexpr double kHalfUnit = 2147483648.0;           // 2^31: the normalised rows' unit
constexpr int kNobody = -1, kRefused = -2;           // a child asked, else

__device__ __forceinline__ uint32_t whole(float x) { return __float2uint_rn(x); }   // a NaN becomes 0

template <typename T>
__device__ __forceinline__ T lowest();   // -inf
template <>
__device__ __forceinline__ float lowest<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ __half lowest<__half>() { return __ushort_as_half(0xFC00); }
template <>
__device__ __forceinline__ __nv_bfloat16 lowest<__nv_bfloat16>() { return __ushort_as_bfloat16(0xFF80); }

// A row of logits: z = x / T, and e = exp(z - max z). The row's vectors of 16
// bytes are numbered from the aligned address at or before its first element;
// element k of vector v is number v * kVec + k - shift.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T* x;
  float inv, top;

  __device__ __forceinline__ int shift() const {
    return static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  }
  __device__ __forceinline__ float z(T v) const { return __fmul_rn(to_f32(v), inv); }
  // kFinite: the maximum is (else it is +inf, and its own places alone count).
  template <bool kFinite>
  __device__ __forceinline__ float e(float z) const {
    if (!kFinite) return z == top ? 1.f : 0.f;
    return expf(__fsub_rn(z, top));
  }
  __device__ __forceinline__ float e(float z) const { return top < INFINITY ? e<true>(z) : e<false>(z); }
  __device__ __forceinline__ int vectors(int vocab) const { return (vocab + shift() + kVec - 1) / kVec; }
  // kVec elements from number i on, those outside [0, vocab) as -inf.
  __device__ __forceinline__ void load(int i, int vocab, T (&v)[kVec]) const {
    if (i >= 0 && i + kVec <= vocab && (reinterpret_cast<uintptr_t>(x + i) & 15) == 0) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(x + i);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] = i + k >= 0 && i + k < vocab ? x[i + k] : lowest<T>();
    }
  }
};

// A warp's part [v0, v1) of a row's vectors: f(number of the first element,
// the elements) for each. Whole vectors come kAhead a lane at a time, so that
// their loads are in flight together; the row's first and last may be cut.
template <int kAhead, typename T, typename F>
__device__ __forceinline__ void sweep(const Row<T>& r, int vocab, int v0, int v1, F f) {
  constexpr int kVec = Row<T>::kVec;
  const int lane = threadIdx.x % 32, shift = r.shift();
  const int f0 = max(v0, shift ? 1 : 0), f1 = min(v1, (vocab + shift) / kVec);   // whole ones
  const uint4* base = reinterpret_cast<const uint4*>(r.x - shift);
  int v = f0 + lane;
  alignas(16) T x[kVec];
  for (; v + 32 * (kAhead - 1) < f1; v += 32 * kAhead) {
    uint4 raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) raw[u] = base[v + 32 * u];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      *reinterpret_cast<uint4*>(x) = raw[u];
      f((v + 32 * u) * kVec - shift, x);
    }
  }
  for (; v < f1; v += 32) {
    *reinterpret_cast<uint4*>(x) = base[v];
    f(v * kVec - shift, x);
  }
  if (lane == 0 && v0 < v1) {
    if (v0 < f0) {
      r.load(v0 * kVec - shift, vocab, x);
      f(v0 * kVec - shift, x);
    }
    if (f1 < v1 && v1 - 1 >= f0) {
      r.load((v1 - 1) * kVec - shift, vocab, x);
      f((v1 - 1) * kVec - shift, x);
    }
  }
}

// The largest element so far, NaNs left out. z grows with x, so the largest z
// is that of the largest x, and 16-bit types are compared two at a time.
struct Largest32 {
  float top = -INFINITY;
  __device__ __forceinline__ void add(const float (&x)[4]) {
    top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
  }
  __device__ __forceinline__ float get() const { return top; }
};
template <typename T, typename T2>
struct Largest16 {
  T2 top;
  __device__ Largest16() { top.x = top.y = lowest<T>(); }
  __device__ __forceinline__ void add(const T (&x)[8]) {
    const T2* y = reinterpret_cast<const T2*>(x);
    top = __hmax2(top, __hmax2(__hmax2(y[0], y[1]), __hmax2(y[2], y[3])));
  }
  __device__ __forceinline__ float get() const { return fmaxf(to_f32(top.x), to_f32(top.y)); }
};
template <typename T>
struct Largest;
template <>
struct Largest<float> : Largest32 {};
template <>
struct Largest<__half> : Largest16<__half, __half2> {};
template <>
struct Largest<__nv_bfloat16> : Largest16<__nv_bfloat16, __nv_bfloat162> {};

// e of two elements of a row with a finite maximum; a NaN stays one (whole()
// makes it 0). (The product and the difference are single instructions: the
// assembler joins packed ones into a multiply-add, which rounds once where
// the definition rounds twice.)
template <typename T>
__device__ __forceinline__ float2 exp_of(const Row<T>& r, T x0, T x1) {
  return float2{r.template e<true>(r.z(x0)), r.template e<true>(r.z(x1))};
}

// A warp's sum of the weights of its part of a row.
template <typename T, bool kFinite>
__device__ __forceinline__ unsigned long long sum_weights(const Row<T>& r, int vocab, int lo, int hi) {
  unsigned long long sum = 0;
  sweep<!kFinite ? 1 : sizeof(T) == 2 ? 2 : 4>(r, vocab, lo, hi, [&](int, const T(&x)[Row<T>::kVec]) {
#pragma unroll
    for (int k = 0; k < Row<T>::kVec; k += 2) {
      if (kFinite) {
        const float2 w = mul2(exp_of(r, x[k], x[k + 1]), float2{kOne, kOne});
        sum += whole(w.x) + whole(w.y);   // at most 2^31
      } else {
        sum += whole(r.template e<false>(r.z(x[k])) * kOne) + whole(r.template e<false>(r.z(x[k + 1])) * kOne);
      }
    }
  });
  return sum;
}

// What is left of p over a draft distribution q, in units of 2^-31.
struct Rest {
  float cp, cq;
  __device__ __forceinline__ uint32_t operator()(float ep, float eq) const {
    const uint32_t x = whole(__fmul_rn(ep, cp)), y = whole(__fmul_rn(eq, cq));
    return x > y ? x - y : 0;
  }
};
template <typename T>
__device__ unsigned long long sum_rest(const Row<T>& p, const Row<T>& q, const Rest& rest, int vocab, int lo, int hi) {
  constexpr int kVec = Row<T>::kVec;
  unsigned long long sum = 0;
  const bool finite = p.top < INFINITY && fabsf(q.top) < INFINITY;
  if (finite && p.shift() == q.shift()) {   // whole vectors of both, several in flight; the row's ends below
    constexpr int kAhead = 2;
    const int lane = threadIdx.x % 32, shift = p.shift();
    const int f0 = max(lo, shift ? 1 : 0), f1 = min(hi, (vocab + shift) / kVec);
    const uint4* pv = reinterpret_cast<const uint4*>(p.x - shift);
    const uint4* qv = reinterpret_cast<const uint4*>(q.x - shift);
    auto add = [&](const uint4& a, const uint4& b) {
      alignas(16) T x[kVec];
      alignas(16) T y[kVec];
      *reinterpret_cast<uint4*>(x) = a;
      *reinterpret_cast<uint4*>(y) = b;
#pragma unroll
      for (int k = 0; k < kVec; k += 2) {
        const float2 u = mul2(exp_of(p, x[k], x[k + 1]), float2{rest.cp, rest.cp});
        const float2 w = mul2(exp_of(q, y[k], y[k + 1]), float2{rest.cq, rest.cq});
        const uint32_t u0 = whole(u.x), u1 = whole(u.y), w0 = whole(w.x), w1 = whole(w.y);
        sum += static_cast<unsigned long long>(u0 > w0 ? u0 - w0 : 0) + (u1 > w1 ? u1 - w1 : 0);
      }
    };
    int v = f0 + lane;
    for (; v + 32 * (kAhead - 1) < f1; v += 32 * kAhead) {
      uint4 a[kAhead], b[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) a[u] = pv[v + 32 * u], b[u] = qv[v + 32 * u];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add(a[u], b[u]);
    }
    for (; v < f1; v += 32) add(pv[v], qv[v]);
    if (lane == 0 && lo < hi) {
      alignas(16) T x[kVec];
      alignas(16) T y[kVec];
      auto end = [&](int at) {
        p.load(at * kVec - shift, vocab, x);
        q.load(at * kVec - shift, vocab, y);
        add(*reinterpret_cast<const uint4*>(x), *reinterpret_cast<const uint4*>(y));
      };
      if (lo < f0) end(lo);
      if (f1 < hi && hi - 1 >= f0) end(hi - 1);
    }
    return sum;
  }
  sweep<1>(p, vocab, lo, hi, [&](int e0, const T(&x)[kVec]) {
    alignas(16) T y[kVec];
    q.load(e0, vocab, y);
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum += rest(p.e(p.z(x[k])), q.top > -INFINITY ? q.e(q.z(y[k])) : 0.f);
  });
  return sum;
}

// What the blocks of a cluster tell one another, twice so that an exchange
// can begin while the one before is still being read.
struct Exchange {
  unsigned long long sum[2][kMaxCluster];
  float top[2][kMaxCluster], qtop[2][kMaxCluster];
  int at[2][kMaxCluster];
};

struct Shared {
  Exchange x;
  unsigned long long sums[kWarps + 1];   // weight before each warp of this block, and all of it
  unsigned long long fine[kWarps];
  float tops[kWarps], qtops[kWarps];
  int ats[kWarps];
  int par[TF_MAX_NODES], tok[TF_MAX_NODES];
  float zp[TF_MAX_NODES], zq[TF_MAX_NODES];   // logits of the node's children's tokens
  float u[TF_MAX_NODES];
  int next_node, verdict;
  unsigned long long goal;
  Rest rest;
  int state[TF_MAX_NODES], out_tok[TF_MAX_NODES];
  float out_lp[TF_MAX_NODES];
};

// Decisions in the workspace, one for each row: the child gone on to + 2 (1:
// none, -1: the row's node is absent), the token and its log-probability; and
// the rows arrived of each sequence. A call leaves all zero.
struct Results {
  int* state;
  int* token;
  float* logprob;
  int* arrived;
};

__device__ __forceinline__ unsigned long long threshold(float u, unsigned long long total) {
  const double x = floor(static_cast<double>(u) * static_cast<double>(total));
  if (!(x > 0.0)) return 0;
  const unsigned long long t = x >= 18446744073709551615.0 ? ~0ull : static_cast<unsigned long long>(x);
  return t < total ? t : total - 1;
}

// One warp: counts a finished row of sequence b, and where it is the last
// one, follows the decisions and writes the sequence's outputs.
__device__ void arrive(const VerifyArgs& a, const Results& r, Shared& s, int b) {
  const int lane = threadIdx.x % 32;
  int last = 0;
  if (lane == 0) {
    __threadfence();
    last = atomicAdd(r.arrived + b, 1) + 1 == a.nodes;
    __threadfence();
  }
  if (!__shfl_sync(~0u, last, 0)) return;
  const int64_t row0 = static_cast<int64_t>(b) * a.nodes;
  for (int j = lane; j < a.nodes; j += 32) {
    s.state[j] = __ldcg(r.state + row0 + j);
    s.out_tok[j] = __ldcg(r.token + row0 + j);
    s.out_lp[j] = __ldcg(r.logprob + row0 + j);
    r.state[row0 + j] = 0;
    r.token[row0 + j] = 0;
    r.logprob[row0 + j] = 0.f;
  }
  if (lane == 0) r.arrived[b] = 0;
  __syncwarp();
  int count = 0;
  for (int node = s.state[0] > 0 ? 0 : -1; node >= 0; node = s.state[node] - 2) {
    if (lane == 0) {
      a.path[row0 + count] = node;
      a.out_tokens[row0 + count] = s.out_tok[node];
      a.logprobs[row0 + count] = s.out_lp[node];
    }
    ++count;
  }
  if (lane == 0) a.counts[b] = count;
  for (int k = count + lane; k < a.nodes; k += 32) {
    a.path[row0 + k] = -1;
    a.out_tokens[row0 + k] = -1;
    a.logprobs[row0 + k] = 0.f;
  }
}

template <typename T, bool kWalk>
__global__ void __launch_bounds__(kThreads, 1) verify_draft_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Shared s;
  // A block's shared memory may be written by the others only once it runs:
  // every block says so here, and hears it of all below, while the kernel
  // before this one still ends.
  cluster_arrive();
  chain();
  cluster_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank(), id = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int b = kWalk ? id : id / a.nodes;
  const int64_t row0 = static_cast<int64_t>(b) * a.nodes;
  int side = 0;   // which half of the exchange is next
  constexpr int kVec = Row<T>::kVec;

  // Sum of x over the cluster, and the maximum of qt; s.sums holds what lies
  // before each warp of this block, *before what lies before this block.
  auto total = [&](unsigned long long x, float qt, unsigned long long* before, float* qt_all) {
    for (int o = 16; o; o >>= 1) {
      x += __shfl_xor_sync(~0u, x, o);
      qt = fmaxf(qt, __shfl_xor_sync(~0u, qt, o));
    }
    __syncthreads();   // the sums before are no longer read
    if (lane == 0) s.sums[warp + 1] = x, s.qtops[warp] = qt;
    if (tid == 0) s.sums[0] = 0;
    __syncthreads();
    if (warp == 0) {
      unsigned long long y = lane < kWarps ? s.sums[lane + 1] : 0;
      qt = lane < kWarps ? s.qtops[lane] : -INFINITY;
      for (int o = 1; o < kWarps; o *= 2) {
        const unsigned long long z = __shfl_up_sync(~0u, y, o);
        if (lane >= o) y += z;
        qt = fmaxf(qt, __shfl_xor_sync(~0u, qt, o));
      }
      if (lane < kWarps) s.sums[lane + 1] = y;
      const unsigned long long all = __shfl_sync(~0u, y, kWarps - 1);
      qt = __shfl_sync(~0u, qt, 0);
      if (lane < ranks) {
        Exchange* to = cluster.map_shared_rank(&s.x, lane);
        to->sum[side][rank] = all;
        to->qtop[side][rank] = qt;
      }
    }
    cluster.sync();
    unsigned long long sum = 0;
    *before = 0;
    *qt_all = -INFINITY;
    for (int k = 0; k < ranks; ++k) {
      if (k == rank) *before = sum;
      sum += s.x.sum[side][k];
      *qt_all = fmaxf(*qt_all, s.x.qtop[side][k]);
    }
    side ^= 1;
    return sum;
  };

  auto part_of = [&](int vecs, int* lo, int* hi, int w) {
    const int per_block = (vecs + ranks - 1) / ranks, b0 = min(vecs, rank * per_block), b1 = min(vecs, b0 + per_block);
    const int per_warp = (b1 - b0 + kWarps - 1) / kWarps;
    *lo = min(b1, b0 + w * per_warp);
    *hi = min(b1, *lo + per_warp);
  };

  const bool draft = a.draft != nullptr;
  int count = 0;   // nodes gone through (a walk)
  // This block's part of a row, to L2.
  auto prefetch_part = [&](const T* row) {
    const Row<T> r{row, 0.f, 0.f};
    const int vecs = (a.vocab + r.shift()) / kVec, per_block = (r.vectors(a.vocab) + ranks - 1) / ranks;
    const int v0 = max(r.shift() ? 1 : 0, rank * per_block), v1 = min(vecs, (rank + 1) * per_block);
    if (v0 < v1)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row - r.shift() + v0 * kVec), "r"((v1 - v0) * 16)
                   : "memory");
  };
#pragma unroll 1
  for (int node = kWalk ? 0 : id - b * a.nodes; node >= 0;) {
    Row<T> p{static_cast<const T*>(a.logits) + b * a.seq + node * a.node, a.inv_temp, 0.f};
    Row<T> q{draft ? static_cast<const T*>(a.draft) + b * a.draft_seq + node * a.draft_node : p.x, a.inv_temp, 0.f};
    const float u_node = a.greedy ? 0.f : a.u_sample[row0 + node];
    // Of the tree's node tid; on their way during the first pass.
    int parent = -2, drafted = -1;
    float u_child = 0.f;
    if (tid < a.nodes) {
      parent = a.parents[b * a.stride_parents + tid];
      drafted = a.tokens[row0 + tid];
      // in [0, 1], a NaN as 0: a child of no weight in p must not be accepted
      if (draft) u_child = fminf(fmaxf(a.u_accept[row0 + tid], 0.f), 1.f);
    }

    // This warp's vectors of each row.
    int v0, v1, q0, q1v;
    part_of(p.vectors(a.vocab), &v0, &v1, warp);
    part_of(q.vectors(a.vocab), &q0, &q1v, warp);

    // The maximum. (The draft's row comes after p's sum, so that p's second
    // pass finds it in L1; it is on its way to L2 meanwhile.)
    if (draft && tid == 0) prefetch_part(q.x);
    Largest<T> most;
    sweep<8>(p, a.vocab, v0, v1, [&](int, const T(&x)[kVec]) { most.add(x); });
    bool child = false;
    float z_child = 0.f, zq_child = 0.f;
    if (tid < a.nodes) {
      if (parent >= tid) {
        // each row's own, or in a walk, which never comes to such a node, all at its start
        if (kWalk ? node == 0 : tid == node) record_index_error(a.err);
        parent = -2;
      }
      child = parent == node && tid > node && drafted >= 0 && drafted < a.vocab;
      s.par[tid] = tid == node ? parent : (child ? node : -2);   // children that may be asked, and the row's own
      s.tok[tid] = drafted;
      s.u[tid] = u_child;
      if (child && draft) z_child = p.z(p.x[drafted]), zq_child = q.z(q.x[drafted]);
    }
    const bool ask = __syncthreads_or(child) && draft;   // a leaf has no use for the draft's row
    float top = __fmul_rn(most.get(), a.inv_temp);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) s.tops[warp] = top;
    __syncthreads();
    if (warp == 0) {
      top = lane < kWarps ? s.tops[lane] : -INFINITY;
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      if (lane < ranks) cluster.map_shared_rank(&s.x.top[side][0], lane)[rank] = top;
    }
    cluster.sync();
    for (int k = 0; k < ranks; ++k) p.top = k ? fmaxf(p.top, s.x.top[side][k]) : s.x.top[side][k];
    side ^= 1;

    // A walk goes on to one of the children, if to any: the first two's rows
    // start on their way to L2 while this one is summed.
    if (kWalk && warp == 0) {
      const unsigned kids = __ballot_sync(~0u, child);
      if (child && __popc(kids & ((1u << lane) - 1)) < 2)
        prefetch_part(static_cast<const T*>(a.logits) + b * a.seq + tid * a.node);
    }
    const int up = s.par[node];
    const bool dead = node == 0 ? up < -1 : up < 0;
    int next = -1, token = -1;
    unsigned long long mass = 0, before = 0;
    bool pick = false;   // the token is still to be found by its cumulative weight
    Rest rest{0.f, 0.f};
    bool refused = false;   // by a child: the token comes from the rest of p
    unsigned long long goal = 0, goal_total = 0;
    if (!dead && p.top > -INFINITY) {
      const unsigned long long sum = p.top < INFINITY ? sum_weights<T, true>(p, a.vocab, v0, v1)
                                                      : sum_weights<T, false>(p, a.vocab, v0, v1);
      float qtop = -INFINITY, unused_top;
      if (ask) {
        Largest<T> qmost;
        sweep<8>(q, a.vocab, q0, q1v, [&](int, const T(&x)[kVec]) { qmost.add(x); });
        qtop = __fmul_rn(qmost.get(), a.inv_temp);
      }
      if (a.greedy) {
        int best = INT32_MAX;
        sweep<2>(p, a.vocab, v0, v1, [&](int e0, const T(&x)[kVec]) {
#pragma unroll
          for (int k = kVec - 1; k >= 0; --k)
            if (p.z(x[k]) == p.top) best = min(best, e0 + k);
        });
        best = __reduce_min_sync(~0u, best);
        if (lane == 0) s.ats[warp] = best;
        __syncthreads();
        if (warp == 0) {
          best = __reduce_min_sync(~0u, lane < kWarps ? s.ats[lane] : INT32_MAX);
          if (lane < ranks) cluster.map_shared_rank(&s.x.at[side][0], lane)[rank] = best;
        }
        const int half = side;
        mass = total(sum, qtop, &before, &q.top);
        token = INT32_MAX;
        for (int k = 0; k < ranks; ++k) token = min(token, s.x.at[half][k]);
      } else {
        mass = total(sum, qtop, &before, &q.top);
        pick = true;
        goal_total = mass;
      }
      if (ask) {
        if (child) s.zp[tid] = z_child, s.zq[tid] = zq_child;
        unsigned long long unused;
        const unsigned long long q_sum = q.top == -INFINITY ? 0
                                         : q.top < INFINITY ? sum_weights<T, true>(q, a.vocab, q0, q1v)
                                                            : sum_weights<T, false>(q, a.vocab, q0, q1v);
        // p's sums, for a node whose token comes from p itself.
        const unsigned long long p_warp = s.sums[warp], p_end = s.sums[warp + 1], p_before = before;
        const unsigned long long qmass = total(q_sum, -INFINITY, &unused, &unused_top);
        // The 64-bit decisions are one thread's, in every block of the cluster
        // alike: an SM has few fp64 units, and sixteen warps dividing at once
        // took longer than a pass over the row.
        double q1 = 0.0, level = 0.0, left = kHalfUnit;   // of thread 0
        if (tid == 0) {
          s.rest.cp = static_cast<float>(kUnit / static_cast<double>(mass));
          q1 = qmass ? kUnit / static_cast<double>(qmass) : 0.0;
        }
        for (int c = node;;) {
          if (tid == 0) {   // the next child is asked
            s.verdict = kNobody;
            while (++c < a.nodes && s.par[c] != node) {
            }
            if (c < a.nodes) {
              const float ep = isnan(s.zp[c]) ? 0.f : p.e(s.zp[c]);
              const float eq = isnan(s.zq[c]) || q.top == -INFINITY ? 0.f : q.e(s.zq[c]);
              const float qt = __fmul_rn(eq, static_cast<float>(q1));
              const double rt =
                  refused ? static_cast<double>(s.rest(ep, eq)) : static_cast<double>(__fmul_rn(ep, s.rest.cp));
              if (static_cast<double>(s.u[c]) * static_cast<double>(qt) * left < rt * kHalfUnit) {
                s.verdict = c;
              } else {
                level += left / kHalfUnit;
                s.rest.cq = static_cast<float>(level * q1);
                s.verdict = kRefused;
              }
            }
          }
          __syncthreads();
          rest = s.rest;
          next = s.verdict;
          if (next != kRefused) break;
          unsigned long long rest_before;
          goal_total = total(sum_rest(p, q, rest, a.vocab, v0, v1), -INFINITY, &rest_before, &unused_top);
          refused = goal_total > 0;
          if (!refused) {   // nothing is left: the token comes from p after all
            goal_total = mass;
            next = kNobody;
            break;
          }
          before = rest_before;
          if (tid == 0) left = static_cast<double>(goal_total);
        }
        if (next >= 0) {
          token = s.tok[next];
          pick = false;
        } else if (!refused) {   // p itself: its sums again
          __syncthreads();
          s.sums[warp] = p_warp;
          if (warp == kWarps - 1) s.sums[kWarps] = p_end;
          before = p_before;
        }
      }
      if (pick) {
        if (tid == 0) s.goal = threshold(u_node, goal_total);
        __syncthreads();
        goal = s.goal;
      }
    }

    // The block that holds the token finds it: the part of one warp is shared
    // out among all its warps, then the part of one of those is looked through.
    bool mine = rank == 0 && warp == 0;   // the warp that writes the decision
    float z_token = 0.f;
    if (pick) {
      mine = false;
      const bool here = goal >= before && goal < before + s.sums[kWarps];
      if (here) {
        const int w = __ffs(__ballot_sync(~0u, lane < kWarps && goal < before + s.sums[min(lane, kWarps - 1) + 1])) - 1;
        unsigned long long run = before + s.sums[w];
        int lo, hi;
        part_of(p.vectors(a.vocab), &lo, &hi, w);
        const int per = (hi - lo + kWarps - 1) / kWarps;
        lo = min(hi, lo + warp * per);
        hi = min(hi, lo + per);
        uint32_t weights[kVec];
        alignas(16) T x[kVec];
        alignas(16) T y[kVec];
        auto weigh = [&](int v) {   // weights of vector v, and their sum
          unsigned long long sum = 0;
          const int e0 = v * kVec - p.shift();
          p.load(e0, a.vocab, x);
          if (refused) q.load(e0, a.vocab, y);
#pragma unroll
          for (int k = 0; k < kVec; ++k) {
            const float ep = p.e(p.z(x[k]));
            weights[k] = refused ? rest(ep, q.top > -INFINITY ? q.e(q.z(y[k])) : 0.f) : whole(ep * kOne);
            sum += weights[k];
          }
          return sum;
        };
        unsigned long long sum = 0;
        for (int v = lo + lane; v < hi; v += 32) sum += weigh(v);
        const bool once = hi - lo <= 32;   // then this lane's weights are still there
        const unsigned long long first = sum;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) s.fine[warp] = sum;
        __syncthreads();
        for (int k = 0; k < warp; ++k) run += s.fine[k];
        mine = goal >= run && goal < run + s.fine[warp];
        if (mine) {
          for (int v = lo; v < hi; v += 32) {
            const unsigned long long own = once ? first : v + lane < hi ? weigh(v + lane) : 0;
            unsigned long long upto = own;
            for (int o = 1; o < 32; o *= 2) {
              const unsigned long long z = __shfl_up_sync(~0u, upto, o);
              if (lane >= o) upto += z;
            }
            const unsigned hit = __ballot_sync(~0u, run + upto > goal);
            if (hit) {
              const int who = __ffs(hit) - 1;
              if (lane == who) {
                unsigned long long at = run + upto - own;
                bool open = true;
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                  at += weights[k];
                  if (open && at > goal) token = (v + lane) * kVec - p.shift() + k, z_token = p.z(x[k]), open = false;
                }
              }
              token = __shfl_sync(~0u, token, who);
              z_token = __shfl_sync(~0u, z_token, who);
              break;
            }
            run += __shfl_sync(~0u, upto, 31);
          }
        }
      }
    } else if (mine && token >= 0) {
      z_token = p.z(p.x[token]);
    }
    if (mine) {
      if (!draft && token >= 0)   // the first child with that token
        for (int c0 = 0; c0 < a.nodes && next < 0; c0 += 32) {
          const int c = c0 + lane;
          const unsigned hit = __ballot_sync(~0u, c > node && c < a.nodes && s.par[c] == node && s.tok[c] == token);
          if (hit) next = c0 + __ffs(hit) - 1;
        }
      if (lane == 0) {
        const float logprob = token < 0 ? 0.f
                                        : __fsub_rn(z_token, p.top) -
                                              logf(static_cast<float>(mass) * 9.31322574615478515625e-10f);
        if (kWalk) {
          if (!dead) {
            a.path[row0 + count] = node;
            a.out_tokens[row0 + count] = token;
            a.logprobs[row0 + count] = logprob;
          }
        } else {
          const size_t rows = static_cast<size_t>(a.batch) * a.nodes;
          __stcg(a.work + row0 + node, dead ? -1 : next + 2);
          __stcg(a.work + rows + row0 + node, token);
          __stcg(reinterpret_cast<float*>(a.work + 2 * rows) + row0 + node, logprob);
        }
      }
      if (!kWalk) {
        const size_t rows = static_cast<size_t>(a.batch) * a.nodes;
        const Results res{a.work, a.work + rows, reinterpret_cast<float*>(a.work + 2 * rows), a.work + 3 * rows};
        arrive(a, res, s, b);
      } else if (lane < ranks) {
        cluster.map_shared_rank(&s.next_node, lane)[0] = next;
      }
    }
    if (!kWalk) break;
    if (!dead) ++count;
    cluster.sync();   // the next node is known; the row's lists may be written again
    node = s.next_node;
  }
  if (kWalk && rank == 0) {
    if (tid == 0) a.counts[b] = count;
    for (int k = count + tid; k < a.nodes; k += kThreads) {
      a.path[row0 + k] = -1;
      a.out_tokens[row0 + k] = -1;
      a.logprobs[row0 + k] = 0.f;
    }
  }
  cluster.sync();     // no block leaves while another may still write to its shared memory
}

// More rows than SMs are walked through. us, all rows together and walked
// (vocabulary 129,280): fp32 without a draft 8 x 8 rows 21 and 30, 32 x 4 34
// and 44, 32 x 16 117 and 69; bf16 with a draft, chains 8 x 8 43 and 91, 16 x 8
// 72 and 98, 8 x 16 73 and 181, trees 8 x 8 50 and 61, 16 x 8 128 and 66, 32 x
// 16 179 and 104. So at 512 rows the walk wins, and at 128 it depends: chains
// and rows without a draft are faster together, by up to 2.5 times, and trees
// with a draft walked, by up to 2. (Those ask more children a node and end
// sooner; which it is only the device knows, and the rule does without.)
bool walks(int batch, int nodes, int num_sms) { return static_cast<int64_t>(batch) * nodes > num_sms; }

template <typename T>
cudaError_t launch_typed(const VerifyArgs& a, cudaStream_t s) {
  // One block an SM: as many blocks for a cluster as leave every cluster its
  // place. One row of fp32: 11 us with 8 blocks, 13 with 4, 17 with 2.
  const int64_t rows = static_cast<int64_t>(a.batch) * a.nodes;
  const bool walk = walks(a.batch, a.nodes, a.num_sms);
  const int64_t clusters = walk ? a.batch : rows;
  int ranks = kMaxCluster;
  while (ranks > 1 && clusters * ranks > a.num_sms) ranks /= 2;
  const dim3 grid(static_cast<unsigned>(clusters * ranks));
  return walk ? launch_chained(verify_draft_kernel<T, true>, grid, dim3(kThreads), 0, ranks, s, a)
              : launch_chained(verify_draft_kernel<T, false>, grid, dim3(kThreads), 0, ranks, s, a);
}

}  // namespace

// Only calls that do not walk use it, with at most num_sms rows, and so at most
// as many sequences. What any of them within these sizes needs, so that a
// workspace made for the largest batch, which may walk, serves the smaller ones.
size_t verify_workspace_bytes(int batch, int nodes, int num_sms) {
  const int64_t rows = std::min<int64_t>(static_cast<int64_t>(batch) * nodes, num_sms);
  return static_cast<size_t>(3 * rows + std::min(batch, num_sms) + 1) * sizeof(int);
}

cudaError_t launch_verify_draft(const VerifyArgs& a, int dtype, cudaStream_t s) {
  if (dtype == TF_F32) return launch_typed<float>(a, s);
  return dtype == TF_F16 ? launch_typed<__half>(a, s) : launch_typed<__nv_bfloat16>(a, s);
}

}  // namespace tfx
