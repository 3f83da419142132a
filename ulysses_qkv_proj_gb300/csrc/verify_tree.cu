// verify_tree.cu -- verification of drafted trees against the target's probabilities, and
// the masks and depths of a tree.
//
// The walk itself is a few comparisons a node; what costs is a rejection, whose sum
// over the vocabulary is R = sum max(p - a q, 0), and the last one's running sum, from which the next token is
// drawn.  A cluster of up to eight CTAs takes one request: every warp of it owns one run of the vocabulary,
// in order, so the sums of a pass are also the prefix that locates the drawn token, and only
// the run that holds it is read again (from L2).  All p(x), q(x) of the drafted tokens are fetched before
// the walk, so a level without a rejection reads nothing.
//
// Numbers.  The integers must not depend on the order of a sum, so sums are exact where it matters: an element
// p - a q is formed as an unevaluated pair of floats (2^-48 relative; a is split the same way), a lane
// adds pairs with the error kept, and lanes, warps and CTAs add 64-bit integers of 2^-56.
// fp64 would serve too, but this chip issues two of its operations a cycle and SM, 64 times fewer.
//
// Bound: latency for few requests, HBM / L2 for many (8 bytes a vocabulary entry and rejection).
#include "../../include/qnre.h"
#include "api_util.cuh"
#include "ptx.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

namespace {

using namespace qnre;
using namespace qnre::api;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 8;
constexpr double kFixed = 72057594037927936.0;  // 2^56
constexpr float kFixedF = 72057594037927936.0f;

struct VerifyArgs {
  const float* p;
  const float* q;
  long long ps0, ps1, qs0, qs1;
  const int32_t *tokens, *parents, *node_counts;
  const float *accept_u, *sample_u;
  int32_t *path, *counts, *next;
  long long vocab;
  int nodes, seg;  // seg: vocabulary entries a warp owns
};

// max(p - a q, 0) as an unevaluated sum hi + lo, a = ah + al.
__device__ __forceinline__ void residual(float p, float q, float ah, float al, float& hi, float& lo) {
  const float ph = __fmul_rn(ah, q);
  const float pl = __fmaf_rn(al, q, __fmaf_rn(ah, q, -ph));
  const float s = __fsub_rn(p, ph);
  const float t = __fsub_rn(s, p);
  float e = __fadd_rn(__fsub_rn(p, __fsub_rn(s, t)), __fsub_rn(-ph, t));  // s + e = p - ph exactly
  e = __fsub_rn(e, pl);
  hi = __fadd_rn(s, e);
  lo = __fsub_rn(e, __fsub_rn(hi, s));
  if (!(hi > 0.f)) hi = lo = 0.f;
}

__device__ __forceinline__ long long to_fixed(float hi, float lo) {
  return __float2ll_rn(__fmul_rn(hi, kFixedF)) + __float2ll_rn(__fmul_rn(lo, kFixedF));
}

struct Shared {
  long long warp_sum[kWarps];
  long long cta_sum[2][kMaxCluster];
  unsigned long long lane_scan[kWarps];
  float px[QNRE_MAX_NODES], qx[QNRE_MAX_NODES], u[QNRE_MAX_NODES];
  int token[QNRE_MAX_NODES], parent[QNRE_MAX_NODES], path[QNRE_MAX_NODES], gone[QNRE_MAX_NODES];
  double a, R;
  int node, todo, gone_count, length, found, last;
};

template <bool HAS_Q>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs g) {
  __shared__ Shared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const uint32_t rank = ptx::cluster_ctarank();
  const int req = blockIdx.x / ncta;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const long long seg0 = static_cast<long long>(rank * kWarps + warp) * g.seg;
  const long long seg1 = min(seg0 + g.seg, g.vocab);

  if (tid < g.nodes) {
    const long long at = static_cast<long long>(req) * g.nodes + tid;
    const int count = g.node_counts != nullptr ? g.node_counts[req] : g.nodes;
    int parent = tid > 0 && tid < count ? g.parents[at] : -1;
    const int x = g.tokens[at];
    if (parent >= tid || parent < 0 || x < 0 || x >= g.vocab) parent = -1;
    sh.parent[tid] = parent;
    sh.token[tid] = x;
    sh.u[tid] = g.accept_u[at];
    sh.px[tid] = parent >= 0 ? g.p[req * g.ps0 + parent * g.ps1 + x] : 0.f;
    sh.qx[tid] = HAS_Q && parent >= 0 ? g.q[req * g.qs0 + parent * g.qs1 + x] : 1.f;
  }
  if (tid == 0) {
    sh.a = 0.0;
    sh.R = 1.0;
    sh.node = sh.path[0] = 0;
    sh.length = 1;
    sh.gone_count = 0;
  }
  __syncwarp();
  ptx::cluster_sync();  // every CTA of the cluster runs before any writes to another's shared memory

  unsigned pass = 0;
  // The sum of max(p - a q, 0) over the vocabulary at `node` (without the tokens in sh.gone where they count),
  // by runs: each warp's in sh.warp_sum, each CTA's in sh.cta_sum, the total returned.
  auto sum_pass = [&](int node, double a, int gone) -> long long {
    const float* p = g.p + req * g.ps0 + node * g.ps1;
    const float* q = HAS_Q ? g.q + req * g.qs0 + node * g.qs1 : nullptr;
    const float ah = static_cast<float>(a), al = static_cast<float>(a - static_cast<double>(ah));
    const bool drafts = HAS_Q && a != 0.0;
    float hi = 0.f, lo = 0.f;
    for (long long x0 = seg0 + lane; x0 < seg1; x0 += 32 * kUnroll) {
      float pv[kUnroll], qv[kUnroll];
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        const bool in = x0 + 32 * e < seg1;
        pv[e] = in ? __ldg(p + x0 + 32 * e) : 0.f;
        qv[e] = in && drafts ? __ldg(q + x0 + 32 * e) : 0.f;
      }
      if (!HAS_Q) {
        for (int i = 0; i < gone; ++i)
#pragma unroll
          for (int e = 0; e < kUnroll; ++e)
            if (x0 + 32 * e == sh.gone[i]) pv[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        float dh, dl;
        residual(pv[e], qv[e], ah, al, dh, dl);
        const float s = __fadd_rn(hi, dh), t = __fsub_rn(s, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(dh, t));
        hi = s;
        lo = __fadd_rn(lo, __fadd_rn(err, dl));
      }
    }
    long long v = to_fixed(hi, lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) sh.warp_sum[warp] = v;
    __syncthreads();
    const unsigned buf = pass++ & 1u;
    if (tid < static_cast<int>(ncta)) {  // this CTA's sum to CTA tid of the cluster
      long long t = 0;
      for (int i = 0; i < kWarps; ++i) t += sh.warp_sum[i];
      const uint32_t at = ptx::mapa_shared(ptx::smem_addr(&sh.cta_sum[buf][rank]), tid);
      asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at), "l"(t) : "memory");
    }
    // two buffers: a CTA writes one again only after a later barrier, which all arrive at having read it
    __syncwarp();
    ptx::cluster_sync();
    long long total = 0;
    for (uint32_t i = 0; i < ncta; ++i) total += sh.cta_sum[buf][i];
    return total;
  };

  // The walk, by warp 0 of every CTA alike (all see the same sums); it stops for a
  // sum (todo 1) or at the last node (todo 0).
  uint64_t children = 0;
  bool fresh = true;
  long long Z = 0;
  bool have_sum = false;
  while (true) {
    if (warp == 0) {
      int node = sh.node, gone = sh.gone_count, length = sh.length;
      double a = sh.a, R = sh.R;
      int todo = 0;
      while (true) {
        if (fresh) {
          const bool c0 = lane < g.nodes && lane > 0 && sh.parent[lane] == node;
          const bool c1 = lane + 32 < g.nodes && sh.parent[lane + 32] == node;
          children = __ballot_sync(0xFFFFFFFFu, c0) |
                     static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, c1)) << 32;
          fresh = false;
        }
        if (children == 0) break;
        const int i = __ffsll(static_cast<long long>(children)) - 1;
        children &= children - 1;
        const double qx = sh.qx[i];
        double left = __dsub_rn(static_cast<double>(sh.px[i]), HAS_Q ? __dmul_rn(a, qx) : 0.0);
        if (!HAS_Q)
          for (int k = 0; k < gone; ++k)
            if (sh.gone[k] == sh.token[i]) left = 0.0;
        if (!(left > 0.0)) left = 0.0;
        if (__dmul_rn(__dmul_rn(static_cast<double>(sh.u[i]), qx), R) < left) {
          node = i;
          a = 0.0;
          R = 1.0;
          gone = 0;
          fresh = true;
          if (lane == 0) sh.path[length] = i;
          ++length;
        } else if (HAS_Q) {
          a = __dadd_rn(a, R);
          todo = 1;
          break;
        } else {
          R = __dsub_rn(R, left);
          __syncwarp();
          if (lane == 0) sh.gone[gone] = sh.token[i];
          ++gone;
        }
        __syncwarp();
      }
      if (lane == 0) {
        sh.node = node;
        sh.a = a;
        sh.R = R;
        sh.gone_count = gone;
        sh.length = length;
        sh.todo = todo;
      }
    }
    __syncthreads();
    const int todo = sh.todo;
    if (todo == 0) {
      // sums of an earlier pass stand only if it was at this node
      if (sh.a == 0.0) have_sum = false;
      break;
    }
    const double a = sh.a;
    Z = sum_pass(sh.node, a, 0);
    have_sum = true;
    if (tid == 0) sh.R = static_cast<double>(Z) / kFixed;
    __syncthreads();
  }

  const int node = sh.node;
  double a = sh.a;
  int gone = sh.gone_count;
  if (!have_sum) Z = sum_pass(node, a, gone);
  if (Z <= 0 && (a != 0.0 || gone != 0)) {  // nothing is left: the target itself
    a = 0.0;
    gone = 0;
    Z = sum_pass(node, a, gone);
  }
  const unsigned buf = (pass - 1) & 1u;

  if (rank == 0) {
    if (tid < g.nodes) g.path[static_cast<long long>(req) * g.nodes + tid] = tid < sh.length ? sh.path[tid] : -1;
    if (tid == 0) g.counts[req] = sh.length;
    if (Z <= 0 && tid == 0) g.next[req] = -1;
  }
  if (Z > 0) {
    // the lowest token whose running sum passes t: its CTA, its warp's run, then itself
    const long long t = min(static_cast<long long>(static_cast<double>(g.sample_u[req]) * static_cast<double>(Z)), Z - 1);
    long long before = 0;
    uint32_t owner = 0;
    while (owner + 1 < ncta && before + sh.cta_sum[buf][owner] <= t) before += sh.cta_sum[buf][owner++];
    if (owner == rank) {
      int w = 0;
      while (w + 1 < kWarps && before + sh.warp_sum[w] <= t) before += sh.warp_sum[w++];
      const long long s0 = static_cast<long long>(rank * kWarps + w) * g.seg, s1 = min(s0 + g.seg, g.vocab);
      const float* p = g.p + req * g.ps0 + node * g.ps1;
      const float* q = HAS_Q ? g.q + req * g.qs0 + node * g.qs1 : nullptr;
      const float ah = static_cast<float>(a), al = static_cast<float>(a - static_cast<double>(ah));
      if (tid == 0) {
        sh.found = 0x7FFFFFFF;
        sh.last = -1;
      }
      __syncthreads();
      for (long long base = s0; base < s1; base += kThreads) {
        const long long x = base + tid;
        float hi = 0.f, lo = 0.f;
        if (x < s1) {
          float pv = __ldg(p + x);
          if (!HAS_Q)
            for (int i = 0; i < gone; ++i)
              if (sh.gone[i] == x) pv = 0.f;
          residual(pv, HAS_Q && a != 0.0 ? __ldg(q + x) : 0.f, ah, al, hi, lo);
        }
        long long v = to_fixed(hi, lo);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xFFFFFFFFu, v, o);
          if (lane >= o) v += up;
        }
        if (lane == 31) sh.lane_scan[warp] = static_cast<unsigned long long>(v);
        __syncthreads();
        long long add = before;
        for (int i = 0; i < warp; ++i) add += static_cast<long long>(sh.lane_scan[i]);
        if (x < s1 && hi > 0.f) {
          atomicMax(&sh.last, static_cast<int>(x));
          if (add + v > t) atomicMin(&sh.found, static_cast<int>(x));
        }
        for (int i = 0; i < kWarps; ++i) before += static_cast<long long>(sh.lane_scan[i]);
        __syncthreads();
        if (sh.found != 0x7FFFFFFF) break;
      }
      // the run's own sum may differ from its elements' by their last bits: then its last token with mass
      if (tid == 0) g.next[req] = sh.found != 0x7FFFFFFF ? sh.found : sh.last;
    }
  }
  __syncwarp();
  ptx::cluster_sync();  // no CTA leaves while another may still write to its shared memory
}

// Pointer doubling over the parents: six rounds cover 64 nodes.
__global__ void __launch_bounds__(QNRE_MAX_NODES) masks_kernel(const int32_t* parents, int nodes, uint64_t* masks,
                                                              int32_t* depths) {
  __shared__ uint64_t anc[QNRE_MAX_NODES];
  __shared__ int up[QNRE_MAX_NODES];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int i = threadIdx.x;
  const long long at = static_cast<long long>(blockIdx.x) * nodes + i;
  const int parent = i < nodes ? parents[at] : -1;
  anc[i] = 1ull << i;
  up[i] = parent >= 0 && parent < i ? parent : -1;
  for (int round = 0; round < 6; ++round) {
    __syncthreads();
    const int u = up[i];
    const uint64_t more = u >= 0 ? anc[u] : 0;
    const int next = u >= 0 ? up[u] : -1;
    __syncthreads();
    anc[i] |= more;
    up[i] = next;
  }
  if (i < nodes) {
    if (masks != nullptr) masks[at] = anc[i];
    if (depths != nullptr) depths[at] = __popcll(anc[i]) - 1;
  }
}

template <typename K, typename... A>
qnre_status_t launch(K kernel, unsigned grid, unsigned block, unsigned cluster, qnre_stream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return from_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

}  // namespace

extern "C" {

qnre_status_t qnre_verify_tree(const float* target_probs, int64_t target_stride0, int64_t target_stride1,
                               const float* draft_probs, int64_t draft_stride0, int64_t draft_stride1, int n, int nodes,
                               int64_t vocab, const int32_t* tokens, const int32_t* parents, const int32_t* node_counts,
                               const float* accept_u, const float* sample_u, int32_t* path, int32_t* counts,
                               int32_t* next_token, qnre_stream_t stream) {
  if (n < 0 || nodes < 1 || vocab < 1) return QNRE_ERR_INVALID_ARG;
  if (nodes > QNRE_MAX_NODES || n > (1 << 20) || vocab >= (int64_t{1} << 31) - 65536) return QNRE_ERR_CAPACITY;
  if (n == 0) return QNRE_OK;
  if (target_probs == nullptr || tokens == nullptr || parents == nullptr || accept_u == nullptr ||
      sample_u == nullptr || path == nullptr || counts == nullptr || next_token == nullptr)
    return QNRE_ERR_INVALID_ARG;
  for (int64_t s : {target_stride0, target_stride1, draft_probs != nullptr ? draft_stride0 : 0,
                    draft_probs != nullptr ? draft_stride1 : 0}) {
    if (s < 0) return QNRE_ERR_INVALID_ARG;
    if (s > (int64_t{1} << 40)) return QNRE_ERR_CAPACITY;
  }
  const void* ptrs[] = {target_probs, draft_probs, tokens, parents, node_counts, accept_u, sample_u, path, counts,
                        next_token};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return QNRE_ERR_ALIGNMENT;
  // outputs against inputs and one another
  auto rows = [&](const float* p, int64_t s0, int64_t s1) {
    return p == nullptr ? ByteRange{0, 0} : span(p, ((n - 1) * s0 + (nodes - 1) * s1 + vocab) * 4);
  };
  const uint64_t tree = static_cast<uint64_t>(n) * nodes * 4, one = static_cast<uint64_t>(n) * 4;
  const ByteRange in[] = {rows(target_probs, target_stride0, target_stride1), rows(draft_probs, draft_stride0, draft_stride1),
                          span(tokens, tree), span(parents, tree),
                          node_counts != nullptr ? span(node_counts, one) : ByteRange{0, 0}, span(accept_u, tree),
                          span(sample_u, one)};
  const ByteRange outs[] = {span(path, tree), span(counts, one), span(next_token, one)};
  for (int i = 0; i < 3; ++i) {
    for (const ByteRange& r : in)
      if (overlaps(outs[i], r)) return QNRE_ERR_ALIAS;
    if (overlaps(outs[i], outs[(i + 1) % 3])) return QNRE_ERR_ALIAS;
  }
  // As many CTAs a request as fill the machine once (four of 512 threads a SM), while each keeps
  // 2048 entries or more.
  unsigned cluster = kMaxCluster;
  while (cluster > 1 && (static_cast<int64_t>(n) * cluster > 152 * 4 || vocab < static_cast<int64_t>(cluster) * 2048))
    cluster /= 2;
  const int64_t warps = static_cast<int64_t>(cluster) * kWarps;
  const int seg = static_cast<int>(((vocab + warps - 1) / warps + 31) / 32 * 32);
  const VerifyArgs a{target_probs, draft_probs, target_stride0, target_stride1, draft_stride0, draft_stride1, tokens,
                     parents, node_counts, accept_u, sample_u, path, counts, next_token, vocab, nodes, seg};
  return draft_probs != nullptr ? launch(verify_kernel<true>, n * cluster, kThreads, cluster, stream, a)
                                : launch(verify_kernel<false>, n * cluster, kThreads, cluster, stream, a);
}

qnre_status_t qnre_tree_masks(const int32_t* parents, int n, int nodes, uint64_t* masks, int32_t* depths,
                              qnre_stream_t stream) {
  if (n < 0 || nodes < 1) return QNRE_ERR_INVALID_ARG;
  if (nodes > QNRE_MAX_NODES || n > (1 << 20)) return QNRE_ERR_CAPACITY;
  if (n == 0) return QNRE_OK;
  if (parents == nullptr) return QNRE_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(masks, 8) || !aligned(depths, 4)) return QNRE_ERR_ALIGNMENT;
  const uint64_t count = static_cast<uint64_t>(n) * nodes;
  const ByteRange in = span(parents, count * 4);
  const ByteRange m = masks != nullptr ? span(masks, count * 8) : ByteRange{0, 0};
  const ByteRange d = depths != nullptr ? span(depths, count * 4) : ByteRange{0, 0};
  if (overlaps(in, m) || overlaps(in, d) || overlaps(m, d)) return QNRE_ERR_ALIAS;
  return launch(masks_kernel, n, QNRE_MAX_NODES, 1, stream, parents, nodes, masks, depths);
}

}  // extern "C"
