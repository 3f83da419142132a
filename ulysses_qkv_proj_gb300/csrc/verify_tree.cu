// verify_tree.cu -- verification of drafted trees against the target's probabilities, and
// the masks and depths of a tree.
//
// The walk itself is a few comparisons a node; what costs is a rejection, whose sum
// over the vocabulary is R = sum max(p - a q, 0), and the last one's running sum, from which the next token is
// drawn.  A cluster of up to 16 CTAs takes one request: every warp of it owns one run of the vocabulary,
// in order, so the sums of a pass are also the prefix that locates the drawn token, and only
// the run that holds it is read again (from L2).  All p(x), q(x) of the drafted tokens are fetched before
// the walk, so a level without a rejection reads nothing.
//
// Numbers.  The integers must not depend on the order of a sum, so sums are exact where it matters: an element
// p - a q is formed as an unevaluated pair of floats (2^-48 relative; a is split the same way), a lane
// adds pairs with the error kept, and lanes, warps and CTAs add 64-bit integers of 2^-56.  The first child of a
// node is tested exactly in fp32 (u q as a product and its error).
// fp64 would serve too, but this chip issues two of its operations a cycle and SM, 64 times fewer.
//
// Bound: latency (start, fetch, one pass, search: 8 us for four requests of 32003 entries); for
// many requests the passes' arithmetic and loads, the longest walk last.  48 trees of 32 nodes over 131075
// entries (1.8 passes a request, four at most): 54 us with 512 threads a CTA, eight CTAs a request
// and fp64 at the ends of a pass (two waves of clusters); 45 with integer conversions by shifts, exact fp32 first tests
// and 256 threads; 35 with 16 CTAs of 128 threads, eight places a thread in the search and the short residual.
// Two or eight loads a lane in flight instead of four: +5 %, +15 %.
#include "../../include/qnre.h"
#include "api_util.cuh"
#include "ptx.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

namespace {

using namespace qnre;
using namespace qnre::api;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kUnroll = 4;  // 16-byte loads of p and of q a lane has in flight
constexpr double kUnfix = 1.0 / 72057594037927936.0;  // 2^-56, the unit of the integer sums

struct VerifyArgs {
  const float* p;
  const float* q;
  long long ps0, ps1, qs0, qs1;
  const int32_t *tokens, *parents, *node_counts;
  const float *accept_u, *sample_u;
  int32_t *path, *counts, *next;
  long long vocab;
  int nodes, seg;  // seg: places a warp owns
};

// Packed pairs of floats: one instruction for two vocabulary entries.  Every operation is one IEEE rounding.
using f2 = uint64_t;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) { return fma2(b, pair(-1.f, -1.f), a); }

// s + e = a + b exactly (Knuth).
__device__ __forceinline__ void two_sum(f2 a, f2 b, f2& s, f2& e) {
  s = add2(a, b);
  const f2 t = sub2(s, a);
  e = add2(sub2(a, sub2(s, t)), sub2(b, t));
}

// max(p - a q, 0) as an unevaluated sum hi + lo, a = ah + al; `neg_ah` is -ah twice.
__device__ __forceinline__ void residual(f2 p, f2 q, f2 neg_ah, f2 neg_al, f2& hi, f2& lo) {
  const f2 ph = fma2(neg_ah, q, 0);                            // -ah q, rounded
  const f2 pl = fma2(neg_al, q, fma2(neg_ah, q, sub2(0, ph)));  // what that lost, and -al q
  hi = add2(p, ph);
  lo = add2(add2(sub2(p, hi), ph), pl);  // exact where p >= ah q; elsewhere nothing is kept
  const float2 v = halves(add2(hi, lo));
  const float2 h = halves(hi), l = halves(lo);
  hi = pair(v.x > 0.f ? h.x : 0.f, v.y > 0.f ? h.y : 0.f);
  lo = pair(v.x > 0.f ? l.x : 0.f, v.y > 0.f ? l.y : 0.f);
}

// x in units of 2^-56, |x| < 64, by shifts (the 64-bit conversion instruction runs at fp64's rate).
__device__ __forceinline__ long long to_fixed(float x) {
  const uint32_t b = __float_as_uint(x);
  const int e = static_cast<int>((b >> 23) & 0xFFu);
  const uint32_t m = (b & 0x7FFFFFu) | (e != 0 ? 0x800000u : 0u);
  const int up = max(e, 1) - (127 + 23 - 56);
  const long long v = up >= 0 ? static_cast<long long>(static_cast<uint64_t>(m) << up) : (up > -32 ? m >> -up : 0u);
  return (b >> 31) ? -v : v;
}

struct Shared {
  long long warp_sum[kWarps];
  long long cta_sum[2][kMaxCluster];
  long long lane_scan[kWarps];
  float px[QNRE_MAX_NODES], qx[QNRE_MAX_NODES], u[QNRE_MAX_NODES];
  int token[QNRE_MAX_NODES], parent[QNRE_MAX_NODES], path[QNRE_MAX_NODES], gone[QNRE_MAX_NODES];
  double a, R;
  long long t;
  float ah, al;  // a as a pair of floats
  int node, todo, gone_count, length, found, last;
};

// The probability rows of a node.  Warps own runs of places y = x + shift, where place 0 lies on a
// 16-byte boundary of p's row; q is read the same way where its row lies alike, else entry by entry.
struct Row {
  const float *p, *q;  // of place 0
  int shift, end;
  bool drafts, alike;
  __device__ __forceinline__ Row(const VerifyArgs& g, int req, int node, bool with_drafts) {
    p = g.p + req * g.ps0 + node * g.ps1;
    q = with_drafts ? g.q + req * g.qs0 + node * g.qs1 : p;
    shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
    alike = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    drafts = with_drafts;
    end = static_cast<int>(g.vocab) + shift;
    p -= shift;
    q -= shift;
  }
  __device__ __forceinline__ float4 load(const float* row, int y) const {
    if (y >= shift && y + 4 <= end && (row == p || alike)) return __ldg(reinterpret_cast<const float4*>(row + y));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (y >= shift && y < end) v.x = __ldg(row + y);
    if (y + 1 >= shift && y + 1 < end) v.y = __ldg(row + y + 1);
    if (y + 2 >= shift && y + 2 < end) v.z = __ldg(row + y + 2);
    if (y + 3 >= shift && y + 3 < end) v.w = __ldg(row + y + 3);
    return v;
  }
};

template <bool HAS_Q>
__global__ void __launch_bounds__(kThreads, 6) verify_kernel(const VerifyArgs g) {
  __shared__ Shared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const uint32_t rank = ptx::cluster_ctarank();
  const int req = blockIdx.x / ncta;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int seg0 = static_cast<int>(rank * kWarps + warp) * g.seg, seg1 = seg0 + g.seg;

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
    sh.ah = sh.al = 0.f;
    sh.node = sh.path[0] = 0;
    sh.length = 1;
    sh.gone_count = 0;
  }
  __syncwarp();
  ptx::cluster_sync();  // every CTA of the cluster runs before any writes to another's shared memory

  unsigned pass = 0;
  // The sum of max(p - a q, 0) over the vocabulary at `node` (without the tokens in sh.gone where they count),
  // by runs: each warp's in sh.warp_sum, each CTA's in sh.cta_sum, the total returned.
  auto sum_pass = [&](int node, float ah, float al, int gone) -> long long {
    const Row r(g, req, node, HAS_Q && ah != 0.f);
    const f2 nh = pair(-ah, -ah), nl = pair(-al, -al);
    f2 hi2 = 0, lo2 = 0;
    for (int y0 = seg0 + 4 * lane; y0 < seg1; y0 += 128 * kUnroll) {
      float4 pv[kUnroll], qv[kUnroll];
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        const int y = y0 + 128 * e;
        pv[e] = qv[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (y < seg1) {
          pv[e] = r.load(r.p, y);
          if (HAS_Q && r.drafts) qv[e] = r.load(r.q, y);
        }
      }
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        if (!HAS_Q) {
          for (int i = 0; i < gone; ++i) {
            const int k = sh.gone[i] + r.shift - (y0 + 128 * e);
            if (k == 0) pv[e].x = 0.f;
            if (k == 1) pv[e].y = 0.f;
            if (k == 2) pv[e].z = 0.f;
            if (k == 3) pv[e].w = 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          f2 dh = k ? pair(pv[e].z, pv[e].w) : pair(pv[e].x, pv[e].y), dl = 0, err;
          if (HAS_Q && r.drafts) residual(dh, k ? pair(qv[e].z, qv[e].w) : pair(qv[e].x, qv[e].y), nh, nl, dh, dl);
          two_sum(hi2, dh, hi2, err);
          lo2 = add2(lo2, add2(err, dl));
        }
      }
    }
    const float2 hs = halves(hi2), ls = halves(lo2);
    long long v = to_fixed(hs.x) + to_fixed(hs.y) + to_fixed(ls.x) + to_fixed(ls.y);
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
  bool fresh = true, untried = true;  // children not listed yet; none of them refused yet
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
        const float px = sh.px[i], qx = sh.qx[i], u = sh.u[i];
        double left = 0.0;
        bool accepted;
        if (untried) {  // u q < p, the product with its error: exact
          const float m = __fmul_rn(u, qx), err = __fmaf_rn(u, qx, -m);
          accepted = m < px || (m == px && err < 0.f);
          if (!HAS_Q) left = px > 0.f ? px : 0.0;
        } else {
          left = __dsub_rn(static_cast<double>(px), HAS_Q ? __dmul_rn(a, static_cast<double>(qx)) : 0.0);
          if (!HAS_Q)
            for (int k = 0; k < gone; ++k)
              if (sh.gone[k] == sh.token[i]) left = 0.0;
          if (!(left > 0.0)) left = 0.0;
          accepted = __dmul_rn(__dmul_rn(static_cast<double>(u), static_cast<double>(qx)), R) < left;
        }
        untried = accepted;
        if (accepted) {
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
        sh.ah = static_cast<float>(a);
        sh.al = static_cast<float>(a - static_cast<double>(sh.ah));
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
      if (sh.ah == 0.f) have_sum = false;
      break;
    }
    Z = sum_pass(sh.node, sh.ah, sh.al, 0);
    have_sum = true;
    if (tid == 0) sh.R = static_cast<double>(Z) * kUnfix;
    __syncthreads();
  }

  const int node = sh.node;
  float ah = sh.ah, al = sh.al;
  int gone = sh.gone_count;
  if (!have_sum) Z = sum_pass(node, ah, al, gone);
  if (Z <= 0 && (ah != 0.f || gone != 0)) {  // nothing is left: the target itself
    ah = al = 0.f;
    gone = 0;
    Z = sum_pass(node, ah, al, gone);
  }
  const unsigned buf = (pass - 1) & 1u;

  if (rank == 0) {
    if (tid < g.nodes) g.path[static_cast<long long>(req) * g.nodes + tid] = tid < sh.length ? sh.path[tid] : -1;
    if (tid == 0) g.counts[req] = sh.length;
    if (Z <= 0 && tid == 0) g.next[req] = -1;
  }
  if (Z > 0) {
    // the lowest token whose running sum passes t: its CTA, its warp's run, then itself
    if (tid == 0)
      sh.t = min(static_cast<long long>(static_cast<double>(g.sample_u[req]) * static_cast<double>(Z)), Z - 1);
    __syncthreads();
    const long long t = sh.t;
    long long before = 0;
    uint32_t owner = 0;
    while (owner + 1 < ncta && before + sh.cta_sum[buf][owner] <= t) before += sh.cta_sum[buf][owner++];
    if (owner == rank) {
      int w = 0;
      while (w + 1 < kWarps && before + sh.warp_sum[w] <= t) before += sh.warp_sum[w++];
      const int s0 = static_cast<int>(rank * kWarps + w) * g.seg, s1 = s0 + g.seg;
      const Row r(g, req, node, HAS_Q && ah != 0.f);
      if (tid == 0) {
        sh.found = 0x7FFFFFFF;
        sh.last = -1;
      }
      __syncthreads();
      // a thread takes eight places in a row, so one scan of the block covers the run
      for (int base = s0; base < s1; base += kThreads * 8) {
        const int y0 = base + tid * 8;
        float4 pv[2], qv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = y0 + 4 * e < s1;
          pv[e] = in ? r.load(r.p, y0 + 4 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
          qv[e] = in && HAS_Q && r.drafts ? r.load(r.q, y0 + 4 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        long long mine[8];
        const float ps[8] = {pv[0].x, pv[0].y, pv[0].z, pv[0].w, pv[1].x, pv[1].y, pv[1].z, pv[1].w};
        const float qs[8] = {qv[0].x, qv[0].y, qv[0].z, qv[0].w, qv[1].x, qv[1].y, qv[1].z, qv[1].w};
        long long v = 0;
        uint32_t mass = 0;  // places with anything left
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          f2 dh = pair(ps[e], ps[e + 1]), dl = 0;
          if (!HAS_Q) {
            float2 d = halves(dh);
            for (int i = 0; i < gone; ++i) {
              if (sh.gone[i] + r.shift == y0 + e) d.x = 0.f;
              if (sh.gone[i] + r.shift == y0 + e + 1) d.y = 0.f;
            }
            dh = pair(d.x, d.y);
          } else if (r.drafts) {
            residual(dh, pair(qs[e], qs[e + 1]), pair(-ah, -ah), pair(-al, -al), dh, dl);
          }
          const float2 h = halves(dh), l = halves(dl);
          mine[e] = to_fixed(h.x) + to_fixed(l.x);
          mine[e + 1] = to_fixed(h.y) + to_fixed(l.y);
          v += mine[e] + mine[e + 1];
          mass |= (h.x + l.x > 0.f ? 1u << e : 0u) | (h.y + l.y > 0.f ? 2u << e : 0u);
        }
        const long long own = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xFFFFFFFFu, v, o);
          if (lane >= o) v += up;
        }
        if (lane == 31) sh.lane_scan[warp] = v;
        __syncthreads();
        long long run = before + v - own;
        for (int i = 0; i < warp; ++i) run += sh.lane_scan[i];
        if (mass != 0) atomicMax(&sh.last, y0 - r.shift + 31 - __clz(mass));
        if (run + own > t) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            run += mine[e];
            if ((mass >> e & 1) && run > t) {
              atomicMin(&sh.found, y0 - r.shift + e);
              break;
            }
          }
        }
        for (int i = 0; i < kWarps; ++i) before += sh.lane_scan[i];
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

// A cluster of more than eight CTAs has to be asked for once a device and kernel.
template <bool HAS_Q>
bool allow_large_clusters() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (ready.load() & bit) return true;
  if (cudaFuncSetAttribute(verify_kernel<HAS_Q>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return false;
  ready.fetch_or(bit);
  return true;
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
  // As many CTAs a request as the machine about holds at once (six to eight a SM), while each keeps 1024
  // entries or more: walks differ in length, and a lone long one is spread over as many SMs as
  // its cluster has CTAs.
  unsigned cluster = kMaxCluster;
  while (cluster > 1 && (static_cast<int64_t>(n) * cluster > 152 * 8 || vocab < static_cast<int64_t>(cluster) * 1024))
    cluster /= 2;
  const int64_t warps = static_cast<int64_t>(cluster) * kWarps;
  const int seg = static_cast<int>(((vocab + 3 + warps - 1) / warps + 127) / 128 * 128);  // + 3: the shift
  const VerifyArgs a{target_probs, draft_probs, target_stride0, target_stride1, draft_stride0, draft_stride1, tokens,
                     parents, node_counts, accept_u, sample_u, path, counts, next_token, vocab, nodes, seg};
  if (cluster > 8 && !(draft_probs != nullptr ? allow_large_clusters<true>() : allow_large_clusters<false>()))
    return QNRE_ERR_CUDA;
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
