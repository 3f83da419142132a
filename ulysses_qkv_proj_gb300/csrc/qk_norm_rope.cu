// qk_norm_rope.cu -- per-head RMSNorm and position rotation of q and k in memory:
// forward, gradient, and the form that writes new tokens' K and V into a paged
// cache.  The operator is the fused projection's epilogue (eps 1e-6, fp32
// throughout, one rounding at the end), for any number of query and key heads.
//
//   r = rsqrt(mean(y^2) + 1e-6),  n = y r w,  o = R n          (R: rotation by the token's angles)
//   gradient:  t = R^T g,  h = y r,  dw = sum t h,  dy = r (t w - h mean(t w h))
//
// Bound: HBM (4 bytes an element forward, 6 backward), with the issue slots close behind: a row pair of
// 512 bytes costs about 100 instructions of the 174 slots its bytes take.  A head row is D/8 lanes of 16
// bytes; a warp takes one token's run of heads, so angles and weights sit in registers
// (weights already times cosines and sines), the channel a rotation mixes in is four word
// shuffles away (half-rotation) or in the same lane, and the arithmetic is on packed pairs of floats.
// Measured on 32768 tokens of 72 heads, D = 128 bf16 (1.22 GB): plain floats 264 us at 155 instructions;
// packed, four blocks of 256 threads a SM, 217; the first loads issued before the position's angles are
// asked for, 209; one resident wave that strides over the items, 199 (three blocks 215, two 268; 128-thread
// blocks 205; streaming stores +2 %).  The gradient (18881 tokens of 70 heads, fp16, 1.02 GB): 282 us
// with plain loads, 209 with the next heads' loads in flight, 183 packed with all heads of a token in one
// item, 175 with the loads through a ring in shared memory (two stages of 16 KB a block in flight; three
// blocks a SM 185, four 246; 16 heads an item 174, 8 205), 165 back to back on warm pages (178 before); 167
// with the weights' sums in three levels.
#include "../../include/qnre.h"
#include "cache.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

namespace {

using namespace qnre;
using namespace qnre::api;

constexpr int kThreads = 256;
constexpr float kEps = 1e-6f;
constexpr int kGradBlocks = 152 * 2;  // blocks of the gradient; each leaves one partial sum of dw

struct View {
  char* data;
  long long sb, ss, sh;  // bytes
  __device__ __forceinline__ char* row(int b, int s, int h) const { return data + b * sb + s * ss + h * sh; }
};

struct NormArgs {
  View q, k, v, q_out, k_out;  // gradient: gq, gk in v_q / v_k below
  View gq, gk;
  const void* wq;
  const void* wk;
  const float* cos_sin;
  const int32_t* positions;
  long long n_pos;
  int rot, B, S, Hq, Hk;
  int cq, ck, hq, hk;  // chunks of q (k, v) heads a token, heads a chunk
  const int32_t* rows;
  const int32_t* counts;
  CacheView cache;
  int layer;
  float* partial;  // gradient: [kGradBlocks][2][D]
};

// Eight 16-bit values as four packed pairs of floats; sm_103 has multiply-adds of such pairs.
using Pairs = uint64_t[4];

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// to += from, from = 0.
__device__ __forceinline__ void fold(Pairs& to, Pairs& from) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    to[i] = add2(to[i], from[i]);
    from[i] = 0;
  }
}

template <bool BF16>
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
  if (BF16) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(p.x, p.y);
}

template <bool BF16>
__device__ __forceinline__ void unpack(const uint4& u, Pairs& f) {
  f[0] = unpack2<BF16>(u.x);
  f[1] = unpack2<BF16>(u.y);
  f[2] = unpack2<BF16>(u.z);
  f[3] = unpack2<BF16>(u.w);
}

template <bool BF16>
__device__ __forceinline__ uint4 pack(const Pairs& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = halves(f[i]);
    if (BF16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __half2 p = __floats2half2_rn(v.x, v.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The dot product of two lanes' eight channels, before the row's lanes are added.
__device__ __forceinline__ float dot(const Pairs& a, const Pairs& b) {
  uint64_t t = mul2(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) t = fma2(a[i], b[i], t);
  const float2 v = halves(t);
  return v.x + v.y;
}

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// One lane's share of a token's rotation: channel 8*l + e of the output is
// c[e] n[e] + s[e] n'[e], n' the other channel of its pair (sign in s).  Half-rotation: the
// pair lies in lane `partner`, else in the neighbouring element.  Channels past the rotated ones have
// c = 1, s = 0 and themselves for a pair.
struct Angles {
  float c[8], s[8];
  int partner;
};

// (Plain loads, not read-only ones: the kernels start beside the launch before theirs, which may write the table.)
template <bool RH, bool BACK>
__device__ __forceinline__ Angles load_angles(const float* row, int rot, int l, int lane) {
  Angles a;
  const int half = rot / 2;
  a.partner = lane;
  if (8 * l >= rot) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a.c[e] = 1.f;
      a.s[e] = 0.f;
    }
    return a;
  }
  if (RH) {
    const bool low = 8 * l < half;
    const int i0 = low ? 8 * l : 8 * l - half;
    a.partner = low ? lane + half / 8 : lane - half / 8;
    const float4* c4 = reinterpret_cast<const float4*>(row + i0);
    const float4* s4 = reinterpret_cast<const float4*>(row + half + i0);
    const float4 c0 = c4[0], c1 = c4[1], s0 = s4[0], s1 = s4[1];
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a.c[e] = c[e];
      a.s[e] = low != BACK ? -s[e] : s[e];
    }
  } else {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * l);
    const float4 s = *reinterpret_cast<const float4*>(row + half + 4 * l);
    const float cc[4] = {c.x, c.y, c.z, c.w}, sc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a.c[2 * e] = a.c[2 * e + 1] = cc[e];
      a.s[2 * e] = BACK ? sc[e] : -sc[e];
      a.s[2 * e + 1] = BACK ? -sc[e] : sc[e];
    }
  }
  return a;
}

// The pairs' other channels of one head row held as `raw`; every lane of the warp takes part.
template <bool RH, bool BF16>
__device__ __forceinline__ void other_channels(const uint4& raw, const Angles& a, Pairs& y) {
  uint4 o;
  if (RH) {
    o.x = __shfl_sync(0xFFFFFFFFu, raw.x, a.partner);
    o.y = __shfl_sync(0xFFFFFFFFu, raw.y, a.partner);
    o.z = __shfl_sync(0xFFFFFFFFu, raw.z, a.partner);
    o.w = __shfl_sync(0xFFFFFFFFu, raw.w, a.partner);
  } else {
    o = make_uint4(__byte_perm(raw.x, 0, 0x1032), __byte_perm(raw.y, 0, 0x1032), __byte_perm(raw.z, 0, 0x1032),
                   __byte_perm(raw.w, 0, 0x1032));
  }
  unpack<BF16>(o, y);
}

__device__ __forceinline__ void pairs_of(const float (&f)[8], Pairs& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
}

// Forward.  Work item = (token, chunk of q, k or v heads); kAppend sends k and v to the cache.
template <int D, bool BF16, bool RH, bool APPEND>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kUnroll = 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % 32, l = lane % kLanes, sub = lane / kLanes;
  const int per_token = a.cq + a.ck + (APPEND ? a.ck : 0);
  const long long items = static_cast<long long>(a.B) * a.S * per_token;
  const long long stride = static_cast<long long>(gridDim.x) * (kThreads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; it < items; it += stride) {
    const long long token = it / per_token;
    int chunk = static_cast<int>(it - token * per_token);
    const int b = static_cast<int>(token / a.S), s = static_cast<int>(token - static_cast<long long>(b) * a.S);
    const int kind = chunk < a.cq ? 0 : (chunk < a.cq + a.ck ? 1 : 2);
    chunk -= kind == 0 ? 0 : (kind == 1 ? a.cq : a.cq + a.ck);
    const int step = kind == 0 ? a.hq : a.hk, heads = kind == 0 ? a.Hq : a.Hk;
    const int h0 = chunk * step, h1 = min(h0 + step, heads);
    const View& in = kind == 0 ? a.q : (kind == 1 ? a.k : a.v);

    int page = -1, at = 0, holders = 0;
    long long pos = s;
    if (APPEND) {
      const int row = a.rows[b];
      const bool row_ok = row >= 0 && row < a.cache.rows;
      at = row_ok ? a.cache.length(row) : 0;
      pos = static_cast<long long>(at) + s;
      if (kind != 0) {
        if (a.counts != nullptr && s >= a.counts[b]) continue;
        if (row_ok && pos <= 0x7FFFFFFF) page = a.cache.page_of(row, static_cast<int>(pos));
        at = static_cast<int>(pos);
        if (page < 0) {
          if (lane == 0) atomicOr(a.cache.status, row_ok ? QNRE_CACHE_BAD_PAGE : QNRE_CACHE_BAD_ROW);
          continue;
        }
        // a page that other rows hold too is not written; the count arrives while the values do
        holders = a.cache.refs[page];
      }
    }
    auto out_row = [&](int h) -> char* {
      if (APPEND && kind != 0) return (kind == 1 ? a.cache.k : a.cache.v) + a.cache.token_offset(a.layer, page, h, at);
      return (kind == 0 ? a.q_out : a.k_out).row(b, s, h);
    };
    if (APPEND && kind == 2) {
      for (int h = h0 + sub; h < h1; h += kRows) {
        const uint4 x = reinterpret_cast<const uint4*>(in.row(b, s, h))[l];
        if (holders <= 1) reinterpret_cast<uint4*>(out_row(h))[l] = x;
      }
      if (holders > 1 && lane == 0) atomicOr(a.cache.status, QNRE_CACHE_BAD_PAGE);
      continue;
    }
    // the first heads are on their way before the position and its angles are asked for
    uint4 raw[kUnroll];
    const char* src = in.row(b, s, h0 + sub) + 16 * l;
    const long long src_step = in.sh * kRows;
    auto load = [&](int h) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        raw[u] = h + u * kRows < h1 ? __ldcs(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
        src += src_step;
      }
    };
    load(h0 + sub);
    if (a.positions != nullptr) pos = a.positions[token];
    const bool bad = pos < 0 || pos >= a.n_pos;
    const Angles ang = load_angles<RH, false>(a.cos_sin + (bad ? 0 : pos) * a.rot, a.rot, l, lane);
    Pairs w, wp;  // weights times cosines, the other channels' weights times sines
    {
      Pairs c, sn;
      pairs_of(ang.c, c);
      pairs_of(ang.s, sn);
      const uint4 raw = static_cast<const uint4*>(kind == 0 ? a.wq : a.wk)[l];
      unpack<BF16>(raw, w);
      other_channels<RH, BF16>(raw, ang, wp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = mul2(w[i], c[i]);
        wp[i] = mul2(wp[i], sn[i]);
      }
    }
    char* dst = out_row(h0 + sub) + 16 * l;
    const long long dst_step = (APPEND && kind != 0 ? static_cast<long long>(a.cache.page_size) * (D * 2)
                                                    : (kind == 0 ? a.q_out : a.k_out).sh) * kRows;
    for (int h = h0 + sub; h - sub < h1; h += kRows * kUnroll) {
      if (h != h0 + sub) load(h);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        Pairs x, y, o;
        unpack<BF16>(raw[u], x);
        float r = rsqrtf(row_sum<kLanes>(dot(x, x)) * (1.0f / D) + kEps);
        if (bad) r = __uint_as_float(0x7FC00000u);
        const uint64_t r2 = pair(r, r);
        other_channels<RH, BF16>(raw[u], ang, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mul2(fma2(x[i], w[i], mul2(y[i], wp[i])), r2);
        if (h + u * kRows < h1 && (!APPEND || holders <= 1)) *reinterpret_cast<uint4*>(dst) = pack<BF16>(o);
        dst += dst_step;
      }
    }
  }
}

// 16 bytes from global to this lane's place in shared memory, in flight until waited for; zeros where !live.
__device__ __forceinline__ void copy_async(uint32_t dst, const char* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// Gradient.  An item is a token's run of heads, taken kRows * kUnroll heads a step; the steps of all of a warp's items
// follow one another through a ring of kStages in shared memory (a lane reads back only what it asked for itself), so
// that loads of two or three steps are in flight whatever the registers hold.  Each thread sums dw of its channels
// over its items, the block sums its threads in a fixed order and leaves one partial row for grad_weights_kernel.
// A thread's terms grow with the batch (131072 tokens of 64 heads: 1700), so it adds them in three levels, of at most
// 62 terms, 64 such sums, and the rest: a term passes 126 additions and one for each 1024 steps of its thread (131072
// tokens of one head are 54 steps), then the block's 16 or 32 and the blocks' 42.  (One level: 165 us on the long case
// instead of 167, and 5.0e-5 off where 3450 equal terms a thread are 1.1e-6 off now.)
template <int D, bool BF16, bool RH>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_grad_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kUnroll = 2, kStep = kRows * kUnroll, kStages = 3;
  // [warp][stage][x or g][head of the step][lane]; afterwards the threads' sums [warp * kRows][D]
  __shared__ uint4 ring[kThreads / 32][kStages][2][kUnroll][32];
  static_assert(sizeof(ring) >= kThreads / 32 * kRows * D * sizeof(float), "the sums fit in the ring");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % 32, l = lane % kLanes, sub = lane / kLanes, warp = threadIdx.x / 32;
  const uint32_t place = static_cast<uint32_t>(__cvta_generic_to_shared(&ring[warp][0][0][0][lane]));
  constexpr uint32_t kStageBytes = sizeof(ring[0][0]), kSideBytes = sizeof(ring[0][0][0]), kHeadBytes = sizeof(ring[0][0][0][0]);
  for (int kind = 0; kind < 2; ++kind) {
    const int chunks = kind == 0 ? a.cq : a.ck, step = kind == 0 ? a.hq : a.hk, heads = kind == 0 ? a.Hq : a.Hk;
    const View& in = kind == 0 ? a.q : a.k;
    const View& grad = kind == 0 ? a.gq : a.gk;
    const View& out = kind == 0 ? a.q_out : a.k_out;
    const long long x_step = in.sh * kRows, g_step = grad.sh * kRows, o_step = out.sh * kRows;
    Pairs dw = {0, 0, 0, 0}, dw1 = {0, 0, 0, 0}, dw2 = {0, 0, 0, 0};
    const int item_steps = (step + kStep - 1) / kStep;  // of kUnroll terms each, 16 at the most
    int steps = 0, folds = 0;  // since the level above was added to
    const long long items = static_cast<long long>(a.B) * a.S * chunks;
    const long long stride = static_cast<long long>(gridDim.x) * (kThreads / 32);
    // k's items from the other end: the warps that had one of q's more than others get one of k's less
    const long long place_of = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
    const long long first = kind == 0 ? place_of : stride - 1 - place_of;
    Pairs w;
    unpack<BF16>(static_cast<const uint4*>(kind == 0 ? a.wq : a.wk)[l], w);

    struct Item {
      long long token;
      int b, s, h0, h1;
    };
    auto item_of = [&](long long it) {
      Item r;
      r.token = it / chunks;
      const int chunk = static_cast<int>(it - r.token * chunks);
      r.b = static_cast<int>(r.token / a.S);
      r.s = static_cast<int>(r.token - static_cast<long long>(r.b) * a.S);
      r.h0 = chunk * step;
      r.h1 = min(r.h0 + step, heads);
      return r;
    };
    // the step to be asked for next
    long long ask_it = first;
    int ask_h = 0, ask_h1 = 0;
    const char *px = nullptr, *pg = nullptr;
    auto begin = [&] {
      if (ask_it >= items) return;
      const Item r = item_of(ask_it);
      ask_h = r.h0 + sub;
      ask_h1 = r.h1;
      px = in.row(r.b, r.s, ask_h) + 16 * l;
      pg = grad.row(r.b, r.s, ask_h) + 16 * l;
    };
    uint32_t ask_stage = 0, stage = 0;
    auto ask = [&] {
      if (ask_it < items) {
        const uint32_t at = place + ask_stage * kStageBytes;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const bool live = ask_h + u * kRows < ask_h1;
          copy_async(at + u * kHeadBytes, live ? px : in.data, live);
          copy_async(at + kSideBytes + u * kHeadBytes, live ? pg : grad.data, live);
          px += x_step;
          pg += g_step;
        }
        ask_h += kStep;
        if (ask_h - sub >= ask_h1) {
          ask_it += stride;
          begin();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      ask_stage = ask_stage + 1 == kStages ? 0 : ask_stage + 1;
    };
    begin();
    for (int i = 0; i < kStages - 1; ++i) ask();

    for (long long it = first; it < items; it += stride) {
      const Item r = item_of(it);
      const long long pos = a.positions != nullptr ? a.positions[r.token] : r.s;
      const bool bad = pos < 0 || pos >= a.n_pos;
      const Angles ang = load_angles<RH, true>(a.cos_sin + (bad ? 0 : pos) * a.rot, a.rot, l, lane);
      Pairs c, sn;
      pairs_of(ang.c, c);
      pairs_of(ang.s, sn);
      char* po = out.row(r.b, r.s, r.h0 + sub) + 16 * l;
      for (int h = r.h0 + sub; h - sub < r.h1; h += kStep) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        const uint4(*here)[kUnroll][32] = ring[warp][stage];
        uint4 xr[kUnroll], gr[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          xr[u] = here[0][u][lane];
          gr[u] = here[1][u][lane];
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
        ask();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const bool live = h + u * kRows < r.h1;
          Pairs x, g, gp, o;
          unpack<BF16>(xr[u], x);
          unpack<BF16>(gr[u], g);
          float rs = rsqrtf(row_sum<kLanes>(dot(x, x)) * (1.0f / D) + kEps);
          if (bad && live) rs = __uint_as_float(0x7FC00000u);
          const uint64_t r2 = pair(rs, rs);
          other_channels<RH, BF16>(gr[u], ang, gp);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t t = fma2(g[i], c[i], mul2(gp[i], sn[i]));
            x[i] = mul2(x[i], r2);
            dw[i] = fma2(t, x[i], dw[i]);
            o[i] = mul2(t, w[i]);
          }
          const float mean = row_sum<kLanes>(dot(o, x)) * (1.0f / D);
          const uint64_t minus = pair(-mean, -mean);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul2(r2, fma2(x[i], minus, o[i]));
          if (live) *reinterpret_cast<uint4*>(po) = pack<BF16>(o);
          po += o_step;
        }
      }
      steps += item_steps;
      if (steps >= 16) {
        fold(dw1, dw);
        steps = 0;
        if (++folds == 64) {
          fold(dw2, dw1);
          folds = 0;
        }
      }
    }
    fold(dw1, dw);
    fold(dw2, dw1);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // every warp is done with the ring
    float(*sums)[D] = reinterpret_cast<float(*)[D]>(ring);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float2*>(&sums[warp * kRows + sub][8 * l + 2 * i]) = halves(dw2[i]);
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.f;
      for (int i = 0; i < kThreads / 32 * kRows; ++i) t += sums[i][threadIdx.x];
      a.partial[(static_cast<long long>(blockIdx.x) * 2 + kind) * D + threadIdx.x] = t;
    }
    __syncthreads();
  }
}

// dw = the blocks' partial sums, in block order: 32 channels and 32 strands of blocks a block.
__global__ void __launch_bounds__(1024) grad_weights_kernel(const float* partial, int blocks, int D, float* dq,
                                                            float* dk) {
  __shared__ float strands[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + x;  // of 2 * D
  float t = 0.f;
  for (int i = y; i < blocks; i += 32) t += partial[static_cast<long long>(i) * 2 * D + col];
  strands[y][x] = t;
  __syncthreads();
  if (y == 0) {
    t = 0.f;
    for (int i = 0; i < 32; ++i) t += strands[i][x];
    (col < D ? dq : dk)[col < D ? col : col - D] = t;
  }
}

// ------------------------------------------------------------------ host side
qnre_status_t check_rows(const qnre_tensor4_t* view, ByteRange* range) {
  if (view == nullptr) return QNRE_ERR_INVALID_ARG;
  qnre_tensor4_t own = *view;
  const qnre_tensor4_t* t = &own;
  // a view without tokens may have no storage
  alignas(16) static char nothing[16];
  if (own.data == nullptr && (own.shape[0] == 0 || own.shape[1] == 0)) own.data = nothing;
  const qnre_status_t st = check_view(t, range);
  if (st != QNRE_OK) return st;
  if (t->dtype != QNRE_DTYPE_BF16 && t->dtype != QNRE_DTYPE_FP16) return QNRE_ERR_UNSUPPORTED;
  if (t->shape[3] != 64 && t->shape[3] != 128) return QNRE_ERR_UNSUPPORTED;
  for (int i = 0; i < 3; ++i)
    if (t->shape[i] > 0x7FFFFFFF) return QNRE_ERR_CAPACITY;
  if (!rows_vectorisable(t, 2)) return QNRE_ERR_ALIGNMENT;
  return QNRE_OK;
}

bool same_shape(const qnre_tensor4_t* a, const qnre_tensor4_t* b, bool heads) {
  for (int i = 0; i < 4; ++i)
    if ((i != 2 || heads) && a->shape[i] != b->shape[i]) return false;
  return a->dtype == b->dtype;
}

bool same_place(const qnre_tensor4_t* a, const qnre_tensor4_t* b) {
  if (a->data != b->data) return false;
  for (int i = 0; i < 4; ++i)
    if (a->shape[i] > 1 && a->stride[i] != b->stride[i]) return false;
  return true;
}

// An output view must not write an element twice: positive strides that do not nest
// in some order overlap.
bool self_overlaps(const qnre_tensor4_t* t) {
  int order[4] = {0, 1, 2, 3};
  std::sort(order, order + 4, [&](int a, int b) { return t->stride[a] < t->stride[b]; });
  int64_t reach = 0;
  for (int i : order) {
    if (t->shape[i] <= 1) continue;
    if (t->stride[i] <= reach) return true;
    reach += (t->shape[i] - 1) * t->stride[i];
  }
  return false;
}

View view4(const qnre_tensor4_t* t) {
  return View{static_cast<char*>(t->data), static_cast<long long>(t->stride[0]) * 2,
              static_cast<long long>(t->stride[1]) * 2, static_cast<long long>(t->stride[2]) * 2};
}

qnre_status_t check_table(const void* wq, const void* wk, const float* cos_sin, int64_t n_pos, int rot, int style, int D,
                          const int32_t* positions) {
  if (wq == nullptr || wk == nullptr || cos_sin == nullptr || n_pos < 1 || rot < 16 || rot > D || rot % 16 != 0)
    return QNRE_ERR_INVALID_ARG;
  if (style != QNRE_ROPE_ROTATE_HALF && style != QNRE_ROPE_INTERLEAVED) return QNRE_ERR_INVALID_ARG;
  if (!aligned(wq, 16) || !aligned(wk, 16) || !aligned(cos_sin, 16) || !aligned(positions, 4))
    return QNRE_ERR_ALIGNMENT;
  return n_pos > (int64_t{1} << 31) ? QNRE_ERR_CAPACITY : QNRE_OK;
}

// Heads a work item takes: few enough that small calls fill the machine with warps, up to
// `most` (whose loads share one read of the angles).
void set_chunks(NormArgs& a, int D, int most_steps) {
  const int rows = 32 / (D / 8);
  const int64_t tokens = static_cast<int64_t>(a.B) * a.S;
  const int64_t warps = 152 * 8 * 4;
  int steps = most_steps;  // of `rows` heads
  while (steps > 1 && tokens * ((a.Hq + a.Hk) / (rows * steps)) < warps) steps /= 2;
  auto split = [&](int heads, int* chunks, int* per) {
    *chunks = (heads + rows * steps - 1) / (rows * steps);
    *per = (heads + *chunks - 1) / *chunks;
    *per = (*per + rows - 1) / rows * rows;
    *chunks = (heads + *per - 1) / *per;
  };
  split(a.Hq, &a.cq, &a.hq);
  split(a.Hk, &a.ck, &a.hk);
}

template <typename K, typename... A>
qnre_status_t launch(K kernel, unsigned grid, unsigned block, qnre_stream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return from_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

template <bool APPEND>
qnre_status_t run_forward(NormArgs& a, int D, bool bf16, bool rh, qnre_stream_t stream) {
  set_chunks(a, D, 8);
  const int64_t items = static_cast<int64_t>(a.B) * a.S * (a.cq + a.ck * (APPEND ? 2 : 1));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((items + 7) / 8, 152 * 4));
  using Fn = void (*)(NormArgs);
  static const Fn fns[8] = {
      norm_rope_kernel<64, false, false, APPEND>, norm_rope_kernel<64, false, true, APPEND>,
      norm_rope_kernel<64, true, false, APPEND>,  norm_rope_kernel<64, true, true, APPEND>,
      norm_rope_kernel<128, false, false, APPEND>, norm_rope_kernel<128, false, true, APPEND>,
      norm_rope_kernel<128, true, false, APPEND>, norm_rope_kernel<128, true, true, APPEND>};
  return launch(fns[(D == 128 ? 4 : 0) + (bf16 ? 2 : 0) + (rh ? 1 : 0)], grid, kThreads, stream, a);
}

// Fills what the three entry points share; checks q, k and the table.
qnre_status_t common(NormArgs& a, const qnre_tensor4_t* q, const qnre_tensor4_t* k, ByteRange* rq, ByteRange* rk,
                     const void* wq, const void* wk, const float* cos_sin, int64_t n_pos, int rot, int style,
                     const int32_t* positions) {
  qnre_status_t st = check_rows(q, rq);
  if (st == QNRE_OK) st = check_rows(k, rk);
  if (st != QNRE_OK) return st;
  if (!same_shape(q, k, false)) return QNRE_ERR_INVALID_ARG;
  st = check_table(wq, wk, cos_sin, n_pos, rot, style, static_cast<int>(q->shape[3]), positions);
  if (st != QNRE_OK) return st;
  if (q->shape[0] * q->shape[1] > (int64_t{1} << 40)) return QNRE_ERR_CAPACITY;
  a.q = view4(q);
  a.k = view4(k);
  a.wq = wq;
  a.wk = wk;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.n_pos = n_pos;
  a.rot = rot;
  a.B = static_cast<int>(q->shape[0]);
  a.S = static_cast<int>(q->shape[1]);
  a.Hq = static_cast<int>(q->shape[2]);
  a.Hk = static_cast<int>(k->shape[2]);
  return QNRE_OK;
}

qnre_status_t check_out(const qnre_tensor4_t* out, const qnre_tensor4_t* like, ByteRange* range) {
  const qnre_status_t st = check_rows(out, range);
  if (st != QNRE_OK) return st;
  if (!same_shape(out, like, true) || self_overlaps(out)) return QNRE_ERR_INVALID_ARG;
  return QNRE_OK;
}

}  // namespace

extern "C" {

qnre_status_t qnre_qk_norm_rope(const qnre_tensor4_t* q, const qnre_tensor4_t* k, const void* q_norm_w,
                                const void* k_norm_w, const float* cos_sin, int64_t n_pos, int rot, int rope_style,
                                const int32_t* positions, const qnre_tensor4_t* q_out, const qnre_tensor4_t* k_out,
                                qnre_stream_t stream) {
  NormArgs a{};
  ByteRange rq, rk, ro, rp;
  qnre_status_t st = common(a, q, k, &rq, &rk, q_norm_w, k_norm_w, cos_sin, n_pos, rot, rope_style, positions);
  if (st == QNRE_OK) st = check_out(q_out, q, &ro);
  if (st == QNRE_OK) st = check_out(k_out, k, &rp);
  if (st != QNRE_OK) return st;
  if ((!same_place(q_out, q) && views_overlap(q_out, ro, q, rq)) || views_overlap(q_out, ro, k, rk) ||
      (!same_place(k_out, k) && views_overlap(k_out, rp, k, rk)) || views_overlap(k_out, rp, q, rq) ||
      views_overlap(q_out, ro, k_out, rp))
    return QNRE_ERR_ALIAS;
  if (a.B == 0 || a.S == 0) return QNRE_OK;
  a.q_out = view4(q_out);
  a.k_out = view4(k_out);
  return run_forward<false>(a, static_cast<int>(q->shape[3]), q->dtype == QNRE_DTYPE_BF16,
                            rope_style == QNRE_ROPE_ROTATE_HALF, stream);
}

qnre_status_t qnre_qk_norm_rope_workspace_bytes(int head_dim, uint64_t* bytes) {
  if (bytes == nullptr) return QNRE_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return QNRE_ERR_UNSUPPORTED;
  *bytes = static_cast<uint64_t>(kGradBlocks) * 2 * head_dim * sizeof(float);
  return QNRE_OK;
}

qnre_status_t qnre_qk_norm_rope_backward(const qnre_tensor4_t* gq, const qnre_tensor4_t* gk, const qnre_tensor4_t* q,
                                         const qnre_tensor4_t* k, const void* q_norm_w, const void* k_norm_w,
                                         const float* cos_sin, int64_t n_pos, int rot, int rope_style,
                                         const int32_t* positions, const qnre_tensor4_t* dq, const qnre_tensor4_t* dk,
                                         float* dq_norm_w, float* dk_norm_w, void* workspace, uint64_t workspace_bytes,
                                         qnre_stream_t stream) {
  NormArgs a{};
  ByteRange rq, rk, rgq, rgk, rdq, rdk;
  qnre_status_t st = common(a, q, k, &rq, &rk, q_norm_w, k_norm_w, cos_sin, n_pos, rot, rope_style, positions);
  if (st == QNRE_OK) st = check_rows(gq, &rgq);
  if (st == QNRE_OK) st = check_rows(gk, &rgk);
  if (st == QNRE_OK && (!same_shape(gq, q, true) || !same_shape(gk, k, true))) st = QNRE_ERR_INVALID_ARG;
  if (st == QNRE_OK) st = check_out(dq, q, &rdq);
  if (st == QNRE_OK) st = check_out(dk, k, &rdk);
  if (st != QNRE_OK) return st;
  const int D = static_cast<int>(q->shape[3]);
  if (dq_norm_w == nullptr || dk_norm_w == nullptr || workspace == nullptr) return QNRE_ERR_INVALID_ARG;
  if (!aligned(dq_norm_w, 4) || !aligned(dk_norm_w, 4) || !aligned(workspace, 16)) return QNRE_ERR_ALIGNMENT;
  uint64_t need = 0;
  qnre_qk_norm_rope_workspace_bytes(D, &need);
  if (workspace_bytes < need) return QNRE_ERR_CAPACITY;
  if ((!same_place(dq, gq) && views_overlap(dq, rdq, gq, rgq)) || views_overlap(dq, rdq, gk, rgk) ||
      (!same_place(dk, gk) && views_overlap(dk, rdk, gk, rgk)) || views_overlap(dk, rdk, gq, rgq) ||
      views_overlap(dq, rdq, q, rq) || views_overlap(dq, rdq, k, rk) || views_overlap(dk, rdk, q, rq) ||
      views_overlap(dk, rdk, k, rk) || views_overlap(dq, rdq, dk, rdk))
    return QNRE_ERR_ALIAS;
  const ByteRange extra[3] = {span(dq_norm_w, D * 4), span(dk_norm_w, D * 4), span(workspace, need)};
  for (int i = 0; i < 3; ++i) {
    for (const ByteRange& r : {rq, rk, rgq, rgk, rdq, rdk})
      if (overlaps(extra[i], r)) return QNRE_ERR_ALIAS;
    if (overlaps(extra[i], extra[(i + 1) % 3])) return QNRE_ERR_ALIAS;
  }
  a.gq = view4(gq);
  a.gk = view4(gk);
  a.q_out = view4(dq);
  a.k_out = view4(dk);
  a.partial = static_cast<float*>(workspace);
  set_chunks(a, D, 32);
  // no tokens: the kernels run all the same and leave zero weight gradients
  const int64_t items = static_cast<int64_t>(a.B) * a.S * std::max(a.cq, a.ck);
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((items + 7) / 8, kGradBlocks)));
  using Fn = void (*)(NormArgs);
  static const Fn fns[8] = {
      norm_rope_grad_kernel<64, false, false>,  norm_rope_grad_kernel<64, false, true>,
      norm_rope_grad_kernel<64, true, false>,   norm_rope_grad_kernel<64, true, true>,
      norm_rope_grad_kernel<128, false, false>, norm_rope_grad_kernel<128, false, true>,
      norm_rope_grad_kernel<128, true, false>,  norm_rope_grad_kernel<128, true, true>};
  const bool bf16 = q->dtype == QNRE_DTYPE_BF16, rh = rope_style == QNRE_ROPE_ROTATE_HALF;
  st = launch(fns[(D == 128 ? 4 : 0) + (bf16 ? 2 : 0) + (rh ? 1 : 0)], grid, kThreads, stream, a);
  if (st != QNRE_OK) return st;
  return launch(grad_weights_kernel, 2 * D / 32, 1024, stream, static_cast<const float*>(a.partial),
                static_cast<int>(grid), D, dq_norm_w, dk_norm_w);
}

qnre_status_t qnre_qkv_norm_rope_append(const qnre_tensor4_t* q, const qnre_tensor4_t* k, const qnre_tensor4_t* v,
                                        const void* q_norm_w, const void* k_norm_w, const float* cos_sin,
                                        int64_t n_pos, int rot, int rope_style, const int32_t* positions,
                                        const qnre_tensor4_t* q_out, const qnre_cache_t* cache, int layer,
                                        const int32_t* rows, const int32_t* counts, qnre_stream_t stream) {
  NormArgs a{};
  ByteRange rq, rk, rv, ro;
  qnre_status_t st = common(a, q, k, &rq, &rk, q_norm_w, k_norm_w, cos_sin, n_pos, rot, rope_style, positions);
  if (st == QNRE_OK) st = check_rows(v, &rv);
  if (st == QNRE_OK && !same_shape(v, k, true)) st = QNRE_ERR_INVALID_ARG;
  if (st == QNRE_OK) st = check_out(q_out, q, &ro);
  if (st == QNRE_OK) st = check_cache(cache, static_cast<int>(std::min<int64_t>(q->shape[0], 0x7FFFFFFF)));
  if (st != QNRE_OK) return st;
  if (cache->heads != k->shape[2] || cache->head_dim != k->shape[3] || cache->dtype != k->dtype || layer < 0 ||
      layer >= cache->layers)
    return QNRE_ERR_INVALID_ARG;
  if (rows == nullptr && a.B > 0) return QNRE_ERR_INVALID_ARG;
  if (!aligned(rows, 4) || !aligned(counts, 4)) return QNRE_ERR_ALIGNMENT;
  if ((!same_place(q_out, q) && views_overlap(q_out, ro, q, rq)) || views_overlap(q_out, ro, k, rk) ||
      views_overlap(q_out, ro, v, rv))
    return QNRE_ERR_ALIAS;
  for (const void* pool : {cache->k, cache->v}) {
    const ByteRange rc = span(pool, pool_bytes(cache));
    if (overlaps(rc, rq) || overlaps(rc, rk) || overlaps(rc, rv) || overlaps(rc, ro)) return QNRE_ERR_ALIAS;
  }
  if (a.B == 0 || a.S == 0) return QNRE_OK;
  a.v = view4(v);
  a.q_out = view4(q_out);
  a.rows = rows;
  a.counts = counts;
  a.cache = view_of(cache);
  a.layer = layer;
  return run_forward<true>(a, static_cast<int>(q->shape[3]), q->dtype == QNRE_DTYPE_BF16,
                           rope_style == QNRE_ROPE_ROTATE_HALF, stream);
}

}  // extern "C"
