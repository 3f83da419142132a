// sample.cu -- tokens, or filtered probabilities, from logits: temperature, top-k, top-p and min-p.
//
//   w_x = exp((l_x - max l) / T);  order: by logit, then by index
//   kept: w_x >= min_p; of those the top_k first; of those the ones before which less than top_p of their weight lies
//   token = lowest x whose running sum of kept weights (by index) exceeds u times their total
//
// A cluster of up to 16 CTAs takes one row.  Few rows are held in its shared memory (KEEP), so that the passes that follow cost
// little latency; with many rows a CTA's share is longer, and the passes read it again, from L2 as far as it reaches.  Nothing is
// sorted but the few tokens around a cut:
//
//   max        while the row arrives; every CTA learns it through the cluster's shared memory,
//   histogram  counts over 4096 bins of log2(e) (max - l) / T, 1/128 wide, which orders tokens coarsely; each CTA adds up its
//              share of the bins over the cluster.  The bin of the top_k-th token is exact from the counts.  For top_p
//              the counts bound the weight up to each bin, and the one behind it, from both sides (a bin spans 0.54 %), so
//              the cut falls into one of a few bins; one pass then adds up exactly the weight before them, theirs by bins
//              and the row's, which the bounds do without,
//   cut        the tokens of the one bin go to the first CTA, which sorts them and finds the last one kept; bins of more
//              than 1024 (ties, logits beyond the bins' range) are cut by four rounds of eight key bits
//              (over the CTAs' lists where these hold them: 64 rows of mixed settings 84 -> 65 us),
//   draw       the kept weight by warps' runs of places; the run that holds the number is added up place by place.
//
// Numbers.  A token is right only if no sum is wrong by more than its distance from a border, and with 10^5 borders
// 32-bit sums would miss one draw in a hundred.  So weights are integers of 2^-(62 - ceil log2 V) of the largest with 31 leading
// bits of their own: the exponent is formed as a pair of floats, its leading ten binary places taken from a table of
// 2^(-j/1024) and the rest by a cubic (Weight; 2^-30 relative at worst, and sums of V of them far closer, as their errors are
// independent; none of its instructions is a conversion or 64 bits wide but the last).  Integer sums do not depend
// on their order, so counters and lists filled in any order change no result.
//
// Bound: for few rows, latency: one row of 32003 logits takes 6.9 us (about 2 each for the maximum over the cluster, the
// weights and the draw), 20 rows with top_k 24 (each phase's code runs once, so it is fetched as it runs). For many rows,
// instructions: counting and weighing a logit are some 60, and every SM issues at about half its rate behind fixed latencies,
// so 256 rows of 131075 take 188 us where reading them once would take 10, and 1024 such rows written as probabilities 545.
// What the passes cost those 256 rows on the way (each step with the ones before): logits read in runs of 16, out of the
// instruction cache, 1014 us; short loops 412; kept tokens packed before they are weighed 318; powers from shared memory
// rather than L1, and the window's weights from the CTA's list rather than a pass of their own, 253; words converted when
// their turn comes 243; no branch around a weight 235; a top_p row weighed once, after its counts, 188.
// Tried and left: more and smaller CTAs for many rows (8 an SM: 246 us for 253, but 64 rows 149 for 93; 16 an SM: 285),
// skipping groups of logits that nobody keeps (331 for 318), loads of 8 bytes (262 for 253), two loads ahead (192 for 188),
// zeros written before the cut is known (24.7 for 24.3), four packed weights at a time (237 for 236).
#include "../../include/qnre.h"
#include "api_util.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

namespace {

using namespace qnre;
using namespace qnre::api;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kGrain = kWarps * 128;     // places of a CTA come in multiples of this: a float4 a lane, warp by warp
constexpr int kBins = 4096;
constexpr int kBinShift = 3;             // a bin is 2^3 steps of 2^-10 in log2; the last holds all beyond 32
constexpr int kList = 1024;              // tokens of one bin that are sorted
constexpr int kOwn = 2048;               // tokens that a CTA lists
constexpr int kWindow = 32;              // bins that a cut by weight is sought in (16-bit logits leave gaps of up to 20)
constexpr int kResident = 152 * 4;       // CTAs that the machine about holds at once
constexpr int64_t kInL2 = 96ll << 20;
constexpr int kKeepSlice = 12288;        // places of a CTA that it holds in shared memory (two or three such CTAs a SM)
constexpr int kMassBits = 40;            // of the histogram's bounds on weights
constexpr int kFixedBytes = kBins * 4 + kOwn * 8 + kList * 8 + 3 * 256 * 4;  // shared memory before the row
constexpr double kLog2e = 1.4426950408889634074;

struct SampleArgs {
  const void* logits;
  long long stride0, stride1;  // elements between requests, between a request's rows
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
  int rows_per, vocab, slice, up;  // rows of a request; places of a CTA; binary places of a weight beyond 31
};

// 2^(-j/1024) in units of 2^-31, from 2^(-i/32) and 2^(-i/1024).  Each CTA holds it in shared memory: 32 lanes' places of it lie
// in as many lines, so that from L1 each look-up of a warp took some 30 turns.
struct alignas(16) PowerTable {
  uint32_t at[1024];
};
constexpr uint64_t kCoarse[32] = {
    0x8000000000000000ull, 0x7D41D96DB915019Dull, 0x7A92BE8A92436616ull, 0x77F25CCDEE6D7AE6ull,
    0x75606373EE921C97ull, 0x72DC8373BE41A454ull, 0x70666F76154A7089ull, 0x6DFDDBCBED791BABull,
    0x6BA27E656B4EB57Aull, 0x69540EC8F895722Dull, 0x6712460A8FC24072ull, 0x64DCDEC3371793D1ull,
    0x62B39508AA836D6Full, 0x6096266533384A2Bull, 0x5E8451CFAC061B5Full, 0x5C7DD7A3B17DCF75ull,
    0x5A827999FCEF3242ull, 0x5891FAC0E95612C8ull, 0x56AC1F752150A563ull, 0x54D0AD5A753E077Cull,
    0x52FF6B54D8A89C75ull, 0x513821818624B40Cull, 0x4F7A993048D088D7ull, 0x4DC69CDCEAA72A9Cull,
    0x4C1BF828C6DC54B8ull, 0x4A7A77D47F7B84B1ull, 0x48E1E9B9D588E19Bull, 0x47521CC5A2E6A9E0ull,
    0x45CAE0F1F545EB73ull, 0x444C0740496D4294ull, 0x42D561B3E6243D8Aull, 0x4166C34C5615D0ECull};
constexpr uint64_t kFine[32] = {
    0x8000000000000000ull, 0x7FE9D3A8E07BF086ull, 0x7FD3AB290E46D769ull, 0x7FBD867FDF0ACB3Bull,
    0x7FA765ACA88F6453ull, 0x7F9148AEC0B9B7B1ull, 0x7F7B2F857D8C51E5ull, 0x7F651A30352731EEull,
    0x7F4F08AE3DC7C426ull, 0x7F38FAFEEDC8DD26ull, 0x7F22F1219BA2B4AEull, 0x7F0CEB159DEAE091ull,
    0x7EF6E8DA4B544F9Aull, 0x7EE0EA6EFAAF4479ull, 0x7ECAEFD302E950AFull, 0x7EB4F905BB0D4F78ull,
    0x7E9F06067A4360BAull, 0x7E8916D497D0E3F4ull, 0x7E732B6F6B18732Aull, 0x7E5D43D64B99DDD7ull,
    0x7E47600890F223DEull, 0x7E31800592DB7078ull, 0x7E1BA3CCA92D152Cull, 0x7E05CB5D2BDB84BEull,
    0x7DEFF6B672F84E24ull, 0x7DDA25D7D6B2177Full, 0x7DC458C0AF549908ull, 0x7DAE8F7055489813ull,
    0x7D98C9E62113E1FAull, 0x7D8308216B594720ull, 0x7D6D4A218CD895E5ull, 0x7D578FE5DE6E95A0ull};
constexpr uint64_t product63(uint64_t a, uint64_t b) {  // a b 2^-63, rounded
  const uint64_t ah = a >> 32, al = a & 0xFFFFFFFFull, bh = b >> 32, bl = b & 0xFFFFFFFFull;
  const uint64_t mid = ah * bl + (al * bl >> 32), mid2 = al * bh + (mid & 0xFFFFFFFFull);
  const uint64_t hi = ah * bh + (mid >> 32) + (mid2 >> 32), lo = mid2 << 32 | (al * bl & 0xFFFFFFFFull);
  return (hi << 1 | lo >> 63) + (lo >> 62 & 1);
}
constexpr PowerTable make_powers() {
  PowerTable t{};
  for (int j = 0; j < 1024; ++j) {
    const uint64_t x = product63(kCoarse[j / 32], kFine[j % 32]);
    t.at[j] = static_cast<uint32_t>((x + (1ull << 31)) >> 32);
  }
  return t;
}
__device__ const PowerTable kPowers = make_powers();

// Logits as integers of the same order (larger logit, larger key); both zeros have one key.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// A row's scale: weights are 2^(-y), y = (max - l) c, c = log2(e) / T as a pair of floats.
struct Weight {
  const uint32_t* power;
  float max, ch, cl;
  static constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer, in the low bits
  static constexpr float kLimit = 4095.f;

  // y in steps of 2^-10, rounded (ordered as the logits are); y itself stays in p, without its last places.
  __device__ __forceinline__ int steps(float l, float& p) const {
    p = fminf(fminf(max - l, 3.4028234664e38f) * ch, kLimit);
    return __float_as_int(fmaf(p, 1024.f, kMagic)) - __float_as_int(kMagic);
  }
  __device__ __forceinline__ int bin(float l) const {
    float p;
    return min(steps(l, p) >> kBinShift, kBins - 1);
  }
  // The least logit of bin b or before (a whole warp: 32 places of the range of floats at a time).
  __device__ float least_of(int b) const {
    if (b >= kBins - 1) return -3.4028234664e38f;
    if (b < 0) return INFINITY;
    uint32_t lo = key_of(-3.4028234664e38f) - 1, hi = key_of(max);  // beyond the bin; within
    while (hi - lo > 1) {
      const uint32_t step = (hi - lo + 31) / 32, k = min(lo + (threadIdx.x % 32 + 1) * step, hi);
      const uint32_t within = __ballot_sync(0xFFFFFFFFu, bin(of_key(k)) <= b);
      const uint32_t first = __ffs(within) - 1;
      hi = min(lo + (first + 1) * step, hi);
      lo += first * step;
    }
    return of_key(hi);
  }
  // 2^-y = m 2^-(31 + n)
  __device__ __forceinline__ uint32_t operator()(float l, int& n) const {
    float p;
    const int k = steps(l, p);
    const float d = max - l, back = d - max, err = (max - (d - back)) - (l + back);  // d + err = max - l
    const float e = fmaf(d, ch, -p) + fmaf(d, cl, err * ch);                          // y = p + e
    const float r = fmaf(e, 1024.f, fmaf(p, 1024.f, static_cast<float>(-k)));         // behind the steps
    const float t = r * 0.00067690154f;                                               // ln 2 / 1024
    const float c = t * fmaf(t, fmaf(t, -0.16666667f, 0.5f), -1.f);                   // e^-t - 1
    const uint32_t bits = power[k & 1023];
    const float value = __uint_as_float((bits >> 7) + (156u << 23));                  // bits, to 23 places
    n = k >> 10;
    return bits + (__float_as_int(fmaf(value, c, kMagic)) - __float_as_int(kMagic));
  }
  // In units of 2^-(31 + up), rounded; without a branch, so that a lane's logits overlap.
  __device__ __forceinline__ uint64_t fixed(float l, int up) const {
    int n;
    const uint64_t x = static_cast<uint64_t>((*this)(l, n)) << up;
    n = min(n, 63);  // (nothing is left of 2^61 and less; up is 31 for a single token alone)
    return (x + ((1ull << n) >> 1)) >> n;
  }
};

// What a row keeps: larger logits than `least`, and of that the tokens up to `last`.
struct Cut {
  float least;
  int last;
  __device__ __forceinline__ bool keeps(float l, int index) const { return l > least || (l == least && index <= last); }
};

struct Shared {
  PowerTable power;
  uint64_t sums[2][2][kMaxCluster];  // two sums of each of the cluster's CTAs, two uses in turn
  uint64_t warp[2][kWarps];
  uint64_t scratch[kWarps];
  float max[kMaxCluster];
  uint64_t before;                   // what lies before the first bin found
  Cut cut;
  uint32_t window[3][kWindow];       // of these bins: tokens, weights' low and high words
  uint32_t runs[2][kWarps];          // a list's weight in each run, low and high words
  uint32_t put_count, list_count;
  int bin[2], tie, low, high;
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16(x); }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half(x); }

// Words of the cluster's CTAs, by the address of this CTA's own.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  return ptx::mapa_shared(ptx::smem_addr(p), rank);
}
__device__ __forceinline__ uint32_t remote_load(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_cta(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void remote_store(void* p, uint32_t rank, uint32_t v) {
  ptx::st_shared_cluster_u32(in_cta(p, rank), v);
}
__device__ __forceinline__ void remote_store64(void* p, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(in_cta(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void remote_min(int* p, uint32_t rank, int v) {
  asm volatile("red.shared::cluster.min.s32 [%0], %1;" ::"r"(in_cta(p, rank)), "r"(v) : "memory");
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v) {  // inclusive
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// One row, as this CTA of its cluster sees it.
template <typename T, bool KEEP>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  Shared& sh;
  uint32_t* hist;    // [kBins]
  uint64_t* own;     // [kOwn]: tokens that this CTA put there, as (~key, index)
  uint64_t* list;    // [kList]: those of one bin from all CTAs; the first CTA's
  uint32_t* rounds;  // [3][256]: counts, weights' low and high words
  float* logit;      // [slice] (KEEP)
  const T* src;      // the row
  uint32_t ncta, rank;
  int place0, shift, end, run, up;  // places are index + shift, up to end; `run` of them to a warp, in order
  Weight weight;
  Cut cut;
  unsigned uses;
  bool listed;       // `own` holds all that may still be kept

  __device__ __forceinline__ static int warp() { return threadIdx.x / 32; }
  __device__ __forceinline__ static int lane() { return threadIdx.x % 32; }

  __device__ __forceinline__ uint64_t weigh(float l) const { return weight.fixed(l, up); }

  // Eight or four logits from place `place` on (a 16-byte boundary), as they lie in memory; what is no logit of the row as -inf.
  __device__ __forceinline__ uint4 fetch(int place) const {
    if (place >= shift && place + kVec <= end) return *reinterpret_cast<const uint4*>(src + (place - shift));
    uint4 w;
    T* t = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      t[i] = place + i >= shift && place + i < end ? src[place + i - shift] : from_float<T>(-INFINITY);
    return w;
  }
  __device__ __forceinline__ static void decode(uint4 w, float (&v)[kVec]) {  // (NaN: -inf)
    const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = clean(to_float(t[i]));
  }
  __device__ __forceinline__ static float clean(float v) { return fminf(fmaxf(v, -INFINITY), 3.4028234664e38f); }  // (NaN: -inf)
  __device__ __forceinline__ float at(int y) const {  // place y of this CTA
    if (KEEP) return logit[y];
    const int place = place0 + y;
    return place >= shift && place < end ? clean(to_float(src[place - shift])) : -INFINITY;
  }

  // f(logit, index) for every place of this warp's run, and some behind it as -inf, and after() behind each few: all lanes call
  // together.  The loops stay short: with 16 logits unrolled the passes that weigh ran out of the instruction cache.
  template <typename F, typename G>
  __device__ __forceinline__ void sweep(F f, G after) const {
    const int from = warp() * run, to = from + run;
    if (KEEP) {
#pragma unroll 1
      for (int y = from + lane() * 4; y < to; y += 128) {
        const float4 v = *reinterpret_cast<const float4*>(logit + y);
        const int index = place0 + y - shift;
        f(v.x, index);
        f(v.y, index + 1);
        f(v.z, index + 2);
        f(v.w, index + 3);
        after();
      }
    } else {
      // (the next words stay as they are: converted here they would be waited for before this step's work)
      uint4 next = fetch(from + lane() * kVec < to ? place0 + from + lane() * kVec : end);
#pragma unroll 1
      for (int first = from; first < to; first += 32 * kVec) {
        const int y = first + lane() * kVec, ahead = y + 32 * kVec;
        float v[kVec];
        decode(next, v);
        next = fetch(ahead < to ? place0 + ahead : end);
        const int index = place0 + y - shift;
#pragma unroll
        for (int i = 0; i < kVec; ++i) f(v[i], index + i);
        after();
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void sweep(F f) const {
    sweep(f, [] {});
  }
  template <typename F>
  __device__ __forceinline__ void sweep_kept(F f) const {
    sweep([&](float l, int index) {
      if (cut.keeps(l, index)) f(l, index);
    });
  }

  // f(logit, index) for every kept token, from the CTA's list where it holds them all.
  template <typename F>
  __device__ __forceinline__ void each_kept(F f) const {
    if (!listed) return sweep_kept(f);
    for (uint32_t i = threadIdx.x; i < sh.put_count; i += kThreads) {
      const uint64_t entry = own[i];
      const float l = logit_of(entry);
      const int index = static_cast<int>(static_cast<uint32_t>(entry));
      if (cut.keeps(l, index)) f(l, index);
    }
  }
  // A thread's share of its run's sum of the kept tokens' weights that pick(logit) names.
  template <typename F>
  __device__ __forceinline__ uint64_t kept_weight(F pick) {
    uint64_t sum = 0;
    if (!listed) {
      sweep_kept([&](float l, int) {
        if (pick(l)) sum += weigh(l);
      });
      return sum;
    }
    if (threadIdx.x < 2 * kWarps) sh.runs[0][threadIdx.x] = 0;
    __syncthreads();
    each_kept([&](float l, int index) {
      if (pick(l)) add_to(sh.runs[0], sh.runs[1], (index + shift - place0) / run, weigh(l));
    });
    __syncthreads();
    return lane() == 0 ? sh.runs[0][warp()] | static_cast<uint64_t>(sh.runs[1][warp()]) << 32 : 0;
  }
  // This warp's share of the weight of the kept tokens from `least` on, of which `few` are handed to f instead.  Kept
  // tokens are packed in shared memory (the histogram's, which is done with) until there are enough for all lanes: weighed where
  // they lie, a few of 32 lanes would cost as much as all.
  template <typename P, typename F>
  __device__ __forceinline__ uint64_t packed_weight(float least, P few, F f) {
    constexpr int kRoom = kBins / kWarps;
    float* queue = reinterpret_cast<float*>(hist) + warp() * kRoom;
    uint64_t sum = 0;
    int fill = 0;
    auto flush = [&] {
      __syncwarp();
      for (int i = lane(); i < fill; i += 32) sum += weigh(queue[i]);
      __syncwarp();
      fill = 0;
    };
    sweep([&](float l, int index) {
      const bool kept = l >= least && cut.keeps(l, index), apart = kept && few(l);
      const uint32_t votes = __ballot_sync(0xFFFFFFFFu, kept && !apart);
      if (kept && !apart) queue[fill + __popc(votes & ((1u << lane()) - 1u))] = l;
      fill += __popc(votes);
      if (apart) f(l, index);
    }, [&] {
      if (fill > kRoom - 32 * kVec) flush();
    });
    flush();
    return sum;
  }
  // A 64-bit sum in two words, by two atomics.
  __device__ __forceinline__ static void add_to(uint32_t* low, uint32_t* high, int at, uint64_t w) {
    const uint32_t part = static_cast<uint32_t>(w), old = atomicAdd(&low[at], part);
    atomicAdd(&high[at], static_cast<uint32_t>(w >> 32) + (old + part < old ? 1u : 0u));
  }

  struct Pair {
    uint64_t x, y;
  };
  // The row's sums of the threads' x and y.  sh.warp and sh.sums[this use] hold the warps' and the CTAs'.
  __device__ Pair exchange(uint64_t x, uint64_t y) {
    x = warp_sum(x);
    y = warp_sum(y);
    __syncthreads();
    if (lane() == 0) {
      sh.warp[0][warp()] = x;
      sh.warp[1][warp()] = y;
    }
    __syncthreads();
    const unsigned buf = uses++ & 1u;
    if (threadIdx.x < 2 * ncta) {
      const int which = threadIdx.x & 1;
      uint64_t s = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += sh.warp[which][i];
      remote_store64(&sh.sums[buf][which][rank], threadIdx.x >> 1, s);
    }
    __syncwarp();
    // two buffers: a CTA writes one again only after a later barrier, which all arrive at having read it
    ptx::cluster_sync();
    Pair t{0, 0};
    for (uint32_t i = 0; i < ncta; ++i) {
      t.x += sh.sums[buf][0][i];
      t.y += sh.sums[buf][1][i];
    }
    return t;
  }
  __device__ Pair before_cta() const {  // of the last exchange
    const unsigned buf = (uses - 1) & 1u;
    Pair t{0, 0};
    for (uint32_t i = 0; i < rank; ++i) {
      t.x += sh.sums[buf][0][i];
      t.y += sh.sums[buf][1][i];
    }
    return t;
  }

  // sh.bin[i]: the first bin with which reach(the bins' sum, i, their running sum) holds (the last bin where none does; never
  // before the first token); sh.before what lies before the first of them in x, sh.high its own x.
  template <typename F, typename G>
  __device__ Pair find_bins(F f, G reach) {
    const int share = kBins / ncta, per = share / kThreads, b0 = rank * share + threadIdx.x * per;
    Pair own{0, 0};
    for (int i = 0; i < per; ++i) {
      const Pair v = f(b0 + i);
      own.x += v.x;
      own.y += v.y;
    }
    if (threadIdx.x < 2) sh.bin[threadIdx.x] = kBins - 1;
    const uint64_t sx = warp_scan(own.x), sy = warp_scan(own.y);
    const Pair all = exchange(own.x, own.y);
    Pair before = before_cta();
    before.x += sx - own.x;
    before.y += sy - own.y;
    for (int i = 0; i < warp(); ++i) {
      before.x += sh.warp[0][i];
      before.y += sh.warp[1][i];
    }
    uint32_t seek = 0;
    const Pair upto{before.x + own.x, before.y + own.y};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (!reach(all, i, before) && reach(all, i, upto)) seek |= 1u << i;
    if (seek != 0) {
      for (int b = b0; b < b0 + per && seek != 0; ++b) {
        const Pair v = f(b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if ((seek >> i & 1) == 0 || !reach(all, i, Pair{before.x + v.x, before.y + v.y})) continue;
          seek &= ~(1u << i);
          for (uint32_t r = 0; r < ncta; ++r) {
            remote_store(&sh.bin[i], r, b);
            if (i == 0) {
              remote_store64(&sh.before, r, before.x);
              remote_store(&sh.high, r, static_cast<uint32_t>(v.x));
            }
          }
        }
        before.x += v.x;
        before.y += v.y;
      }
    }
    __syncwarp();
    ptx::cluster_sync();
    return all;
  }

  // This CTA's tokens that a cut may fall on, or (listed) all that may be kept; only the first kOwn find room.
  __device__ __forceinline__ void put(float l, int index) {
    const uint32_t at = atomicAdd(&sh.put_count, 1u);
    if (at < kOwn) own[at] = static_cast<uint64_t>(~key_of(l)) << 32 | static_cast<uint32_t>(index);
  }
  __device__ __forceinline__ static float logit_of(uint64_t entry) { return of_key(~static_cast<uint32_t>(entry >> 32)); }

  // The first CTA: the cluster's kept tokens of bin b into its list (no more than kList); returns how many (all were put,
  // and a barrier passed).
  __device__ int gather(int b) {
    uint32_t counts[kMaxCluster], all = 0;
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      counts[i] = i < static_cast<int>(ncta) ? remote_load(&sh.put_count, i) : 0;
      all += counts[i];
    }
    for (uint32_t at = threadIdx.x; at < all; at += kThreads) {
      uint32_t i = 0, in = at;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k)
        if (i == k && in >= counts[k]) {
          in -= counts[k];
          ++i;
        }
      uint64_t entry;
      asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(entry) : "r"(in_cta(&own[in], i)) : "memory");
      const float l = logit_of(entry);
      if (weight.bin(l) == b && cut.keeps(l, static_cast<int>(static_cast<uint32_t>(entry))))
        list[atomicAdd(&sh.list_count, 1u)] = entry;
    }
    __syncthreads();
    return static_cast<int>(sh.list_count);
  }

  __device__ void sort_list(int m) {  // ascending (bitonic), padded to a power of two
    int size = 32;
    while (size < m) size *= 2;
    for (int i = m + threadIdx.x; i < size; i += kThreads) list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = threadIdx.x; i < size / 2; i += kThreads) {
          const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
          const uint64_t x = list[lo], y = list[hi];
          if ((x > y) == ((lo & k) == 0)) {
            list[lo] = y;
            list[hi] = x;
          }
        }
        __syncthreads();
      }
  }

  // Cuts off what lies in bins [b0, b1] behind the first tokens that make up `want`, counted as tokens or by weight; where
  // b0 = b1 and the bin's `m` tokens fit the list, they were put there (and a cluster barrier passed).
  template <bool BY_WEIGHT>
  __device__ void cut_at(uint64_t want, int b0, int b1, uint32_t m, bool room) {
    if (b0 != b1 || m > kList || !room) {
      const Rounds found = cut_by_rounds<BY_WEIGHT>(*this, want, b0, b1);
      cut = found.cut;
      uses = found.uses;
    } else {
      if (rank == 0) {
        m = gather(b0);
        sort_list(m);
        int stay;  // entries before which less than `want` lies
        if (BY_WEIGHT) {
          constexpr int kPer = kList / kThreads;
          uint64_t w[kPer], own = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int at = threadIdx.x * kPer + i;
            w[i] = at < static_cast<int>(m) ? weigh(logit_of(list[at])) : 0;
            own += w[i];
          }
          const uint64_t upto = warp_scan(own);
          if (lane() == 31) sh.scratch[warp()] = upto;
          if (threadIdx.x == 0) sh.high = 0;
          __syncthreads();
          uint64_t before = upto - own;
          for (int i = 0; i < warp(); ++i) before += sh.scratch[i];
          int most = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int at = threadIdx.x * kPer + i;
            if (at < static_cast<int>(m) && before < want) most = at + 1;
            before += w[i];
          }
          if (most > 0) atomicMax(&sh.high, most);
          __syncthreads();
          stay = sh.high;
        } else {
          stay = static_cast<int>(want < m ? want : m);
        }
        const uint64_t entry = list[max(stay - 1, 0)];
        const int last = static_cast<int>(static_cast<uint32_t>(entry)) - (stay > 0 ? 0 : 1);
        if (threadIdx.x < ncta) {
          remote_store(&sh.cut.least, threadIdx.x, __float_as_uint(logit_of(entry)));
          remote_store(&sh.cut.last, threadIdx.x, static_cast<uint32_t>(last));
        }
        __syncwarp();
      }
      ptx::cluster_sync();
      cut = sh.cut;
    }
    if (threadIdx.x == 0) {  // (read before the last barrier)
      sh.list_count = 0;
      if (!listed) sh.put_count = 0;
    }
    __syncthreads();
  }

  // (a copy, so that the caller's row stays in registers)
  struct Rounds {
    Cut cut;
    unsigned uses;
  };
  template <bool BY_WEIGHT>
  __device__ static Rounds cut_by_rounds(Row r, uint64_t want, int b0, int b1);
};

// The same without a list, for bins of many tokens (ties, or logits beyond the bins' range): four rounds of eight bits of
// the key, then the ties by index.
template <typename T, bool KEEP>
template <bool BY_WEIGHT>
__device__ __noinline__ typename Row<T, KEEP>::Rounds Row<T, KEEP>::cut_by_rounds(Row r, uint64_t want, int b0, int b1) {
  Shared& sh = r.sh;
  uint32_t* rounds = r.rounds;
  uint32_t prefix = 0;
  uint64_t count_here = 0;
  for (int level = 24; level >= 0; level -= 8) {
    for (int i = threadIdx.x; i < 3 * 256; i += kThreads) rounds[i] = 0;
    if (threadIdx.x == 0) {
      sh.low = 255;
      sh.high = 0;
    }
    __syncthreads();
    r.each_kept([&](float l, int) {  // (from the CTAs' lists where these hold the bins' tokens)
      const uint32_t k = key_of(l);
      const int b = r.weight.bin(l);
      if (b < b0 || b > b1 || (level < 24 && (k ^ prefix) >> (level + 8) != 0)) return;
      const int digit = 255 - (k >> level & 255);  // the largest first
      atomicAdd(&rounds[digit], 1u);
      if (BY_WEIGHT) {
        add_to(rounds + 256, rounds + 512, digit, r.weigh(l));
      }
    });
    __syncthreads();
    ptx::cluster_sync();
    static_assert(kThreads == 256, "a thread a digit");
    uint64_t count = 0, mass = 0;  // every CTA adds up all of them
    for (uint32_t i = 0; i < r.ncta; ++i) {
      count += remote_load(&rounds[threadIdx.x], i);
      if (BY_WEIGHT)
        mass += remote_load(&rounds[256 + threadIdx.x], i) +
                (static_cast<uint64_t>(remote_load(&rounds[512 + threadIdx.x], i)) << 32);
    }
    const uint64_t mine = BY_WEIGHT ? mass : count, upto = warp_scan(mine);
    if (r.lane() == 31) sh.scratch[r.warp()] = upto;
    __syncthreads();
    uint64_t before = upto - mine;
    for (int i = 0; i < r.warp(); ++i) before += sh.scratch[i];
    // the digit where the sum reaches what is wanted, or the last that holds anything
    if (count > 0) {
      if (before + mine >= want) atomicMin(&sh.low, threadIdx.x);
      atomicMax(&sh.high, threadIdx.x);
    }
    __syncthreads();
    const int digit = min(sh.low, sh.high);
    __syncthreads();
    if (threadIdx.x == digit) {
      sh.scratch[0] = count;
      sh.scratch[1] = before;
    }
    __syncthreads();
    count_here = sh.scratch[0];
    want -= min(want, sh.scratch[1]);
    prefix |= static_cast<uint32_t>(255 - digit) << level;
    ptx::cluster_sync();  // all have read the counters
  }
  uint64_t stay = want;
  if (BY_WEIGHT) {
    const uint64_t w = r.weigh(of_key(prefix));
    stay = w > 0 ? (want + w - 1) / w : count_here;
  }
  const Cut old = r.cut;
  const float least = of_key(prefix);
  Cut cut{least, INT_MAX};
  if (stay < count_here) {
    uint32_t ties = 0;
    r.sweep([&](float l, int index) { ties += l == least && old.keeps(l, index); });
    r.exchange(ties, 0);
    uint64_t seen = r.before_cta().x;
    for (int i = 0; i < r.warp(); ++i) seen += sh.warp[0][i];
    if (seen < stay && seen + sh.warp[0][r.warp()] >= stay) {
      for (int y = r.warp() * r.run + r.lane(); y < (r.warp() + 1) * r.run; y += 32) {
        const int index = r.place0 + y - r.shift;
        const bool tie = r.at(y) == least && old.keeps(least, index);
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, tie);
        if (tie && seen + __popc(votes & (0xFFFFFFFFu >> (31 - r.lane()))) == stay)
          for (uint32_t i = 0; i < r.ncta; ++i) remote_store(&sh.tie, i, static_cast<uint32_t>(index));
        seen += __popc(votes);
      }
    } else if (stay == 0) {
      sh.tie = -1;
    }
    __syncwarp();
    ptx::cluster_sync();
    cut.last = sh.tie;
    __syncthreads();
  } else {
    cut.last = old.least == least ? old.last : INT_MAX;
  }
  return Rounds{cut, r.uses};
}

template <typename T, bool FILTER, bool KEEP>
__global__ void __launch_bounds__(kThreads, KEEP ? 3 : 4) sample_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  extern __shared__ __align__(16) char dynamic[];
  static_assert(sizeof(PowerTable) == kThreads * sizeof(uint4), "16 bytes a thread");
  reinterpret_cast<uint4*>(sh.power.at)[threadIdx.x] = reinterpret_cast<const uint4*>(kPowers.at)[threadIdx.x];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const long long line = blockIdx.x / ncta;
  const int req = static_cast<int>(line / a.rows_per);
  const T* src = static_cast<const T*>(a.logits) + req * a.stride0 + (line - static_cast<long long>(req) * a.rows_per) * a.stride1;
  using R = Row<T, KEEP>;

  R r{sh,
        reinterpret_cast<uint32_t*>(dynamic),
        reinterpret_cast<uint64_t*>(dynamic + kBins * 4),
        reinterpret_cast<uint64_t*>(dynamic + kBins * 4 + kOwn * 8),
        reinterpret_cast<uint32_t*>(dynamic + kBins * 4 + kOwn * 8 + kList * 8),
        reinterpret_cast<float*>(dynamic + kFixedBytes),
        src,
        ncta,
        ptx::cluster_ctarank(),
        0,
        static_cast<int>(reinterpret_cast<uintptr_t>(src) % 16 / sizeof(T)),  // place 0 lies on a 16-byte boundary
        0,
        a.slice / kWarps,
        a.up,
        Weight{sh.power.at, 0.f, 0.f, 0.f},
        Cut{-INFINITY, INT_MIN},  // (places before the row's first have indexes below 0)
        0,
        false};
  r.place0 = static_cast<int>(r.rank) * a.slice;
  r.end = a.vocab + r.shift;

  const float temperature = a.temperature != nullptr ? a.temperature[req] : 1.f;
  const int top_k = a.top_k != nullptr ? a.top_k[req] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[req] : 1.f;
  const float min_p = a.min_p != nullptr && a.min_p[req] > 0.f ? fminf(a.min_p[req], 1.f) : 0.f;
  const bool greedy = !(temperature > 0.f);
  const bool by_count = top_k > 0 && top_k < a.vocab, by_weight = top_p < 1.f;

  // ---------------- the row, and its maximum
  float mx = -INFINITY;
  constexpr int kVec = R::kVec, kAhead = 32 / kVec;
  for (int y0 = tid * kVec; y0 < a.slice; y0 += kThreads * kVec * kAhead) {
    uint4 words[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (y0 + kThreads * kVec * k < a.slice) words[k] = r.fetch(r.place0 + y0 + kThreads * kVec * k);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int y = y0 + kThreads * kVec * k;
      if (y >= a.slice) break;
      float v[kVec];
      R::decode(words[k], v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) mx = fmaxf(mx, v[i]);
      if (KEEP) {
#pragma unroll
        for (int i = 0; i < kVec; i += 4)
          *reinterpret_cast<float4*>(r.logit + y + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
  }
  if (!greedy && (by_count || by_weight))
    for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(r.hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    sh.put_count = sh.list_count = 0;
    sh.tie = INT_MAX;
  }
  if (tid < 3 * kWindow) sh.window[0][tid] = 0;
  static_assert(3 * kWindow <= kThreads && kWindow == 32, "a lane a bin");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  float* warp_max = reinterpret_cast<float*>(sh.scratch);
  if (lane == 0) warp_max[warp] = mx;
  __syncthreads();
  ptx::cluster_sync();  // every CTA of the cluster runs, and its words are set
  if (tid < static_cast<int>(ncta)) {
    float m = warp_max[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) m = fmaxf(m, warp_max[i]);
    remote_store(&sh.max[r.rank], tid, __float_as_uint(m));
  }
  __syncwarp();
  ptx::cluster_sync();
  mx = sh.max[0];
  for (uint32_t i = 1; i < ncta; ++i) mx = fmaxf(mx, sh.max[i]);

  // ---------------- which tokens are kept, and their weight
  const double c = kLog2e / static_cast<double>(temperature);
  r.weight.max = mx;
  r.weight.ch = fminf(static_cast<float>(c), 3.4028234664e38f);
  r.weight.cl = c > 3e38 ? 0.f : static_cast<float>(c - static_cast<double>(r.weight.ch));
  uint64_t total = 0;
  if (mx == -INFINITY) {
    // none
  } else if (greedy) {
    int lowest = INT_MAX;
    r.sweep([&](float l, int index) {
      if (l == mx) lowest = min(lowest, index);
    });
    lowest = __reduce_min_sync(0xFFFFFFFFu, lowest);
    if (lane == 0 && lowest != INT_MAX)
      for (uint32_t i = 0; i < ncta; ++i) remote_min(&sh.tie, i, lowest);
    __syncwarp();
    ptx::cluster_sync();
    r.cut = Cut{mx, sh.tie};
    total = 1;
  } else {
    if (min_p > 0.f) {  // l >= max + T ln min_p, the bound rounded up to the next float
      const double least = static_cast<double>(mx) + static_cast<double>(temperature) * log(static_cast<double>(min_p));
      if (least > -INFINITY) r.cut.least = nextafterf(__double2float_ru(least), -INFINITY);
    }
    uint64_t kept = 0;  // this thread's
    // Without a bound every logit is weighed, so that a lane's are not branches of their own (and -inf is taken out: behind
    // an infinite temperature its weight is 1).
    auto weigh = [&](float l) {
      const uint64_t w = r.weigh(l);
      return l > -INFINITY ? w : 0;
    };
    const bool late = by_weight && !by_count && !(min_p > 0.f);  // weighed when the cut's bins are known
    if (late) {
      r.sweep([&](float l, int) {
        if (l > -INFINITY) atomicAdd(&r.hist[r.weight.bin(l)], 1u);
      });
    } else if (min_p > 0.f || by_count) {
      r.sweep_kept([&](float l, int) {
        if (by_count || by_weight) atomicAdd(&r.hist[r.weight.bin(l)], 1u);
        if (!by_count) kept += r.weigh(l);
      });
    } else {
      r.sweep([&](float l, int) { kept += weigh(l); });
    }
    int k_bin = kBins;
    uint32_t k_rest = 0;  // what is kept of it
    if (by_count || by_weight) {
      ptx::cluster_sync();
      const int share = kBins / ncta;
      for (int b = r.rank * share + tid; b < static_cast<int>(r.rank + 1) * share; b += kThreads) {
        uint32_t n = 0;
        for (uint32_t i = 0; i < ncta; ++i) n += remote_load(&r.hist[b], i);
        r.hist[b] = n;  // (nobody else reads these bins)
      }
      __syncthreads();
    }
    if (by_count) {
      const uint64_t want = top_k;
      const auto all = r.find_bins([&](int b) { return typename R::Pair{r.hist[b], 0}; },
                                   [&](typename R::Pair, int i, typename R::Pair upto) { return i == 0 && upto.x >= want; });
      if (want < all.x) {
        k_bin = sh.bin[0];
        k_rest = static_cast<uint32_t>(want - sh.before);
        const uint32_t m = sh.high;
        const bool all_listed = sh.before + m <= kOwn;
        const float from = r.weight.least_of(k_bin), to = all_listed ? INFINITY : r.weight.least_of(k_bin - 1);
        if (all_listed || m <= kList)
          r.sweep_kept([&](float l, int index) {
            if (l >= from && l < to) r.put(l, index);
          });
        __syncthreads();
        ptx::cluster_sync();
        r.listed = all_listed;
        r.template cut_at<false>(k_rest, k_bin, k_bin, m, true);
      }
      kept = r.kept_weight([](float) { return true; });
    }
    if (!late) total = r.exchange(kept, 0).x;
    if (by_weight) {
      // The most and the least weight that each bin can hold bound the bins that the cut can fall into: with X up to a bin and Y
      // behind it, it lies no further where X >= p (X + Y), or (1 - p) X >= p Y, for the least X and the most Y, and
      // no earlier where not even the most X and the least Y fulfil that.  (The total does not have to be known for that.)
      auto bounds = [&](int b) {
        const uint64_t n = b < k_bin ? r.hist[b] : (b == k_bin ? k_rest : 0);
        // (a bin's steps are rounded: it reaches half a step of 2^-10 to either side)
        constexpr float kSpan = 1.f / (1 << (10 - kBinShift)), kHalf = 1.f / 2048.f;
        const float most = exp2f(kMassBits + kHalf - b * kSpan), least = exp2f(kMassBits + kHalf - (b + 1) * kSpan);
        return typename R::Pair{n * (static_cast<uint64_t>(most * 1.00001f) + 1),
                                b + 1 < kBins ? n * static_cast<uint64_t>(least * 0.99999f) : 0};
      };
      const uint64_t p = __float2ull_rz(fmaxf(top_p, 0.f) * 18446744073709551616.f), rest = ~p;  // 2^-64
      r.find_bins(bounds, [&](typename R::Pair all, int i, typename R::Pair upto) {  // (3: what rounding down may lose)
        if (upto.x == 0) return false;
        if (i == 0) return __umul64hi(upto.x, rest) + __umul64hi(upto.y, p) + 3 >= __umul64hi(all.y, p);
        return __umul64hi(upto.y, rest) + __umul64hi(upto.x, p) >= __umul64hi(all.x, p) + 3;
      });
      const int first = sh.bin[0], last = max(first, sh.bin[1]);
      const bool narrow = last - first < kWindow;
      // The weight before the window, the window's by bins, and its tokens; with what lies before them where that is little.
      bool list_now = false;
      if (!r.listed) {
        const int share = kBins / ncta;
        uint64_t tokens = 0;
        for (int b = r.rank * share + tid; b < static_cast<int>(r.rank + 1) * share; b += kThreads)
          if (b <= last) tokens += r.hist[b];
        list_now = r.exchange(tokens, 0).x <= kOwn;
      }
      if (r.listed && tid < 2 * kWarps) sh.runs[0][tid] = 0;
      __syncthreads();
      const float from = r.weight.least_of(last), before = r.weight.least_of(first - 1);
      auto in_window = [&](float l, uint64_t w) {
        const int b = r.weight.bin(l) - first;
        atomicAdd(&sh.window[0][b], 1u);
        R::add_to(sh.window[1], sh.window[2], b, w);
      };
      kept = 0;
      uint64_t weighed = 0;  // (late) this thread's of all tokens
      if (late) {
        r.sweep([&](float l, int index) {
          const uint64_t w = weigh(l);
          const bool above = l >= before;
          weighed += w;
          kept += above ? w : 0;
          if (l >= from && (list_now || (narrow && !above))) {
            r.put(l, index);
            if (narrow && !above) in_window(l, w);
          }
        });
      } else if (!r.listed && !list_now) {
        kept = r.packed_weight(from, [&](float l) { return l < before; }, [&](float l, int index) {
          if (!narrow) return;
          r.put(l, index);
          in_window(l, r.weigh(l));
        });
      } else {
        r.each_kept([&](float l, int index) {
          if (l < from) return;
          if (list_now) r.put(l, index);
          if (l < before) {
            if (narrow) in_window(l, r.weigh(l));
          } else if (r.listed) {
            R::add_to(sh.runs[0], sh.runs[1], (index + r.shift - r.place0) / r.run, r.weigh(l));
          } else {
            kept += r.weigh(l);
          }
        });
      }
      if (r.listed) {
        __syncthreads();
        kept = lane == 0 ? sh.runs[0][warp] | static_cast<uint64_t>(sh.runs[1][warp]) << 32 : 0;
      }
      const auto sums = r.exchange(kept, weighed);
      if (late) total = sums.y;
      uint64_t above = sums.x;
      const double part = static_cast<double>(fmaxf(top_p, 0.f)) * static_cast<double>(total);
      const uint64_t want = max(static_cast<uint64_t>(ceil(part)), static_cast<uint64_t>(1));
      r.listed |= list_now;
      int at = first;
      uint32_t m = 0;
      bool room = true;
      if (narrow) {  // the bin that the cut falls into, by every CTA alike: warp 0 adds up the cluster's windows
        if (warp == 0) {
          uint64_t sum = 0;
          uint32_t n = 0;
          for (uint32_t i = 0; i < ncta; ++i) {
            n += remote_load(&sh.window[0][lane], i);
            sum += remote_load(&sh.window[1][lane], i) + (static_cast<uint64_t>(remote_load(&sh.window[2][lane], i)) << 32);
          }
          const bool full = lane < static_cast<int>(ncta) && remote_load(&sh.put_count, lane) > kOwn;
          const uint64_t upto = above + warp_scan(sum);
          const uint32_t hit = __ballot_sync(0xFFFFFFFFu, n > 0 && upto >= want), any = __ballot_sync(0xFFFFFFFFu, n > 0);
          const int pick = hit != 0 ? __ffs(hit) - 1 : (any != 0 ? 31 - __clz(any) : 0);
          const bool crowded = __any_sync(0xFFFFFFFFu, full);
          if (lane == pick) {
            sh.low = crowded ? -1 : pick;
            sh.high = static_cast<int>(n);
            sh.scratch[0] = upto - sum;
          }
        }
        __syncthreads();
        room = sh.low >= 0;
        m = sh.high;
        if (room) {
          at = first + sh.low;
          above = sh.scratch[0];
        }
        ptx::cluster_sync();  // (all have read the windows before a list is gathered and the counts are reset)
      }
      const bool whole = r.listed;
      r.listed |= narrow && room && m > 0;  // (of what lies behind `before`, all that may be kept)
      const int to = narrow && room ? at : last;
      if (!narrow || !room || m > 0) r.template cut_at<true>(want - min(want, above), at, to, m, narrow && room);
      kept += r.kept_weight([&](float l) { return l < before; });
      r.listed = whole;
      total = r.exchange(kept, 0).x;
    }
  }

  if (FILTER) {
    const float inv = static_cast<float>(exp2(static_cast<double>(a.up)) / static_cast<double>(total));
    const int lo = max(r.place0 - r.shift, 0), hi = min(r.place0 + a.slice - r.shift, a.vocab);
    float* out = a.probs + line * a.vocab;
    auto prob = [&](float l, int x) {
      if (!r.cut.keeps(l, x)) return 0.f;
      int n;
      const uint32_t m = r.weight(l, n);
      if (n > 160) return 0.f;
      return __uint2float_rn(m) * inv * __int_as_float((127 - n / 2) << 23) * __int_as_float((127 - n + n / 2) << 23);
    };
    // few tokens: zeros, then the tokens' own
    const bool sparse = total == 0 || greedy || r.listed;
    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(out) / 4 % 4);  // out - lead lies on 16 bytes
    for (int x = (lo + lead) / 4 * 4 - lead + tid * 4; x < hi; x += kThreads * 4) {
      if (x >= lo && x + 4 <= hi) {
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!sparse) {
          const int y = x + r.shift - r.place0;
          p = make_float4(prob(r.at(y), x), prob(r.at(y + 1), x + 1), prob(r.at(y + 2), x + 2), prob(r.at(y + 3), x + 3));
        }
        __stcs(reinterpret_cast<float4*>(out + x), p);
      } else {
        for (int i = max(x, lo); i < min(x + 4, hi); ++i) out[i] = sparse ? 0.f : prob(r.at(i + r.shift - r.place0), i);
      }
    }
    if (sparse && total != 0) {
      __syncthreads();
      if (greedy) {
        if (tid == 0 && r.cut.last >= lo && r.cut.last < hi) out[r.cut.last] = 1.f;
      } else {
        r.each_kept([&](float l, int x) { out[x] = prob(l, x); });
      }
    }
  } else if (total == 0 || greedy) {
    if (r.rank == 0 && tid == 0) a.tokens[line] = total == 0 ? -1 : r.cut.last;
  } else {
    // the lowest token whose running sum passes t: its CTA, its warp's run, then itself
    const float u = a.u[req];
    const uint64_t t = u >= 1.f ? total - 1
                       : (u > 0.f ? min(static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total)), total - 1) : 0);
    const uint64_t* ctas = sh.sums[(r.uses - 1) & 1u][0];
    uint64_t before = 0;
    uint32_t owner = 0;
    while (owner + 1 < ncta && before + ctas[owner] <= t) before += ctas[owner++];
    if (owner == r.rank) {
      int w = 0;
      while (w + 1 < kWarps && before + sh.warp[0][w] <= t) before += sh.warp[0][w++];
      for (int base = w * r.run; base < (w + 1) * r.run; base += kThreads) {
        const int y = base + tid, index = r.place0 + y - r.shift;
        const float l = y < (w + 1) * r.run ? r.at(y) : -INFINITY;
        const uint64_t mine = r.cut.keeps(l, index) ? r.weigh(l) : 0, upto = warp_scan(mine);
        if (lane == 31) sh.scratch[warp] = upto;
        __syncthreads();
        uint64_t run = before + upto;
        for (int i = 0; i < warp; ++i) run += sh.scratch[i];
        if (run > t && run - mine <= t) a.tokens[line] = index;
        for (int i = 0; i < kWarps; ++i) before += sh.scratch[i];
        __syncthreads();
        if (before > t) break;
      }
    }
  }
  __syncwarp();
  ptx::cluster_sync();  // no CTA leaves while another may still read or write its shared memory
}

// Per device, once for each kernel: shared memory beyond 48 KB and clusters of more than eight CTAs.
template <typename T, bool FILTER, bool KEEP>
bool prepare_kernel() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (ready.load() & bit) return true;
  const auto kernel = sample_kernel<T, FILTER, KEEP>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFixedBytes + kKeepSlice * 4) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return false;
  ready.fetch_or(bit);
  return true;
}

template <typename T, bool FILTER, bool KEEP>
qnre_status_t launch(const SampleArgs& a, int64_t rows, unsigned cluster, qnre_stream_t stream) {
  if (!prepare_kernel<T, FILTER, KEEP>()) return QNRE_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kFixedBytes + (KEEP ? a.slice * 4 : 0);
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
  return from_cuda(cudaLaunchKernelEx(&cfg, sample_kernel<T, FILTER, KEEP>, a));
}

template <typename T, bool FILTER>
qnre_status_t choose(SampleArgs a, int64_t rows, qnre_stream_t stream) {
  // As many CTAs a row as the machine holds at once, while each keeps a grain of places.
  const int64_t places = a.vocab + 16 / sizeof(T) - 1;
  unsigned cluster = kMaxCluster;
  while (cluster > 1 && (rows * cluster > kResident || places <= static_cast<int64_t>(cluster / 2) * kGrain)) cluster /= 2;
  // Rows that are read again should fit in L2 together.
  while (cluster < kMaxCluster && places > static_cast<int64_t>(cluster) * kKeepSlice &&
         std::min<int64_t>(kResident / cluster, rows) * places * static_cast<int64_t>(sizeof(T)) > kInL2)
    cluster *= 2;
  a.slice = static_cast<int>(((places + cluster - 1) / cluster + kGrain - 1) / kGrain * kGrain);
  a.up = 31;  // sums of V weights stay below 2^63
  while ((int64_t{1} << (31 - a.up)) < a.vocab) --a.up;
  return a.slice <= kKeepSlice ? launch<T, FILTER, true>(a, rows, cluster, stream)
                               : launch<T, FILTER, false>(a, rows, cluster, stream);
}

template <bool FILTER>
qnre_status_t run(const void* logits, int64_t stride0, int64_t stride1, int32_t dtype, int n, int nodes, int64_t vocab,
                  const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                  void* out, uint64_t out_bytes, qnre_stream_t stream) {
  if (n < 0 || nodes < 1 || vocab < 1 || stride0 < 0 || stride1 < 0) return QNRE_ERR_INVALID_ARG;
  const int size = dtype_size(dtype);
  if (size == 0) return QNRE_ERR_UNSUPPORTED;
  if (vocab > QNRE_MAX_VOCAB || n > (1 << 20) || nodes > QNRE_MAX_NODES || stride0 > (int64_t{1} << 40) ||
      stride1 > (int64_t{1} << 40))
    return QNRE_ERR_CAPACITY;
  if (n == 0) return QNRE_OK;
  if (logits == nullptr || out == nullptr || (!FILTER && u == nullptr)) return QNRE_ERR_INVALID_ARG;
  if (!aligned(logits, size)) return QNRE_ERR_ALIGNMENT;
  const void* words[] = {temperature, top_k, top_p, min_p, u, out};
  for (const void* p : words)
    if (!aligned(p, 4)) return QNRE_ERR_ALIGNMENT;
  const ByteRange w = span(out, out_bytes);
  if (overlaps(w, span(logits, (static_cast<uint64_t>(n - 1) * stride0 + static_cast<uint64_t>(nodes - 1) * stride1 + vocab) * size)))
    return QNRE_ERR_ALIAS;
  for (int i = 0; i < 5; ++i)
    if (words[i] != nullptr && overlaps(w, span(words[i], static_cast<uint64_t>(n) * 4))) return QNRE_ERR_ALIAS;
  SampleArgs a{logits, stride0, stride1, temperature, top_p, min_p, u, top_k,
               FILTER ? nullptr : static_cast<int32_t*>(out), FILTER ? static_cast<float*>(out) : nullptr, nodes,
               static_cast<int>(vocab), 0, 0};
  const int64_t rows = static_cast<int64_t>(n) * nodes;
  switch (dtype) {
    case QNRE_DTYPE_FP32: return choose<float, FILTER>(a, rows, stream);
    case QNRE_DTYPE_BF16: return choose<__nv_bfloat16, FILTER>(a, rows, stream);
    default: return choose<__half, FILTER>(a, rows, stream);
  }
}

}  // namespace

extern "C" {

qnre_status_t qnre_sample(const void* logits, int64_t stride, int32_t dtype, int n, int64_t vocab, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                          qnre_stream_t stream) {
  return run<false>(logits, stride, 0, dtype, n, 1, vocab, temperature, top_k, top_p, min_p, u, tokens,
                    static_cast<uint64_t>(std::max(n, 0)) * 4, stream);
}

qnre_status_t qnre_filter_probs(const void* logits, int64_t stride0, int64_t stride1, int32_t dtype, int n, int nodes,
                                int64_t vocab, const float* temperature, const int32_t* top_k, const float* top_p,
                                const float* min_p, float* probs, qnre_stream_t stream) {
  const uint64_t cells = static_cast<uint64_t>(std::max(n, 0)) * std::max(nodes, 0) * std::max<int64_t>(vocab, 0);
  return run<true>(logits, stride0, stride1, dtype, n, nodes, vocab, temperature, top_k, top_p, min_p, nullptr, probs,
                   cells * 4, stream);
}

}  // extern "C"
