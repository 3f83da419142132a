// sample.cu -- tokens, or filtered probabilities, from logits: temperature, top-k, top-p and min-p.
//
//   w_x = exp((l_x - max l) / T);  order: by logit, then by index
//   kept: w_x >= min_p; of those the top_k first; of those the ones before which less than top_p of their weight lies
//   token = lowest x whose running sum of kept weights (by index) exceeds u times their total
//
// A cluster of up to 16 CTAs takes one row and holds it in shared memory, so a row is read from HBM once whatever
// passes follow.  Nothing is sorted but the few tokens around a cut:
//
//   max        while the row arrives; every CTA learns it through the cluster's shared memory,
//   histogram  counts over 4096 bins of (max - l) / T, which orders tokens coarsely; each CTA adds up its share of the
//              bins over the cluster.  The bin of the top_k-th token is exact from the counts.  For top_p the counts
//              bound the weight above each bin from both sides (a bin spans a factor e^(1/256)), so the tokens that the
//              cut can fall on lie in a window of a few bins,
//   cut        the tokens of that bin or window go to the first CTA's list, which sorts them and finds the last one kept;
//              lists that overflow (ties, logits out of the bins' range) are cut by four rounds of eight key bits,
//   draw       the kept weight by warps' runs of places; the run that holds the number is added up place by place.
//
// Numbers.  A token is right only if no sum is wrong by more than its distance from a border, and with 10^5 borders
// 32-bit sums would miss one draw in a hundred.  So weights are integers of 2^-(63 - ceil log2 V) of the largest: the
// exponent is formed as a pair of floats, its leading ten binary places taken from a table of 2^(-j/1024) and the rest by
// a cubic (Weight; 2^-42 relative at worst, 2^-44 near the largest, 40 instructions, where fp64 runs at a 64th of the rate).  Integer sums
// do not depend on their order, so counters and lists filled in any order change no result.
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
constexpr float kRange = 16.f;           // (max - l) / T that the bins cover; the last holds all beyond
constexpr int kList = 1024;
constexpr int kMaxSlice = 49152;         // places of a CTA
static_assert(kMaxSlice * kMaxCluster == QNRE_MAX_VOCAB, "the largest row");
constexpr int kMassBits = 40;            // of the histogram's bounds on weights
constexpr int kFixedBytes = kBins * 4 + kList * 8 + 3 * 256 * 4;  // shared memory before the row
constexpr double kLog2e = 1.4426950408889634074;
constexpr float kBinLog2 = kRange * 1.44269504f / kBins;  // a bin's span in powers of two

struct SampleArgs {
  const void* logits;
  long long stride0, stride1;  // elements between requests, between a request's rows
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
  int rows_per, vocab, slice, scale;  // rows of a request; places of a CTA; binary places of a weight
};

// 2^(-j/1024) in units of 2^-63, from 2^(-i/32) and 2^(-i/1024).
struct PowerTable {
  uint64_t at[1024];
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
  for (int j = 0; j < 1024; ++j) t.at[j] = product63(kCoarse[j / 32], kFine[j % 32]);
  return t;
}
__device__ const PowerTable kPowers = make_powers();

// A row's scale: weights are 2^(-y), y = (max - l) c, c = log2(e) / T as a pair of floats.
struct Weight {
  float max, ch, cl;

  // y = whole + fraction; false where the weight is below 2^-`limit`.  The value is mantissa 2^-(63 + whole).
  __device__ __forceinline__ bool operator()(float l, float limit, uint64_t& mantissa, int& whole) const {
    mantissa = 1ull << 63;
    whole = 0;
    if (l == max) return true;
    const float d = max - l, back = d - max, err = (max - (d - back)) - (l + back);  // d + err = max - l
    const float p = d * ch;
    if (!(p < limit)) return false;  // (NaN, too: an infinite distance times c = 0)
    const float e = fmaf(d, ch, -p) + fmaf(d, cl, err * ch);
    whole = static_cast<int>(p);
    const float places = (p - static_cast<float>(whole)) * 8388608.f;  // of 2^-23
    const int lead = static_cast<int>(places);
    const float rest = (places - static_cast<float>(lead)) + e * 8388608.f;
    // y mod 2^-10: 13 of those places and the rest, which may be a little below 0 or above 1
    const int low = lead & 8191, part = __float2int_rn(rest * 16777216.f);                     // 2^-23, 2^-47
    const float t = (static_cast<float>(low) + rest) * 8.262958294867817e-08f;                 // ln 2 2^-23
    const int curve = __float2int_rn(t * t * fmaf(t, -0.16666667f, 0.5f) * 140737488355328.f);  // t^2/2 - t^3/6, 2^-47
    // 1 - e^-t in units of 2^-64, with ln 2 to 2^-41 of a place of 2^-23 and to 2^-31 of the rest
    const long long loss = low * 1524246769572ll + (static_cast<long long>(part) * 1488522236 >> 14) - (static_cast<long long>(curve) << 17);
    const uint64_t power = __ldg(&kPowers.at[lead >> 13]);
    mantissa = loss >= 0 ? power - __umul64hi(power, static_cast<uint64_t>(loss))
                         : power + __umul64hi(power, static_cast<uint64_t>(-loss));
    return true;
  }
  __device__ __forceinline__ uint64_t fixed(float l, int scale) const {
    uint64_t m;
    int whole;
    if (!(*this)(l, 64.f, m, whole)) return 0;
    const int shift = whole + 63 - scale;
    return shift > 63 ? 0 : (m + (1ull << (shift - 1))) >> shift;
  }
};

// Logits as integers of the same order (larger logit, larger key); both zeros have one key.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// What a row keeps: larger keys than `key`, and of that key the tokens up to `last`.
struct Cut {
  uint32_t key;
  int last;
  __device__ __forceinline__ bool keeps(uint32_t k, int index) const { return k > key || (k == key && index <= last); }
};

struct Shared {
  uint64_t sums[2][2][kMaxCluster];  // two sums of each of the cluster's CTAs, two uses in turn
  uint64_t warp[2][kWarps];
  uint64_t scratch[kWarps];
  float max[kMaxCluster];
  uint64_t before;                   // what lies before the first bin found
  Cut cut;
  uint32_t list_count;
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
__device__ __forceinline__ uint32_t remote_add(uint32_t* p, uint32_t rank, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(in_cta(p, rank)), "r"(v) : "memory");
  return old;
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
struct Row {
  Shared& sh;
  uint32_t* hist;    // [kBins]
  uint64_t* list;    // [kList]: (~key, index); the first CTA's
  uint32_t* rounds;  // [3][256]: counts, weights' low and high words
  float* logit;      // [slice]
  uint32_t ncta, rank;
  int place0, shift, run, scale;  // places are index + shift; `run` of them to a warp, in order
  float bin_scale;
  Weight weight;
  Cut cut;
  unsigned uses;

  __device__ __forceinline__ static int warp() { return threadIdx.x / 32; }
  __device__ __forceinline__ static int lane() { return threadIdx.x % 32; }

  __device__ __forceinline__ uint64_t weigh(float l) const { return weight.fixed(l, scale); }
  __device__ __forceinline__ int bin_of(float l) const {
    return min(static_cast<int>((weight.max - l) * bin_scale), kBins - 1);
  }

  // f(logit, index) for every place of this warp's run.
  template <typename F>
  __device__ __forceinline__ void sweep(F f) const {
    for (int y = warp() * run + lane() * 4; y < (warp() + 1) * run; y += 128) {
      const float4 v = *reinterpret_cast<const float4*>(logit + y);
      const int index = place0 + y - shift;
      f(v.x, index);
      f(v.y, index + 1);
      f(v.z, index + 2);
      f(v.w, index + 3);
    }
  }
  template <typename F>
  __device__ __forceinline__ void sweep_kept(F f) const {
    sweep([&](float l, int index) {
      if (cut.keeps(key_of(l), index)) f(l, index);
    });
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

  // sh.bin[0], sh.bin[1]: the first bins whose running sums of f(bin).x and .y reach the targets (the last bin where
  // none does), sh.before the sum of x before the first.  Bins lie in the CTAs' histograms by equal shares.  Returns the sums.
  template <typename F>
  __device__ Pair find_bins(F f, uint64_t target_x, uint64_t target_y) {
    const int share = kBins / ncta, per = share / kThreads, b0 = rank * share + threadIdx.x * per;
    Pair own{0, 0};
    for (int i = 0; i < per; ++i) {
      const Pair v = f(b0 + i);
      own.x += v.x;
      own.y += v.y;
    }
    if (threadIdx.x == 0) sh.bin[0] = sh.bin[1] = kBins - 1;
    const uint64_t sx = warp_scan(own.x), sy = warp_scan(own.y);
    const Pair all = exchange(own.x, own.y);
    Pair before = before_cta();
    before.x += sx - own.x;
    before.y += sy - own.y;
    for (int i = 0; i < warp(); ++i) {
      before.x += sh.warp[0][i];
      before.y += sh.warp[1][i];
    }
    const bool here_x = before.x < target_x && before.x + own.x >= target_x;
    const bool here_y = before.y < target_y && before.y + own.y >= target_y;
    if (here_x || here_y) {
      bool seek_x = here_x, seek_y = here_y;
      for (int i = 0; i < per; ++i) {
        const Pair v = f(b0 + i);
        if (seek_x && before.x + v.x >= target_x) {
          seek_x = false;
          for (uint32_t r = 0; r < ncta; ++r) {
            remote_store(&sh.bin[0], r, b0 + i);
            remote_store64(&sh.before, r, before.x);
          }
        }
        if (seek_y && before.y + v.y >= target_y) {
          seek_y = false;
          for (uint32_t r = 0; r < ncta; ++r) remote_store(&sh.bin[1], r, b0 + i);
        }
        before.x += v.x;
        before.y += v.y;
      }
    }
    __syncwarp();
    ptx::cluster_sync();
    return all;
  }

  // Kept tokens go to the first CTA's list; only the first kList find room.
  __device__ __forceinline__ void put(float l, int index) {
    const uint32_t at = remote_add(&sh.list_count, 0, 1);
    if (at < kList)
      remote_store64(&list[at], 0, static_cast<uint64_t>(~key_of(l)) << 32 | static_cast<uint32_t>(index));
  }
  __device__ __forceinline__ static float logit_of(uint64_t entry) { return of_key(~static_cast<uint32_t>(entry >> 32)); }

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

  // Cuts off what lies in bins [b0, b1] behind the first tokens that make up `want`, counted as tokens or by weight.
  // The list holds the kept tokens of those bins (after a cluster barrier).
  template <bool BY_WEIGHT>
  __device__ void cut_at(uint64_t want, int b0, int b1) {
    const uint32_t m = remote_load(&sh.list_count, 0);
    if (m > kList) {
      const Rounds found = cut_by_rounds<BY_WEIGHT>(*this, want, b0, b1);
      cut = found.cut;
      uses = found.uses;
    } else if (m > 0) {
      if (rank == 0) {
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
          remote_store(&sh.cut.key, threadIdx.x, ~static_cast<uint32_t>(entry >> 32));
          remote_store(&sh.cut.last, threadIdx.x, static_cast<uint32_t>(last));
        }
        __syncwarp();
      }
      ptx::cluster_sync();
      cut = sh.cut;
    }
    if (threadIdx.x == 0) sh.list_count = 0;  // (all read it before the last barrier)
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
template <bool BY_WEIGHT>
__device__ __noinline__ Row::Rounds Row::cut_by_rounds(Row r, uint64_t want, int b0, int b1) {
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
    r.sweep_kept([&](float l, int) {
      const uint32_t k = key_of(l);
      const int b = r.bin_of(l);
      if (b < b0 || b > b1 || (level < 24 && (k ^ prefix) >> (level + 8) != 0)) return;
      const int digit = 255 - (k >> level & 255);  // the largest first
      atomicAdd(&rounds[digit], 1u);
      if (BY_WEIGHT) {
        const uint64_t w = r.weigh(l);
        const uint32_t part = static_cast<uint32_t>(w), old = atomicAdd(&rounds[256 + digit], part);
        atomicAdd(&rounds[512 + digit], static_cast<uint32_t>(w >> 32) + (old + part < old ? 1u : 0u));
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
  Cut cut{prefix, INT_MAX};
  if (stay < count_here) {
    uint32_t ties = 0;
    r.sweep([&](float l, int index) { ties += key_of(l) == prefix && old.keeps(prefix, index); });
    r.exchange(ties, 0);
    uint64_t seen = r.before_cta().x;
    for (int i = 0; i < r.warp(); ++i) seen += sh.warp[0][i];
    if (seen < stay && seen + sh.warp[0][r.warp()] >= stay) {
      for (int y = r.warp() * r.run + r.lane(); y < (r.warp() + 1) * r.run; y += 32) {
        const int index = r.place0 + y - r.shift;
        const bool tie = key_of(r.logit[y]) == prefix && old.keeps(prefix, index);
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
    cut.last = old.key == prefix ? old.last : INT_MAX;
  }
  return Rounds{cut, r.uses};
}

template <typename T, bool FILTER>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  extern __shared__ __align__(16) char dynamic[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const long long line = blockIdx.x / ncta;
  const int req = static_cast<int>(line / a.rows_per);
  const T* src = static_cast<const T*>(a.logits) + req * a.stride0 + (line - static_cast<long long>(req) * a.rows_per) * a.stride1;
  constexpr int kVec = 16 / sizeof(T);

  Row r{sh,
        reinterpret_cast<uint32_t*>(dynamic),
        reinterpret_cast<uint64_t*>(dynamic + kBins * 4),
        reinterpret_cast<uint32_t*>(dynamic + kBins * 4 + kList * 8),
        reinterpret_cast<float*>(dynamic + kFixedBytes),
        ncta,
        ptx::cluster_ctarank(),
        0,
        static_cast<int>(reinterpret_cast<uintptr_t>(src) % 16 / sizeof(T)),  // place 0 lies on a 16-byte boundary
        a.slice / kWarps,
        a.scale,
        0.f,
        Weight{0.f, 0.f, 0.f},
        Cut{0, 0},
        0};
  r.place0 = static_cast<int>(r.rank) * a.slice;
  const int end = a.vocab + r.shift;

  const float temperature = a.temperature != nullptr ? a.temperature[req] : 1.f;
  const int top_k = a.top_k != nullptr ? a.top_k[req] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[req] : 1.f;
  const float min_p = a.min_p != nullptr ? fminf(a.min_p[req], 1.f) : 0.f;
  const bool greedy = !(temperature > 0.f);
  const bool by_count = top_k > 0 && top_k < a.vocab, by_weight = top_p < 1.f;

  // ---------------- the row, and its maximum
  float mx = -INFINITY;
  for (int y = tid * kVec; y < a.slice; y += kThreads * kVec) {
    const int place = r.place0 + y;
    float v[kVec];
    if (place >= r.shift && place + kVec <= end) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(src + (place - r.shift)));
      const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = to_float(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[i] = place + i >= r.shift && place + i < end ? to_float(src[place + i - r.shift]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (v[i] != v[i]) v[i] = -INFINITY;  // a NaN counts as left out
      mx = fmaxf(mx, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kVec; i += 4)
      *reinterpret_cast<float4*>(r.logit + y + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
  if (!greedy && (by_count || by_weight))
    for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(r.hist)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    sh.list_count = 0;
    sh.tie = INT_MAX;
  }
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
  r.weight.ch = static_cast<float>(c);
  r.weight.cl = isinf(r.weight.ch) ? 0.f : static_cast<float>(c - static_cast<double>(r.weight.ch));
  r.bin_scale = kBins / (kRange * temperature);
  r.cut = Cut{key_of(-INFINITY), -1};
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
    r.cut = Cut{key_of(mx), sh.tie};
    total = 1;
  } else {
    if (min_p > 0.f) {  // l >= max + T ln min_p, the bound rounded up to the next float
      const double least = static_cast<double>(mx) + static_cast<double>(temperature) * log(static_cast<double>(min_p));
      if (least > -INFINITY) r.cut.key = max(r.cut.key, key_of(__double2float_ru(least)) - 1);
    }
    uint64_t kept = 0;  // this thread's
    r.sweep_kept([&](float l, int) {
      if (by_count || by_weight) atomicAdd(&r.hist[r.bin_of(l)], 1u);
      if (!by_count) kept += r.weigh(l);
    });
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
      const auto all = r.find_bins([&](int b) { return Row::Pair{r.hist[b], 0}; }, want, ~0ull);
      if (want < all.x) {
        k_bin = sh.bin[0];
        k_rest = static_cast<uint32_t>(want - sh.before);
        r.sweep_kept([&](float l, int index) {
          if (r.bin_of(l) == k_bin) r.put(l, index);
        });
        ptx::cluster_sync();
        r.template cut_at<false>(k_rest, k_bin, k_bin);
      }
      r.sweep_kept([&](float l, int) { kept += r.weigh(l); });
    }
    total = r.exchange(kept, 0).x;
    if (by_weight) {
      // The most and the least weight that each bin can hold bound the bins that the cut can fall into.
      const double part = static_cast<double>(fmaxf(top_p, 0.f)) * static_cast<double>(total);
      const double coarse = part * exp2(static_cast<double>(kMassBits - a.scale));
      auto bounds = [&](int b) {
        const uint64_t n = b < k_bin ? r.hist[b] : (b == k_bin ? k_rest : 0);
        const float most = exp2f(kMassBits - b * kBinLog2), least = exp2f(kMassBits - (b + 1) * kBinLog2);
        return Row::Pair{n * (static_cast<uint64_t>(most * 1.00001f) + 1),
                         b + 1 < kBins ? n * static_cast<uint64_t>(least * 0.99999f) : 0};
      };
      r.find_bins(bounds, max(static_cast<uint64_t>(coarse * 0.99999), static_cast<uint64_t>(1)),
                  static_cast<uint64_t>(coarse * 1.00001) + 1);
      const int first = sh.bin[0], last = max(sh.bin[0], sh.bin[1]);
      kept = 0;
      r.sweep_kept([&](float l, int index) {
        const int b = r.bin_of(l);
        if (b < first) kept += r.weigh(l);
        if (b >= first && b <= last) r.put(l, index);
      });
      const uint64_t above = r.exchange(kept, 0).x, want = max(static_cast<uint64_t>(ceil(part)), static_cast<uint64_t>(1));
      r.template cut_at<true>(want - min(want, above), first, last);
      r.sweep_kept([&](float l, int) {
        const int b = r.bin_of(l);
        if (b >= first && b <= last) kept += r.weigh(l);
      });
      total = r.exchange(kept, 0).x;
    }
  }

  if (FILTER) {
    const float inv = static_cast<float>(exp2(static_cast<double>(a.scale)) / static_cast<double>(total)) * 4.656612873077393e-10f;  // 2^-31
    const int lo = max(r.place0 - r.shift, 0), hi = min(r.place0 + a.slice - r.shift, a.vocab);
    float* out = a.probs + line * a.vocab;
    const float* logit = r.logit + r.shift - r.place0;  // by index
    auto prob = [&](int x) {
      const float l = logit[x];
      if (total == 0 || !r.cut.keeps(key_of(l), x)) return 0.f;
      if (greedy) return 1.f;
      uint64_t m;
      int whole;
      if (!r.weight(l, 160.f, m, whole)) return 0.f;
      const int half = whole / 2;
      return __uint2float_rn(static_cast<uint32_t>(m >> 32)) * inv * __int_as_float((127 - half) << 23) *
             __int_as_float((127 - whole + half) << 23);
    };
    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(out) / 4 % 4);  // out - lead lies on 16 bytes
    for (int x = (lo + lead) / 4 * 4 - lead + tid * 4; x < hi; x += kThreads * 4) {
      if (x >= lo && x + 4 <= hi) {
        __stcs(reinterpret_cast<float4*>(out + x), make_float4(prob(x), prob(x + 1), prob(x + 2), prob(x + 3)));
      } else {
        for (int i = max(x, lo); i < min(x + 4, hi); ++i) out[i] = prob(i);
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
        const bool in = y < (w + 1) * r.run && r.cut.keeps(key_of(r.logit[min(y, a.slice - 1)]), index);
        const uint64_t mine = in ? r.weigh(r.logit[y]) : 0, upto = warp_scan(mine);
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
template <typename T, bool FILTER>
bool prepare_kernel() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (ready.load() & bit) return true;
  const auto kernel = sample_kernel<T, FILTER>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFixedBytes + kMaxSlice * 4) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return false;
  ready.fetch_or(bit);
  return true;
}

template <typename T, bool FILTER>
qnre_status_t launch(SampleArgs a, int64_t rows, qnre_stream_t stream) {
  if (!prepare_kernel<T, FILTER>()) return QNRE_ERR_CUDA;
  // As many CTAs a row as the machine holds at once, while each keeps a grain of places; and as many as hold the row.
  const int64_t places = a.vocab + 16 / sizeof(T) - 1;
  unsigned cluster = kMaxCluster;
  while (cluster > 1 && (rows * cluster > 152 * 3 || places <= static_cast<int64_t>(cluster / 2) * kGrain)) cluster /= 2;
  while (cluster < kMaxCluster && places > static_cast<int64_t>(cluster) * 16384) cluster *= 2;
  a.slice = static_cast<int>(((places + cluster - 1) / cluster + kGrain - 1) / kGrain * kGrain);
  a.scale = 62;
  while (a.scale > 0 && (int64_t{1} << (62 - a.scale)) < a.vocab) --a.scale;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kFixedBytes + a.slice * 4;
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
  return from_cuda(cudaLaunchKernelEx(&cfg, sample_kernel<T, FILTER>, a));
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
    case QNRE_DTYPE_FP32: return launch<float, FILTER>(a, rows, stream);
    case QNRE_DTYPE_BF16: return launch<__nv_bfloat16, FILTER>(a, rows, stream);
    default: return launch<__half, FILTER>(a, rows, stream);
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
