// prefix_attention.cu -- attention over a paged cache whose rows share their leading pages (samples, drafts or requests
// of one prompt): the common tokens are read once for the whole group.  Scores may be capped by a tanh and get a bias
// that falls with distance.
//
//   o = sum_x p_x v_x,  p = softmax(cap tanh(scale q.k_x / cap) + slope (pos_x - pos_q)) over the tokens a node sees
//
// A softmax over two sets of tokens is the join of two softmaxes, so each row has two parts: its group's common tokens,
// where all members' nodes and query heads of a K head are rows of one matrix product, and its own tokens behind them.
// Units are 128 rows of (request, node, query head of a K head).  A unit of common tokens sees every tile; as many of them as a
// cluster has CTAs fetch K and V for one another by multicast, what is left over of a group goes to single CTAs.  A unit
// of own tokens holds the same rows of up to 128 requests (16 of one node with 8 heads) and runs through the requests' tiles
// one request after another: a tile's P is zero for the others' rows, so they share the unit's start and end, which cost as much
// as three tiles, and the softmax of one request's tile runs beside the next one's, as their rows lie with
// different warps.  Clusters and single CTAs take equal runs of tiles in proportion to the work, side by side in one
// launch.  A second kernel joins a row's parts: the group's in the order of its tiles, then its own.  Everything is found from
// lengths in device memory by each CTA itself (the number of common tokens too), so a captured call follows them, and the
// order of sums depends on them alone.
//
// In a CTA the roles are those of tree_attention.cu: two TMA warps, two threads that issue the products, eight softmax
// warps of which two threads share a row of 128.
//
// Values that a row must not see: as in tree_attention.cu scores are replaced before use.  In a unit of several requests a row's
// P is zero, whatever its scores, in the tiles of the others, and as 0 inf is NaN the warp that issues the product
// zeroes V's non-finite elements before it, and V behind a request's tokens.  (It has the time, while the softmax of the tile
// runs.  Where the softmax threads cleaned the last tokens' V themselves, 8, 128, 48 and 24 requests took 24.8, 123, 97 and 108
// us, the search for common tokens included, for 22.9, 123, 89 and 102.)  The rows of a request with such an element are marked,
// and the join gives them their infinite and NaN columns, which it looks up in V (own_strange); all else is the product's, so
// nothing that one request holds changes a bit of another's result.
//
// Bound: long common prefixes and many rows, by a tile of 128 tokens by 128 rows of D = 128: 1840 cycles where its products alone
// are 1024.  That is what the softmax takes, and about what TMA takes to bring its 64 KB into an SM (34 bytes a cycle); the two
// were not told apart.  128 requests of 64 + 8 heads with 6 prefixes of 1500 to 30011 tokens take 115 us (the tensor pipe busy 44 %
// of it), against 658 when each request reads its prefix: 72 tiles a CTA are 65-70 us of them, setup and join 7, and the rest is
// own tiles and units' ends, which were not measured apart.  Own tokens, by latency and the bytes that a few rows each
// need: 48 requests of up to 3000 own tokens under a cap 86 us, floor 27, over 4000 cycles a tile, as one pair of warps has a
// tile's one live row.  Short calls, by latency: 8 requests of 2011 + up to 400 tokens 16.3 us, of them the setup 4, a
// unit's start and end 4, the join 3.
// Blocks of many requests' own tokens brought the first case from 124 us to 117, a form with smaller tables and a third V stage
// to 115, the capped case 122 -> 107, and the polynomial for tanh 107 -> 85.  Divisors as products took the setup from 9500
// cycles to 7640.  Tried and left: turns of four requests' tiles in a block (127 us for 121); V cleaned by softmax warps without a
// row of the tile (the four cases of more_operators.py 22.7, 129, 110 and 126 us), by the TMA warp a ring behind (25, 148, 100, 117).
#include "../../include/qnre.h"
#include "attention_tile.cuh"
#include "cache.cuh"
#include "ptx.cuh"
#include "tma_map.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>

namespace {

using namespace qnre;
using namespace qnre::api;
using namespace qnre::attention;

constexpr int kSoftThreads = 256;
constexpr int kThreads = kSoftThreads + 128;
constexpr int kMaxCtas = 152;  // one a SM
constexpr int kTmemS = 0, kTmemO = 256, kTmemP = 384;  // columns: S 2 x 128, O D, P 2 x 64
constexpr int kMaxCluster = 4;
constexpr int kUnitCost = 4;  // a unit's start and end, in tiles
constexpr int kSmallRequests = 128, kSmallGroups = 31, kSmallBlocks = 32;  // (see Smem)
constexpr float kLog2e = 1.4426950408889634f;

// Division of 0 <= x < 2^31 by a number that the host knows: a product and a shift (the divide is some 200 cycles of latency,
// and every CTA's setup and every unit have several).
struct Divisor {
  uint32_t mul, shift;
  static Divisor of(int d) {
    uint32_t shift = 31;
    while ((1ull << (shift - 31)) < static_cast<uint32_t>(d)) ++shift;
    return Divisor{static_cast<uint32_t>((1ull << shift) / static_cast<uint32_t>(d) + 1), shift};  // (mul is below 2^32)
  }
  __device__ __forceinline__ int operator()(int x) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(x)) * mul >> shift);
  }
};

// Where a unit's results are: `parts` runs of it from CTA `cta` on, `step` apart; 0: one piece, in the rows' own places.
struct Desc {
  int cta, step, parts;
};

struct PrefixArgs {
  CUtensorMap tk, tv, tq;
  CacheView c;
  const int32_t *rows, *groups, *shared, *counts, *depths;
  const uint64_t* mask;
  const float* slopes;
  char* out;
  float* lse;
  int2* requests;     // [n]: the first request of the group whose common tokens a request reads, or -1; how many
  Desc* row_units;    // [n][Hk][row_tiles], by the first request of the unit
  Desc* group_units;  // the same
  float4* part_ml;    // [2 kMaxCtas 128 + rows of both kinds]: maximum (base 2), sum, marks of either half of the columns
  float4* part_o;     // the same rows of D, laid out by piece_of
  long long own_rows, group_rows;  // where the rows' own places begin, for each kind
  float scale_log2, cap_in, cap_log2;  // capped: scale / cap, cap log2(e)
  float cap_near, cap_poly[3];         // the nearer polynomial of run_softmax in powers of q.k, and up to where it serves
  int layer, n, n_groups, nodes, Hq, Hk, G, box, cl;
  int unit_nodes, unit_members, row_tiles;  // nodes and requests of a unit; units that one request's nodes take
  int warp_members;                         // requests whose rows one warp has
  Divisor by_page, by_G, by_nodes, by_members, by_tiles, by_cl;  // of page_size, G, unit_nodes, unit_members, row_tiles, cl
  bool backward;  // tiles from the last to the first: where the bias favours near tokens the maxima do not grow tile by tile
};

// Eight rows' pieces of 16 bytes lie side by side, so that the threads that write, a row each, fill whole lines.
template <int D>
__device__ __forceinline__ long long piece_of(long long row, int i) {
  return ((row >> 3) * (D / 4) + i) * 8 + (row & 7);
}

// Shared memory.  Three tiles of K and of V in flight feed the products (two of V: 2200 cycles a shared tile instead of
// 1840); at D = 128 they leave 3 KB, which tables of up to 128 requests and 31 groups fit into (SMALL).
template <int D, bool SMALL>
struct Smem {
  static constexpr int kRequests = SMALL ? kSmallRequests : QNRE_MAX_CALL_ROWS;
  static constexpr int kGroups = SMALL ? kSmallGroups : QNRE_MAX_CALL_ROWS;
  static constexpr int kBlocks = SMALL ? kSmallBlocks : QNRE_MAX_CALL_ROWS;
  static constexpr int kMlBuffers = SMALL ? 1 : 2;
  static constexpr int kKStages = D == 128 ? 3 : 5;
  static constexpr int kVStages = D == 128 ? (SMALL ? 3 : 2) : 5;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kTileBytes;
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kBars = kV + kVStages * kTileBytes;
  static constexpr int kWords = kBars + 8 * (2 * kKStages + 2 * kVStages + 13);
  static constexpr int kMl = kWords + 32;                           // float [kMlBuffers][2][128]
  static constexpr int kBase = kMl + kMlBuffers * 1024;             // int [kRequests]
  static constexpr int kLen = kBase + kRequests * 4;
  static constexpr int kCommon = kLen + kRequests * 4;              // int [kGroups]
  static constexpr int kStarts = kCommon + kGroups * 4;             // int [kGroups + 1]
  static constexpr int kSingle = kStarts + kGroups * 4 + 4;         // int [kBlocks + kGroups + 1]
  static constexpr int kWide = kSingle + (kBlocks + kGroups) * 4 + 4;  // int [kGroups + 1]
  static constexpr int kDrafts = kWide + kGroups * 4 + 4;           // uint8 [kRequests]
  static constexpr int kBytes = kDrafts + kRequests;
  static_assert(kBytes <= 232448, "one CTA's shared memory");
};

struct Words {
  unsigned long long marked[3];  // requests of a unit (pairs of them, above 64) with non-finite drafts, segments in turn
  uint32_t tmem, abort;
};

struct Bars {
  uint32_t kfull, kempty, vfull, vempty, qfull, qempty, sfull, sfree, pready, pvdone, ofree, drain, drain2;
};

// The tables that every CTA makes for itself.
struct Tables {
  int *base, *len;           // requests: tokens of their own from base on, context up to len
  uint8_t* drafts;           // behind it
  int *starts, *common;      // groups: first requests, common tokens
  int *single, *wide;        // where the items begin in the run of the single CTAs and of the clusters
  int blocks, n_groups;      // single items: blocks of requests, then what the clusters leave of each group
};

// One unit's part of a CTA's run.
struct Seg {
  bool group, whole;
  int kvh, rt, t0, t1;
  int start, members;  // requests
  int tokens;          // of a group
  int begin, tiles;    // the run's place of its first tile
  int slot;
};

__device__ __forceinline__ int tiles_of(int tokens) { return tokens > 0 ? (tokens + kTile - 1) / kTile : 1; }

// A CTA's run over the units of its kind.
struct Cursor {
  Tables t;
  const int* pre;
  int cur, end, item, index, count, quot, rem;  // run `index` of `count`
  int n, Hk, cl, rank, row_tiles, unit_members;
  Divisor by_members, by_cl;
  bool wide;

  // Units of a group for one K head, and those of them that clusters take.
  __device__ __forceinline__ int units_of(int members) const { return by_members(members + unit_members - 1) * row_tiles; }
  __device__ __forceinline__ int shared_units(int units) const { return cl > 1 ? by_cl(units) * cl : 0; }
  __device__ __forceinline__ int start_of(int c) const { return c * quot + c * rem / count; }
  __device__ __forceinline__ bool next(Seg& s) {
    while (cur < end) {
      while (cur >= pre[item + 1]) ++item;
      s.group = wide || item >= t.blocks;
      int per_head = row_tiles, first = 0;
      if (s.group) {
        const int g = wide ? item : item - t.blocks;
        s.start = t.starts[g];
        s.members = t.starts[g + 1] - s.start;
        s.tokens = t.common[g];
        const int units = units_of(s.members), full = shared_units(units);
        per_head = wide ? by_cl(full) : units - full;
        first = wide ? 0 : full;
      } else {
        s.start = item * unit_members;
        s.members = min(unit_members, n - s.start);
        s.tokens = 0;
      }
      const int per = (pre[item + 1] - pre[item]) / (per_head * Hk);
      const int off = cur - pre[item];
      const int unit = off / per, o = off - unit * per;
      const int take = min(per - o, end - cur);
      s.tiles = per - kUnitCost;
      s.begin = cur - o + kUnitCost;
      cur += take;
      s.t0 = max(0, o - kUnitCost);
      s.t1 = max(0, o + take - kUnitCost);
      if (s.t0 == s.t1) continue;  // the unit's cost falls to this CTA, its tiles to the next
      s.kvh = unit / per_head;
      s.rt = first + (unit - s.kvh * per_head) * (wide ? cl : 1) + rank;
      s.whole = s.t0 == 0 && s.t1 == s.tiles;
      // a CTA goes on with one unit at most, and leaves one unfinished at most
      s.slot = 2 * static_cast<int>(blockIdx.x) + (s.t0 == 0 ? 1 : 0);
      return true;
    }
    return false;
  }
};

// The way through the requests' tiles of a unit of own tokens: one request after another, in steps of the requests whose rows
// one warp has, so that neighbours lie with different warps.  (Turns of a tile each, over four requests in different
// quarters, cost more in bookkeeping than they overlap: 128 rows in 6 groups 127 us against 121.)
struct Walk {
  int mi, column, tile, tiles, step, members;
  int base, len, total;  // of the request
  const int *bases, *lens;
  const uint8_t* drafts;  // from the unit's first request on

  __device__ __forceinline__ int position(bool backward) const { return base + (backward ? tiles - 1 - tile : tile) * kTile; }
  __device__ __forceinline__ void enter() {
    base = bases[mi];
    len = lens[mi];
    total = len + drafts[mi];
    tiles = tiles_of(total - base);
  }
  __device__ __forceinline__ void next_request() {
    mi += step;
    if (mi >= members) mi = ++column;
    enter();
  }
  __device__ __forceinline__ void begin(const Tables& t, const Seg& s, int requests_a_warp) {
    if (s.group) return;
    step = requests_a_warp;
    members = s.members;
    bases = t.base + s.start;
    lens = t.len + s.start;
    drafts = t.drafts + s.start;
    mi = column = 0;
    tile = s.t0;
    for (enter(); tile >= tiles; next_request()) tile -= tiles;
  }
  __device__ __forceinline__ void next() {  // (not behind the unit's last tile)
    if (++tile < tiles) return;
    tile = 0;
    next_request();
  }
};

__device__ __forceinline__ int group_position(const Seg& s, int t, bool backward) { return (backward ? s.tiles - 1 - t : t) * kTile; }

// What row `ur` of a unit stands for.
struct UnitRow {
  int member, node, head;  // member: of the unit
  bool there;
};
__device__ __forceinline__ int unit_tile(const PrefixArgs& a, const Seg& s) { return s.group ? a.by_tiles(s.rt) : 0; }
__device__ __forceinline__ UnitRow unit_row(const PrefixArgs& a, const Seg& s, int ur) {
  const int q = a.by_G(ur), tile = unit_tile(a, s), block = s.rt - tile * a.row_tiles;
  UnitRow r;
  r.member = a.by_nodes(q);
  r.node = block * a.unit_nodes + q - r.member * a.unit_nodes;
  r.head = ur - q * a.G;
  r.there = r.member < a.unit_members && tile * a.unit_members + r.member < s.members && r.node < a.nodes;
  return r;
}

// Among the softmax threads.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }

// ------------------------------------------------------------------ TMA warps
// One warp brings K, another Q and V (so that K of the next unit does not wait for the last use of Q).  With `share` each CTA
// of the cluster fetches its share of a tile's boxes for all.
template <typename L, int D>
__device__ void run_producer(const PrefixArgs& a, const Bars& bars, uint32_t smem, Cursor cur, Seg s, bool more, int kv,
                             bool share, volatile uint32_t* abort_flag) {
  constexpr int kHalves = D / 64;
  const int lane = threadIdx.x % 32;
  const int chunk = lane / kHalves, half = lane % kHalves;
  const bool active = chunk < kTile / a.box && (!share || lane % a.cl == cur.rank);
  const int ps = a.c.page_size;
  const int none = a.c.layers * a.c.pages;  // past the end: the box is filled with zeros
  const uint16_t everyone = static_cast<uint16_t>((1u << a.cl) - 1u);
  const CUtensorMap* map = kv ? &a.tv : &a.tk;
  const uint32_t dst = smem + (kv ? L::kV : L::kK) + half * (kTile * 128) + chunk * a.box * 128;
  const uint32_t q_bytes = static_cast<uint32_t>(D * 2 * a.G * a.unit_nodes * a.unit_members);
  const uint32_t full = kv ? bars.vfull : bars.kfull, empty = kv ? bars.vempty : bars.kempty;
  const uint32_t stages = kv ? L::kVStages : L::kKStages;
  uint32_t slot = 0, phase = 1;
  auto settle = [] {  // stop: what is in flight lands in microseconds; the kernel's end waits for it
    const uint64_t t0 = ptx::global_timer_ns();
    while (ptx::global_timer_ns() - t0 < 50000) {
    }
  };
  for (uint32_t seg = 0; more; ++seg, more = cur.next(s)) {
    if (kv == 1) {  // the unit's Q rows (one buffer: the last unit's scores are done)
      if (!wait(bars.qempty, (seg & 1u) ^ 1u, abort_flag, a.c.status)) return settle();
      if (lane == 0) ptx::mbar_arrive_expect_tx(bars.qfull, q_bytes);
      __syncwarp();
      const int tile = unit_tile(a, s);
      const int node = (s.rt - tile * a.row_tiles) * a.unit_nodes, request = s.start + tile * a.unit_members;
      if (lane < kHalves)
        tma_load_4d(smem + L::kQ + lane * (kTile * 128), &a.tq, bars.qfull, lane * 64, s.kvh * a.G, node, request);
    }
    Walk walk;
    walk.begin(cur.t, s, a.warp_members);
    // the tile ahead: this lane's token, the tokens' end, and its entry of the block table
    bool fetches = false;
    const int32_t* table = nullptr;
    int pos = 0, end = 0, entry = -1, off = 0;
    auto enter = [&](int request) {
      const int row = a.rows[request];
      fetches = active && row >= 0 && row < a.c.rows;
      table = a.c.table + static_cast<long long>(fetches ? row : 0) * a.c.max_blocks;
    };
    auto look = [&] {
      const int block = a.by_page(pos);
      off = pos - block * ps;
      entry = fetches && pos < end && block < a.c.max_blocks ? table[block] : -1;
    };
    if (s.group) {
      enter(s.start);
      pos = group_position(s, s.t0, a.backward) + chunk * a.box;
      end = s.tokens;
    } else {
      enter(s.start + walk.mi);
      pos = walk.position(a.backward) + chunk * a.box;
      end = walk.total;
    }
    look();
    for (int t = s.t0; t < s.t1; ++t) {
      const bool there = entry >= 0 && entry < a.c.pages;
      if (fetches && !there && pos < end) atomicOr(a.c.status, QNRE_CACHE_BAD_PAGE);
      const int page = there ? a.layer * a.c.pages + entry : none, at = off;
      if (t + 1 < s.t1) {  // the next tile's entry is on its way while this tile's place is waited for
        if (s.group) {
          pos = group_position(s, t + 1, a.backward) + chunk * a.box;
        } else {
          walk.next();
          enter(s.start + walk.mi);
          pos = walk.position(a.backward) + chunk * a.box;
          end = walk.total;
        }
        look();
      }
      if (!wait(empty + 8 * slot, phase, abort_flag, a.c.status)) return settle();
      if (lane == 0) ptx::mbar_arrive_expect_tx(full + 8 * slot, L::kTileBytes);
      __syncwarp();
      if (active) {
        if (share)
          tma_load_4d_multicast(dst + slot * L::kTileBytes, map, full + 8 * slot, half * 64, at, s.kvh, page, everyone);
        else
          tma_load_4d(dst + slot * L::kTileBytes, map, full + 8 * slot, half * 64, at, s.kvh, page);
      }
      if (++slot == stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

// ------------------------------------------------------------------ MMA threads
__device__ __forceinline__ void release(uint32_t bar, bool share, uint16_t everyone) {
  if (share)
    umma_commit_multicast(bar, everyone);
  else
    ptx::umma_commit(bar);
}

// S = Q K^T, tile after tile, across units.
template <typename L, int D, bool BF16>
__device__ void run_scores(const PrefixArgs& a, const Bars& bars, uint32_t smem, uint32_t tmem, Cursor cur, Seg s,
                           bool more, bool share, volatile uint32_t* abort_flag) {
  constexpr uint32_t kFmt = BF16 ? (1u << 7 | 1u << 10) : 0u;
  constexpr uint32_t kIdesc = (1u << 4) | kFmt | ((kTile >> 3) << 17) | ((128u >> 4) << 24);
  const uint64_t ring0 = ptx::smem_desc_sw128(smem + L::kK, 16, 1024);
  const uint64_t q = ptx::smem_desc_sw128(smem + L::kQ, 16, 1024);
  const uint16_t everyone = static_cast<uint16_t>((1u << a.cl) - 1u);
  uint32_t g = 0, slot = 0, phase = 0;
  for (uint32_t seg = 0; more; ++seg, more = cur.next(s)) {
    if (!wait(bars.qfull, seg & 1u, abort_flag, a.c.status)) return drain_mma(bars.drain);
    for (int t = s.t0; t < s.t1; ++t, ++g) {
      const uint32_t b = g & 1u;
      if (!wait(bars.kfull + 8 * slot, phase, abort_flag, a.c.status) ||
          !wait(bars.sfree + 8 * b, ((g >> 1) & 1u) ^ 1u, abort_flag, a.c.status))
        return drain_mma(bars.drain);
      ptx::tc_fence_after_sync();
      const uint64_t k = desc_at(ring0, slot * L::kTileBytes);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (kTile * 128) + (kk % 4) * 32;
        ptx::umma_f16(tmem + kTmemS + b * 128, desc_at(q, off), desc_at(k, off), kIdesc, kk > 0 ? 1u : 0u);
      }
      ptx::umma_commit(bars.sfull + 8 * b);
      release(bars.kempty + 8 * slot, share, everyone);
      if (t + 1 == s.t1) ptx::umma_commit(bars.qempty);
      if (++slot == L::kKStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

// Makes a V tile fit for zero weights (a whole warp): rows [from, to) without their infinite and NaN elements, rows [to, end),
// which hold no token, zero.  True where there were any such elements.
template <int D, bool BF16>
__device__ __forceinline__ bool clean_v_tile(uint32_t tile, int from, int to, int end) {
  constexpr int kPieces = D / 8;
  const int lane = threadIdx.x % 32;
  auto piece_at = [&](int x, int i) { return tile + x * 128 + (i / 8) * (kTile * 128) + ((i ^ lane) % 8) * 16; };
  bool found = false;
#pragma unroll 1
  for (int x = from + lane; x < to; x += 32) {
    uint32_t sum[4] = {0, 0, 0, 0};  // 0 x is 0 for every finite x
#pragma unroll 16
    for (int i = 0; i < kPieces; ++i) {
      uint32_t w[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(piece_at(x, i))
                   : "memory");
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (BF16)
          asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[e]) : "r"(w[e]), "r"(0));
        else
          asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum[e]) : "r"(w[e]), "r"(0));
      }
    }
    if (((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7FFF7FFFu) != 0)
      found |= clean_v_row<D, BF16>(reinterpret_cast<char*>(__cvta_shared_to_generic(tile + x * 128)), true, 0, kPieces);
  }
  if (to < end) {
#pragma unroll 1
    for (int x = to + lane; x < end; x += 32)
#pragma unroll 1
      for (int i = 0; i < kPieces; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(piece_at(x, i)), "r"(0) : "memory");
    ptx::fence_proxy_async_smem();
  }
  return found;
}

// The same as a call: where the softmax takes all registers, a copy in line cost its schedule more (24 drafted trees with cap and
// bias 106 us, in line 116; 128 requests' plain scores 129 and 121, 64 channels with a cap 95 and 94).
template <int D, bool BF16>
__device__ __noinline__ bool clean_v_tile_apart(uint32_t tile, int from, int to, int end) {
  return clean_v_tile<D, BF16>(tile, from, to, end);
}

// O += P V, tile after tile; names the places of the units begun here for the join.  Lane 0 issues; in units of several requests the
// warp takes the infinite and NaN elements out of the context's V first, while the softmax of the tile runs.
template <typename L, int D, bool BF16, bool APART>
__device__ void run_outputs(const PrefixArgs& a, const Bars& bars, char* smem_base, uint32_t tmem, Cursor cur, Seg s,
                            bool more, bool share, volatile uint32_t* abort_flag, unsigned long long* marked) {
  constexpr uint32_t kFmt = BF16 ? (1u << 7 | 1u << 10) : 0u;
  constexpr uint32_t kIdesc =
      (1u << 4) | kFmt | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24);
  const uint64_t ring0 = ptx::smem_desc_sw128(ptx::smem_addr(smem_base) + L::kV, kTile * 128, 1024);
  const uint16_t everyone = static_cast<uint16_t>((1u << a.cl) - 1u);
  const int lane = threadIdx.x % 32, mark_shift = a.unit_members > 64 ? 1 : 0;
  uint32_t g = 0, slot = 0, phase = 0;
  bool stopped = false;  // lane 0: a wait ran out
  for (uint32_t seg = 0; more; ++seg, more = cur.next(s)) {
    if (s.t0 == 0 && lane == 0) {
      int parts = 0;
      if (!s.whole) {
        int lo = cur.index, hi = cur.count - 1;  // the last run that starts by the last tile
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (cur.start_of(mid) <= s.begin + s.tiles - 1) lo = mid; else hi = mid - 1;
        }
        parts = lo - cur.index + 1;
      }
      const int tile = unit_tile(a, s), request = s.start + tile * a.unit_members;
      (s.group ? a.group_units : a.row_units)[(request * a.Hk + s.kvh) * a.row_tiles + s.rt - tile * a.row_tiles] =
          Desc{static_cast<int>(blockIdx.x), share ? a.cl : 1, parts};
    }
    Walk walk;
    if (!s.group) {
      __syncwarp();  // lane 0 has seen every tile before: a wait for one of the ring's next phases means that phase
      walk.begin(cur.t, s, a.warp_members);
    }
    for (int t = s.t0; t < s.t1; ++t, ++g) {
      const uint32_t b = g & 1u;
      const bool first = t == s.t0;
      if (!s.group) {
        const int pos0 = walk.position(a.backward), tokens = walk.total - walk.base, member = walk.mi;
        const int from = a.unit_members > 1 ? 0 : max(walk.len - pos0, 0);  // (alone, a request meets its own context's values)
        const int to = min(walk.total - pos0, kTile), end = min(((tokens + a.box - 1) & -a.box) + walk.base - pos0, kTile);
        if (t + 1 < s.t1) walk.next();
        if (from < end && wait(bars.vfull + 8 * slot, phase, abort_flag, a.c.status)) {
          const uint32_t v = ptx::smem_addr(smem_base) + L::kV + slot * L::kTileBytes;
          if (APART ? clean_v_tile_apart<D, BF16>(v, from, to, end) : clean_v_tile<D, BF16>(v, from, to, end)) {
            atomicOr(marked + seg % 3, 1ull << (member >> mark_shift));
            __threadfence_block();
          }
        }
        __syncwarp();
      }
      if (lane == 0 && !stopped) {
        if (!wait(bars.vfull + 8 * slot, phase, abort_flag, a.c.status) ||
            (first && !wait(bars.ofree, (seg & 1u) ^ 1u, abort_flag, a.c.status)) ||
            !wait(bars.pready + 8 * b, (g >> 1) & 1u, abort_flag, a.c.status)) {
          drain_mma(bars.drain2);
          stopped = true;
        } else {
          ptx::tc_fence_after_sync();
          const uint64_t v = desc_at(ring0, slot * L::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma_f16_ts(tmem + kTmemO, tmem + kTmemP + b * 64 + kk * 8, desc_at(v, kk * 2048), kIdesc,
                        (t > s.t0 || kk > 0) ? 1u : 0u);
          ptx::umma_commit(bars.pvdone + 8 * b);
          release(bars.vempty + 8 * slot, share, everyone);
        }
      }
      if (!s.group) __syncwarp();  // (lanes that waited for the next tile meanwhile could hold lane 0 up)
      if (++slot == L::kVStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax warps
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Of the drafts that a row's mask names, those that have a place (`slots`).
__device__ __forceinline__ uint64_t seen_drafts(int slots, uint64_t mask) {
  return slots < 64 ? mask & ((1ull << slots) - 1) : mask;
}

// Two threads a row, half a tile each.  SCORED: scores are capped or biased, and come out in base 2; else the scale is
// applied with the maximum.
template <typename L, int D, bool BF16, bool SCORED>
__device__ void run_softmax(const PrefixArgs& a, const Bars& bars, char* smem_base, uint32_t tmem, Cursor cur, Seg next,
                            bool more, volatile uint32_t* abort_flag, unsigned long long* marked) {
  constexpr int kCols = kTile / 2, kOut = D / 2;  // tokens of a tile, columns of O this thread has
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int ur = tid % 128, copy = tid / 128, c0 = copy * kCols, o0 = copy * kOut;
  const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
  float* ml = reinterpret_cast<float*>(smem_base + L::kMl);
  const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
  const int mark_shift = a.unit_members > 64 ? 1 : 0;

  // what this thread's row of a segment is
  struct RowInfo {
    UnitRow at;
    bool row_ok;    // of a node that sees anything
    int request;
    uint64_t bits;  // the drafts it sees
    int place;      // its position
    float slope;    // in base 2
  };
  auto row_info = [&](const Seg& s) {
    RowInfo r{unit_row(a, s, ur), false, 0, 0, 0, 0.f};
    if (!r.at.there) return r;
    const int i = r.request = s.start + unit_tile(a, s) * a.unit_members + r.at.member;
    r.row_ok = a.counts == nullptr || r.at.node < a.counts[i];
    if (!s.group)
      r.bits = a.mask != nullptr ? a.mask[static_cast<long long>(i) * a.nodes + r.at.node] : (2ull << r.at.node) - 1;
    if (SCORED && a.slopes != nullptr) {
      r.slope = a.slopes[s.kvh * a.G + r.at.head] * kLog2e;
      r.place = cur.t.len[i] + (a.depths != nullptr ? a.depths[static_cast<long long>(i) * a.nodes + r.at.node] : r.at.node);
    }
    return r;
  };

  uint32_t g = 0;
  Seg s;
  RowInfo row{}, next_row{};
  if (more) next_row = row_info(next);
  for (uint32_t seg = 0; more; ++seg) {
    s = next;
    row = next_row;
    const bool in_out = row.at.there, row_ok = row.row_ok;
    Walk walk;
    walk.begin(cur.t, s, a.warp_members);
    float m = -INFINITY, l = 0.f;
    for (int t = s.t0; t < s.t1; ++t, ++g) {
      const uint32_t b = g & 1u;
      int pos0 = group_position(s, t, a.backward), len = s.tokens, total = s.tokens, member = 0;
      bool mine = true;  // a row that sees this tile
      if (!s.group) {
        member = walk.mi;
        pos0 = walk.position(a.backward);
        len = walk.len;
        total = walk.total;
        mine = row.at.member == member;
        if (t + 1 < s.t1) walk.next();
      }
      const bool active = __any_sync(0xFFFFFFFFu, mine);
      const bool tail = pos0 + kTile > len;
      wait(bars.pvdone + 8 * b, ((g >> 1) & 1u) ^ 1u, abort_flag, a.c.status);
      uint32_t p[kCols / 2];
      if (active) {
        uint32_t v[kCols / 32][32];
        wait(bars.sfull + 8 * b, (g >> 1) & 1u, abort_flag, a.c.status);
        __syncwarp();  // the tensor-memory instructions are warp-wide
        ptx::tc_fence_after_sync();
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j)
          ptx::tmem_ld_32x32b_x32(tmem + lane_base + kTmemS + b * 128 + c0 + 32 * j, v[j]);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j) tmem_fence_regs(v[j]);
        ptx::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.sfree + 8 * b);

        float offset = 0.f;  // (SCORED) of the first eight columns; the next ones' lie 8 slopes apart
        if (SCORED) {
          // c tanh(x / c) = x + x (x / c)^2 P: the polynomial P is fitted by least squares up to 0.35 (4e-8 relative) and up to
          // 1 (6e-8); beyond, 1 - 2 / (1 + e^2z): to 2^-22 of the cap, however large.  The largest score that a thread's row sees
          // of its half tile says which, so that no other row, unused slot or hidden draft changes a bit of it.
          // The distance bias of a column is slope (i % 8), added here, and its eight columns' offset, added to their maximum and
          // with the row's maximum before the exponential.
          const int d0 = pos0 + c0;
          uint64_t within[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) within[i] = pair(row.slope * (2 * i), row.slope * (2 * i + 1));
          offset = a.slopes != nullptr ? row.slope * static_cast<float>(d0 - row.place) : 0.f;
          auto each_pair = [&](auto f) {
#pragma unroll
            for (int i = 0; i < kCols; i += 2) {
              uint32_t *x0 = &v[i / 32][i % 32], *x1 = &v[i / 32][(i + 1) % 32];
              float y0, y1;
              unpair(f(pair(__uint_as_float(*x0), __uint_as_float(*x1)), within[i / 2 % 4]), y0, y1);
              *x0 = __float_as_uint(y0);
              *x1 = __float_as_uint(y1);
            }
          };
          float most = 0.f;
          if (a.cap_log2 > 0.f) {
            float most1 = 0.f;
            if (!tail) {
#pragma unroll
              for (int i = 0; i < kCols; i += 4) {
                most = max3(most, fabsf(__uint_as_float(v[i / 32][i % 32])), fabsf(__uint_as_float(v[i / 32][(i + 1) % 32])));
                most1 = max3(most1, fabsf(__uint_as_float(v[i / 32][(i + 2) % 32])), fabsf(__uint_as_float(v[i / 32][(i + 3) % 32])));
              }
            } else {
              const uint64_t bits = seen_drafts(total - len, row.bits);
#pragma unroll
              for (int j = 0; j < kCols / 32; ++j) {
                const uint32_t see = seen_word(pos0 + c0 + 32 * j - len, bits);
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                  most = max3(most, see & (1u << i) ? fabsf(__uint_as_float(v[j][i])) : 0.f,
                              see & (2u << i) ? fabsf(__uint_as_float(v[j][i + 1])) : 0.f);
              }
            }
            most = mine && row_ok ? fmaxf(most, most1) * a.cap_in : 0.f;
          }
          auto both = [](float x) { return pair(x, x); };
          if (a.cap_log2 <= 0.f) {
            each_pair([&](uint64_t x, uint64_t bias) { return fma2(x, scale2, bias); });
          } else if (most <= a.cap_near) {
            const uint64_t k0 = both(a.cap_poly[0]), k1 = both(a.cap_poly[1]), k2 = both(a.cap_poly[2]);
            auto near = [&](uint64_t y, uint64_t z, uint64_t lead) {
              return fma2(y, fma2(z, fma2(z, fma2(z, k2, k1), k0), 0), lead);
            };
            if (a.slopes == nullptr)
              each_pair([&](uint64_t x, uint64_t) {
                const uint64_t y = fma2(x, scale2, 0);
                return near(y, fma2(x, x, 0), y);
              });
            else
              each_pair([&](uint64_t x, uint64_t bias) {
                return near(fma2(x, scale2, 0), fma2(x, x, 0), fma2(x, scale2, bias));
              });
          } else if (most <= 1.f) {
            const uint64_t in2 = both(a.cap_in);
            each_pair([&](uint64_t x, uint64_t bias) {
              const uint64_t y = fma2(x, scale2, 0), t = fma2(x, in2, 0), z = fma2(t, t, 0);
              uint64_t k = fma2(z, both(0.0010582602117210627f), both(-0.006259326823055744f));
              k = fma2(z, k, both(0.020359747111797333f));
              k = fma2(z, k, both(-0.05349870026111603f));
              k = fma2(z, k, both(0.13326409459114075f));
              k = fma2(z, k, both(-0.33332985639572144f));
              return fma2(y, fma2(z, k, 0), fma2(x, scale2, bias));
            });
          } else {
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
              const float e = exp2_fast(__uint_as_float(v[i / 32][i % 32]) * a.cap_in * 2.885390043258667f);  // 2 log2(e)
              v[i / 32][i % 32] = __float_as_uint(fmaf(rcp_fast(e + 1.f), -2.f * a.cap_log2, a.cap_log2 + row.slope * (i % 8)));
            }
          }
          __syncwarp();
          if (tail && a.slopes != nullptr && a.depths != nullptr && !s.group) {  // a draft lies at its depth, not at its slot
            const int32_t* depths = a.depths + static_cast<long long>(s.start + member) * a.nodes;
#pragma unroll 1
            for (int j = max(len - d0, 0); j < min(total - d0, kCols); ++j) {
              const int node = d0 + j - len;
              const float off = row.slope * static_cast<float>(depths[node] - node);
#pragma unroll
              for (int i = 0; i < kCols; ++i)
                if (i == j) v[i / 32][i % 32] = __float_as_uint(__uint_as_float(v[i / 32][i % 32]) + off);
            }
          }
        }
        if (tail) {
          const uint64_t bits = seen_drafts(total - len, row.bits);
#pragma unroll
          for (int j = 0; j < kCols / 32; ++j) {
            const uint32_t see = seen_word(pos0 + c0 + 32 * j - len, bits);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see & (1u << i))) v[j][i] = 0xFF800000u;
          }
        }
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int k = 0; k < kCols / 8; ++k) {
          const uint32_t* x = &v[k / 4][k % 4 * 8];
          float m0 = SCORED ? -INFINITY : mx0, m1 = SCORED ? -INFINITY : mx1;
#pragma unroll
          for (int i = 0; i < 8; i += 4) {
            m0 = max3(m0, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            m1 = max3(m1, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          }
          mx0 = SCORED ? fmaxf(mx0, fmaxf(m0, m1) + fmaf(row.slope, 8.f * k, offset)) : m0;
          mx1 = SCORED ? mx1 : m1;
        }
        float mx = fmaxf(mx0, mx1) * (SCORED ? 1.f : a.scale_log2);
        {  // with the other half's (two buffers: one is written again only when its tile's product is done)
          float* at = ml + (L::kMlBuffers == 2 ? b * 256 : 0) + ur;
          if (L::kMlBuffers == 1) pair_sync(warp % 4);
          at[copy * 128] = mx;
          pair_sync(warp % 4);
          mx = fmaxf(mx, at[(copy ^ 1) * 128]);
        }
        if (!mine) mx = -INFINITY;
        mx -= kLift<BF16>;  // m: the row's maximum less the lift, which leaves O / l and m + log2 l as they are
        const bool grow = mx > m + kRescale, fresh = m == -INFINITY;  // (a row that has seen nothing has no O to rescale)
        if (__any_sync(0xFFFFFFFFu, grow && !fresh)) {
          const uint32_t last = g - 1;
          wait(bars.pvdone + 8 * (last & 1u), (last >> 1) & 1u, abort_flag, a.c.status);
          __syncwarp();
          ptx::tc_fence_after_sync();
          const float f = grow && !fresh ? exp2_fast(m - mx) : 1.f;
          l *= f;
#pragma unroll 1
          for (int c = o0; c < o0 + kOut; c += 32) {
            uint32_t o[32];
            ptx::tmem_ld_32x32b_x32(tmem + lane_base + kTmemO + c, o);
            ptx::tmem_ld_wait();
            tmem_fence_regs(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st_x32(tmem + lane_base + kTmemO + c, o);
          }
          tmem_st_wait();
        }
        if (grow) m = mx;
        const float ms = mine ? (m == -INFINITY ? 0.f : m) : INFINITY;  // (a row that does not see the tile gets zeros)
        uint64_t neg = pair(-ms, -ms);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
          float e0, e1;
          const uint64_t x = pair(__uint_as_float(v[i / 16][(2 * i) % 32]), __uint_as_float(v[i / 16][(2 * i + 1) % 32]));
          if (SCORED && i % 4 == 0) {
            const float off = fmaf(row.slope, 2.f * i, offset) - ms;
            neg = pair(off, off);
          }
          unpair(SCORED ? add2(x, neg) : fma2(x, scale2, neg), e0, e1);
          e0 = exp2_fast(e0);
          e1 = exp2_fast(e1);
          sum[i & 1] = add2(sum[i & 1], pair(e0, e1));
          p[i] = pack2<BF16>(e0, e1);
        }
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        s0 += s1;
        if (__any_sync(0xFFFFFFFFu, !mine && s0 != 0.f)) {  // infinite or NaN scores of another request's keys (NaN is not 0)
          if (!mine) s0 = 0.f;
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i) p[i] = mine ? p[i] : 0u;
        }
        l += s0;
      } else {  // the tile of a request whose rows other warps have
        __syncwarp();
        ptx::tc_fence_after_sync();
        if (lane == 0) ptx::mbar_arrive(bars.sfree + 8 * b);
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) p[i] = 0;
      }
      tmem_st_x32(tmem + lane_base + kTmemP + b * 64 + c0 / 2, p);
      tmem_st_wait();
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars.pready + 8 * b);
    }
    if (!row_ok) {  // nothing seen: its scores were those of some other row's place
      m = -INFINITY;
      l = 0.f;
    }
    more = cur.next(next);
    if (more) next_row = row_info(next);  // on its way during this segment's end

    // ---------------- the segment's result
    const uint32_t last = g - 1;
    wait(bars.pvdone + 8 * (last & 1u), (last >> 1) & 1u, abort_flag, a.c.status);
    ml[tid] = l;  // (every warp is done with the maxima of its tiles)
    soft_sync();
    ptx::tc_fence_after_sync();
    // every warp has read the word of the segment before, and none uses it again before the next segment's end
    if (tid == 0) marked[(seg + 2) % 3] = 0;
    bool mark = row_ok && !s.group && (marked[seg % 3] >> (row.at.member >> mark_shift) & 1);
    l += ml[tid ^ 128];
    pair_sync(warp % 4);  // read by both before the next tile's maxima go there
    const bool done = s.whole && !s.group && in_out && cur.t.base[row.request] == 0;  // no other part of this row
    const float inv = !done ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
    const long long token = static_cast<long long>(row.request) * a.nodes + row.at.node;
    const long long orow = token * a.Hq + s.kvh * a.G + row.at.head;
    const long long prow = s.whole ? (s.group ? a.group_rows : a.own_rows) +
                                         (static_cast<long long>(s.kvh) * a.n * a.nodes + token) * a.G + row.at.head
                                   : static_cast<long long>(s.slot) * 128 + ur;
    // Warps without rows, and such whose requests have no tile here, have nothing to read.
    const bool any = __any_sync(0xFFFFFFFFu, in_out && (done || m != -INFINITY || l != 0.f));
    if (!any) {
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars.ofree);
    }
#pragma unroll 1
    for (int c = o0; any && c < o0 + kOut; c += 32) {
      uint32_t o[32];
      ptx::tmem_ld_32x32b_x32(tmem + lane_base + kTmemO + c, o);
      ptx::tmem_ld_wait();
      tmem_fence_regs(o);
      if (c + 32 == o0 + kOut) {
        ptx::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.ofree);
      }
      float x[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]);
      uint64_t odd = 0;  // 0 x is 0 for every finite x
#pragma unroll
      for (int i = 0; i < 32; i += 2) odd = fma2(pair(x[i], x[i + 1]), 0, odd);
      float odd0, odd1;
      unpair(odd, odd0, odd1);
      const bool strange = row_ok && odd0 + odd1 != 0.f;  // (NaN compares unequal)
      if (!s.group) {
        mark |= strange;
      } else if (__any_sync(0xFFFFFFFFu, strange)) {
        const int from = a.backward ? s.tiles - s.t1 : s.t0;
        const Kinds k = search_context<BF16>(a.c, a.layer, a.rows[s.start], s.kvh, from * kTile,
                                             min((from + s.t1 - s.t0) * kTile, s.tokens), c);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t bit = 1u << i;
          if ((k.plus | k.minus | k.nan) & bit)
            x[i] = (k.nan | (k.plus & k.minus)) & bit ? NAN : (k.plus & bit ? INFINITY : -INFINITY);
        }
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = row_ok ? x[i] * inv : 0.f;
      if (done) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack2<BF16>(x[2 * e], x[2 * e + 1]);
        uint4* dst = reinterpret_cast<uint4*>(a.out + (orow * D + c) * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      } else if (in_out && (m != -INFINITY || l != 0.f)) {  // (the join leaves out what has seen nothing)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          a.part_o[piece_of<D>(prow, c / 4 + i)] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
      __syncwarp();
    }
    if (in_out) {
      float* dst = reinterpret_cast<float*>(a.part_ml + prow);
      if (copy == 0) {
        *reinterpret_cast<float2*>(dst) = make_float2(m, l);
        if (done && a.lse != nullptr) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
      dst[2 + copy] = mark ? 1.f : 0.f;
    }
  }
}

// x[0 .. n) to its running sums or maxima; one warp.  One copy of the code: a CTA runs its setup once, so each line of it is
// fetched from L2.
__device__ __noinline__ void scan_table(int* x, int n, bool maximum) {
  const int lane = threadIdx.x % 32;
  int carry = 0;
  for (int base = 0; base < n; base += 32) {
    int v = base + lane < n ? x[base + lane] : 0;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v = maximum ? max(v, u) : v + u;
    }
    v = maximum ? max(v, carry) : v + carry;
    if (base + lane < n) x[base + lane] = v;
    carry = __shfl_sync(0xFFFFFFFFu, v, 31);
  }
}

template <int D, bool BF16, bool SMALL, bool SCORED>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ PrefixArgs a) {
  using L = Smem<D, SMALL>;
  extern __shared__ __align__(1024) char smem_base[];
  const uint32_t smem = ptx::smem_addr(smem_base);
  Words* words = reinterpret_cast<Words*>(smem_base + L::kWords);
  constexpr int kSoftWarps = kSoftThreads / 32;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  Bars bars;
  {
    uint32_t at = smem + L::kBars;
    auto take = [&](int n) {
      const uint32_t r = at;
      at += 8 * n;
      return r;
    };
    bars.kfull = take(L::kKStages);
    bars.kempty = take(L::kKStages);
    bars.vfull = take(L::kVStages);
    bars.vempty = take(L::kVStages);
    bars.qfull = take(1);
    bars.qempty = take(1);
    bars.sfull = take(2);
    bars.sfree = take(2);
    bars.pready = take(2);
    bars.pvdone = take(2);
    bars.ofree = take(1);
    bars.drain = take(1);
    bars.drain2 = take(1);
  }
  auto table = [&](int at) { return reinterpret_cast<int*>(smem_base + at); };
  Cursor cur;
  Tables& t = cur.t;
  t.base = table(L::kBase);
  t.len = table(L::kLen);
  t.drafts = reinterpret_cast<uint8_t*>(smem_base + L::kDrafts);
  t.starts = table(L::kStarts);
  t.common = table(L::kCommon);
  t.single = table(L::kSingle);
  t.wide = table(L::kWide);
  t.blocks = a.by_members(a.n + a.unit_members - 1);
  t.n_groups = a.n_groups;
  cur.n = a.n;
  cur.Hk = a.Hk;
  cur.cl = a.cl;
  cur.row_tiles = a.row_tiles;
  cur.unit_members = a.unit_members;
  cur.by_members = a.by_members;
  cur.by_cl = a.by_cl;
  if (warp == kSoftWarps) ptx::tmem_alloc(ptx::smem_addr(&words->tmem), 512);
  if (warp == kSoftWarps + 1 && lane == 0) {
    words->abort = 0;
    words->marked[0] = words->marked[1] = words->marked[2] = 0;
    ptx::prefetch_tensormap(&a.tk);
    ptx::prefetch_tensormap(&a.tv);
    ptx::prefetch_tensormap(&a.tq);
  }
  for (int i = tid; i < t.blocks; i += kThreads) t.single[i + 1] = kUnitCost * a.Hk * a.row_tiles;

  // Lengths, common tokens, and where the items begin in the two concatenated runs.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ps = a.c.page_size, room = a.c.max_blocks * ps;
  for (int i = tid; i < max(a.n, a.n_groups + 1); i += kThreads) {
    const int row = i < a.n ? a.rows[i] : -1;
    const int start = a.n_groups > 0 && i <= a.n_groups ? a.groups[i] : 0;
    const int common = i < a.n_groups ? a.shared[i] : 0;
    int cnt = i < a.n && a.counts != nullptr ? min(max(a.counts[i], 0), a.nodes) : a.nodes;
    int len = 0;
    if (row >= 0 && row < a.c.rows) {
      len = min(a.c.length(row), room);
    } else {
      cnt = 0;
      if (i < a.n && blockIdx.x == 0) atomicOr(a.c.status, QNRE_CACHE_BAD_ROW);
    }
    if (i <= a.n_groups) t.starts[i] = min(max(start, 0), a.n);
    if (i < a.n_groups) t.common[i] = a.by_page(min(max(common, 0), room)) * ps;
    if (i < a.n) {
      t.len[i] = len;
      t.drafts[i] = static_cast<uint8_t>(min(len + cnt, room) - len);
    }
  }
  __syncthreads();
  if (a.n_groups > 0) {
    if (warp == 0) scan_table(t.starts, a.n_groups + 1, true);  // (ascending, whatever is given)
    __syncthreads();
    for (int i = tid; i < a.n; i += kThreads) {
      int lo = -1, hi = a.n_groups - 1;  // the last group that starts by i
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.starts[mid] <= i) lo = mid; else hi = mid - 1;
      }
      const int g = lo >= 0 && i < t.starts[lo + 1] ? lo : -1;
      t.base[i] = g;
      // no more than every member has, in whole pages; nothing where there is only one
      if (g >= 0) atomicMin(&t.common[g], t.starts[g + 1] - t.starts[g] > 1 ? a.by_page(t.len[i]) * ps : 0);
    }
    __syncthreads();
  }
  for (int i = tid; i < a.n; i += kThreads) {
    const int g = a.n_groups > 0 ? t.base[i] : -1;
    const int base = g >= 0 ? t.common[g] : 0;
    t.base[i] = base;
    atomicAdd(&t.single[a.by_members(i) + 1], tiles_of(t.len[i] + t.drafts[i] - base) * a.Hk * a.row_tiles);
    if (blockIdx.x == 0) a.requests[i] = make_int2(base > 0 ? t.starts[g] : -1, base);
  }
  for (int g = kThreads - 1 - tid; g < a.n_groups; g += kThreads) {  // a unit's tiles and its start and end, times units
    const int units = cur.units_of(t.starts[g + 1] - t.starts[g]), full = cur.shared_units(units);
    const int each = t.common[g] > 0 ? (tiles_of(t.common[g]) + kUnitCost) * a.Hk : 0;
    t.single[t.blocks + g + 1] = each * (units - full);
    t.wide[g + 1] = each * a.by_cl(full);
  }
  __syncthreads();
  const int n_single = t.blocks + a.n_groups;
  if (tid == 0) t.single[0] = t.wide[0] = 0;
  if (warp < 2) scan_table((warp == 0 ? t.single : t.wide) + 1, warp == 0 ? n_single : a.n_groups, false);
  __syncthreads();

  // The clusters that share tiles: in proportion to the work, so that the longest run of either kind is the shortest.
  const int W_single = t.single[n_single], W_wide = t.wide[a.n_groups];
  const int clusters = static_cast<int>(gridDim.x) / a.cl;
  int for_wide = 0;
  if (W_wide > 0) {
    // (a single CTA's tile takes a fifth longer: masks, cleaning, and its units' ends come more often)
    const float wide = static_cast<float>(W_wide) * a.cl, single = 1.2f * static_cast<float>(W_single);
    const int low = static_cast<int>(clusters * (wide / (wide + single)));
    auto longest = [&](int c) {
      return c < 1 || c >= clusters ? 3e38f
                                    : fmaxf(static_cast<float>(W_wide) / c,
                                            single / static_cast<float>((clusters - c) * a.cl));
    };
    for_wide = longest(low) <= longest(low + 1) ? low : low + 1;
    for_wide = min(max(for_wide, 1), clusters - 1);
  }
  const int cluster = static_cast<int>(blockIdx.x) / a.cl;
  const bool share = cluster < for_wide;
  cur.wide = share;
  cur.pre = share ? t.wide : t.single;
  cur.rank = share ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int W = share ? W_wide : W_single;
  cur.index = share ? cluster : static_cast<int>(blockIdx.x) - for_wide * a.cl;
  cur.count = min(share ? for_wide : (clusters - for_wide) * a.cl, W);
  cur.quot = W / cur.count;
  cur.rem = W - cur.quot * cur.count;
  cur.cur = cur.index < cur.count ? cur.start_of(cur.index) : 0;
  cur.end = cur.index < cur.count ? cur.start_of(cur.index + 1) : 0;
  if (warp == kSoftWarps + 1 && lane == 0) {
    const uint32_t readers = share ? a.cl : 1;
    for (int i = 0; i < L::kKStages; ++i) {
      ptx::mbar_init(bars.kfull + 8 * i, 1);
      ptx::mbar_init(bars.kempty + 8 * i, readers);
    }
    for (int i = 0; i < L::kVStages; ++i) {
      ptx::mbar_init(bars.vfull + 8 * i, 1);
      ptx::mbar_init(bars.vempty + 8 * i, readers);
    }
    ptx::mbar_init(bars.qfull, 1);
    ptx::mbar_init(bars.qempty, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars.sfull + 8 * i, 1);
      ptx::mbar_init(bars.sfree + 8 * i, kSoftWarps);
      ptx::mbar_init(bars.pready + 8 * i, kSoftWarps);
      ptx::mbar_init(bars.pvdone + 8 * i, 1);
    }
    ptx::mbar_init(bars.ofree, kSoftWarps);
    ptx::mbar_init(bars.drain, 1);
    ptx::mbar_init(bars.drain2, 1);
    ptx::fence_mbar_init();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (a.cl > 1) ptx::cluster_sync();  // every CTA's barriers stand before another sends to it
  ptx::tc_fence_after_sync();
  const uint32_t tmem = words->tmem;
  int lo = 0, hi = (share ? a.n_groups : n_single) - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (cur.pre[mid] <= cur.cur) lo = mid; else hi = mid - 1;
  }
  cur.item = lo;
  Seg first;  // found once for all roles
  const bool more = cur.next(first);

  if (warp < kSoftWarps) {
    run_softmax<L, D, BF16, SCORED>(a, bars, smem_base, tmem, cur, first, more, &words->abort, words->marked);
  } else if (warp == kSoftWarps || warp == kSoftWarps + 3) {
    run_producer<L, D>(a, bars, smem, cur, first, more, warp == kSoftWarps ? 0 : 1, share, &words->abort);
  } else if (warp == kSoftWarps + 1) {
    if (lane == 0) run_scores<L, D, BF16>(a, bars, smem, tmem, cur, first, more, share, &words->abort);
  } else {
    run_outputs<L, D, BF16, SCORED && D == 128>(a, bars, smem_base, tmem, cur, first, more, share, &words->abort, words->marked);
  }
  __syncwarp();
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  if (warp == kSoftWarps) {
    ptx::tmem_relinquish_alloc_permit();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (a.cl > 1) {
    __syncwarp();
    ptx::cluster_sync();  // none leaves while another may still write to it
  }
}

// ------------------------------------------------------------------ join
// The sums of the infinite and NaN elements of V that a row sees among its own tokens, whatever their weights, in columns
// [4 i4, 4 i4 + 4); 0 where there are none.  Eight lanes have the same columns and take every eighth token.
template <int D, bool BF16>
__device__ __noinline__ float4 own_strange(const PrefixArgs& a, int i, int node, int kvh, int i4) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  const int row = a.rows[i], cnt = a.counts != nullptr ? min(max(a.counts[i], 0), a.nodes) : a.nodes;
  if (row >= 0 && row < a.c.rows && node < cnt) {
    const int room = a.c.max_blocks * a.c.page_size, len = min(a.c.length(row), room), total = min(len + cnt, room);
    const uint64_t bits = a.mask != nullptr ? a.mask[static_cast<long long>(i) * a.nodes + node] : (2ull << node) - 1;
#pragma unroll 4
    for (int x = a.requests[i].y + static_cast<int>(threadIdx.x % 8); x < total; x += 8) {
      const int page = a.c.page_of(row, x);  // (a missing one is read as zeros)
      uint2 w = make_uint2(0, 0);
      if (page >= 0) w = *reinterpret_cast<const uint2*>(a.c.v + a.c.token_offset(a.layer, page, kvh, x) + 8 * i4);
      if (((nonfinite_mask<BF16>(w.x) | nonfinite_mask<BF16>(w.y)) == 0) || (x >= len && !(bits >> (x - len) & 1))) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bits16 = (e < 2 ? w.x : w.y) >> (e % 2 * 16) & 0xFFFFu;
        if (nonfinite_mask<BF16>(bits16) & 0xFFFFu) sum[e] += to_float<BF16>(bits16);
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum[e] += __shfl_xor_sync(0xFFFFFFFFu, sum[e], o);
  return make_float4(sum[0], sum[1], sum[2], sum[3]);
}

// A thread has four columns of a row, a warp eight rows' (whole lines of the parts).  Rows go by K head, request, node, head.
// TEAMS of 256 threads take every TEAMS-th part of the block's rows: few rows have many parts.
template <int D, bool BF16, int TEAMS>
__global__ void __launch_bounds__(256 * TEAMS) join_kernel(const __grid_constant__ PrefixArgs a) {
  constexpr int kWarps = D / 16;  // that share eight rows
  __shared__ float sums[TEAMS > 1 ? TEAMS - 1 : 1][7][256];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % 8, team = threadIdx.x / 256;
  const int rr = (blockIdx.x * (8 / kWarps) + warp / kWarps) * 8 + lane % 8;  // (at most 2^31 - 1 rows)
  const int i4 = warp % kWarps * 4 + lane / 8;
  const int per_head = a.n * a.nodes * a.G;
  const bool there = rr < per_head * a.Hk;
  const int kvh = there ? rr / per_head : 0, in_head = there ? rr - kvh * per_head : 0;
  const int token = in_head / a.G, h = in_head - token * a.G;
  const int i = token / a.nodes, node = token - i * a.nodes;
  const int block = node / a.unit_nodes, in_block = node - block * a.unit_nodes;
  const int2 request = a.requests[i];
  auto unit = [&](const Desc* units, int member) { return units[((i - member) * a.Hk + kvh) * a.row_tiles + block]; };
  // places of a unit's runs: p-th run of `d`, whose rows of this request begin at member `member`
  auto row_of = [&](const Desc& d, int member, long long whole, int p) -> long long {
    return d.parts == 0 ? whole + (there ? rr : 0)
                        : static_cast<long long>(2 * (d.cta + p * d.step) + (p == 0 ? 1 : 0)) * 128 +
                              (member * a.unit_nodes + in_block) * a.G + h;
  };
  const int own_member = i % a.unit_members;
  const Desc own = unit(a.row_units, own_member);
  const int own_parts = max(own.parts, 1);
  Desc group{0, 0, 0};
  int group_member = 0, group_parts = 0;
  if (request.x >= 0) {
    group_member = (i - request.x) % a.unit_members;
    group = unit(a.group_units, group_member);
    group_parts = max(group.parts, 1);
  }
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m1, float l1, float4 o1) {
    if (m1 == -INFINITY && l1 == 0.f) return;  // nothing seen
    const float mx = fmaxf(M, m1);
    const float f = M == -INFINITY ? 0.f : part_weight(M - mx), w = m1 == -INFINITY ? 1.f : part_weight(m1 - mx);
    M = mx;
    l = fmaf(l1, w, l * f);
    acc.x = fmaf(o1.x, w, acc.x * f);
    acc.y = fmaf(o1.y, w, acc.y * f);
    acc.z = fmaf(o1.z, w, acc.z * f);
    acc.w = fmaf(o1.w, w, acc.w * f);
  };
  const int parts = group_parts + own_parts;
  bool marked = false;
  for (int p0 = team; p0 < parts; p0 += 4 * TEAMS) {  // four parts' loads at once
    float4 ml[4], v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = min(p0 + k * TEAMS, parts - 1);
      const long long row = p < group_parts ? row_of(group, group_member, a.group_rows, p)
                                            : row_of(own, own_member, a.own_rows, p - group_parts);
      ml[k] = a.part_ml[row];
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (parts > 1 || own.parts > 0) v[k] = a.part_o[piece_of<D>(row, i4)];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = p0 + k * TEAMS;
      if (p >= parts) break;
      if (p >= group_parts && (ml[k].z != 0.f || ml[k].w != 0.f)) marked = true;
      add(ml[k].x, ml[k].y, v[k]);
    }
  }
  if (TEAMS > 1) {  // the teams' sums, in their order
    const int at = threadIdx.x % 256;
    if (team > 0) {
      float(*mine)[256] = sums[team - 1];
      mine[0][at] = M;
      mine[1][at] = l;
      mine[2][at] = acc.x;
      mine[3][at] = acc.y;
      mine[4][at] = acc.z;
      mine[5][at] = acc.w;
      mine[6][at] = marked ? 1.f : 0.f;
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int k = 0; k < TEAMS - 1; ++k) {
      marked |= sums[k][6][at] != 0.f;
      add(sums[k][0][at], sums[k][1][at], make_float4(sums[k][2][at], sums[k][3][at], sums[k][4][at], sums[k][5][at]));
    }
  }
  marked = marked && there && l != 0.f;
  float4 strange = make_float4(0.f, 0.f, 0.f, 0.f);
  for (uint32_t rows = __ballot_sync(0xFFFFFFFFu, marked) & 0xFFu; rows != 0; rows &= rows - 1) {  // the warp's, one after another
    const int from = __ffs(rows) - 1;
    const float4 x = own_strange<D, BF16>(a, __shfl_sync(0xFFFFFFFFu, i, from), __shfl_sync(0xFFFFFFFFu, node, from),
                                          __shfl_sync(0xFFFFFFFFu, kvh, from), i4);
    if (lane % 8 == from) strange = x;
  }
  if (!there) return;
  const bool there_already = request.x < 0 && own.parts == 0;
  if (there_already && !marked) return;
  const long long orow = static_cast<long long>(token) * a.Hq + kvh * a.G + h;
  uint2* dst = reinterpret_cast<uint2*>(a.out + (orow * D + 4 * i4) * 2);
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (marked) {  // infinite and NaN columns, the common tokens' among them; the others are right
    auto join_in = [](float& sum, float x) {
      if (!(fabsf(x) <= 3.4028234664e38f)) sum += x;
    };
    for (int p = 0; p < group_parts; ++p) {
      const long long row = row_of(group, group_member, a.group_rows, p);
      if (a.part_ml[row].x == -INFINITY && a.part_ml[row].y == 0.f) continue;
      const float4 c = a.part_o[piece_of<D>(row, i4)];
      join_in(strange.x, c.x), join_in(strange.y, c.y), join_in(strange.z, c.z), join_in(strange.w, c.w);
    }
    if (there_already) {
      const uint2 w = *dst;
      o = make_float4(to_float<BF16>(w.x & 0xFFFFu), to_float<BF16>(w.x >> 16), to_float<BF16>(w.y & 0xFFFFu),
                      to_float<BF16>(w.y >> 16));
    }
    o = make_float4(strange.x != 0.f ? strange.x : o.x, strange.y != 0.f ? strange.y : o.y, strange.z != 0.f ? strange.z : o.z,
                    strange.w != 0.f ? strange.w : o.w);  // (NaN compares unequal)
  }
  *dst = make_uint2(pack2<BF16>(o.x, o.y), pack2<BF16>(o.z, o.w));
  if (there_already) return;
  if (a.lse != nullptr && i4 == 0) a.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool BF16, bool SMALL, bool SCORED>
qnre_status_t launch_prefix(const PrefixArgs& a, int sms, cudaStream_t stream) {
  const auto kernel = prefix_kernel<D, BF16, SMALL, SCORED>;
  // per device, kept: the raised shared-memory limit, and how many clusters of each size are resident at once
  static std::atomic<uint64_t> ready{0};
  static std::atomic<int> resident[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QNRE_ERR_CUDA;
  dev &= 63;
  if (!(ready.load() >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, SMALL>::kBytes) != cudaSuccess)
      return QNRE_ERR_CUDA;
    ready.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<D, SMALL>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cl;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cl > 1 ? 2 : 1;
  int ctas = std::min(sms, kMaxCtas);
  if (a.cl > 1) {
    int fit = resident[dev][a.cl].load();
    if (fit == 0) {
      cudaLaunchConfig_t ask = cfg;
      ask.gridDim = dim3(kMaxCtas / a.cl * a.cl);
      ask.attrs = attr + 1;
      ask.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&fit, kernel, &ask) != cudaSuccess || fit < 1) return QNRE_ERR_CUDA;
      resident[dev][a.cl].store(fit);
    }
    ctas = std::min(fit, ctas / a.cl) * a.cl;
  }
  if (ctas < 2 * a.cl) return QNRE_ERR_CUDA;  // both kinds of units need a cluster
  cfg.gridDim = dim3(ctas);
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return QNRE_ERR_CUDA;
  constexpr int kJoinRows = 1024 / D;  // a block
  const int64_t rows = static_cast<int64_t>(a.n) * a.nodes * a.Hq;
  const bool few = rows <= kJoinRows * 2 * sms;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kJoinRows - 1) / kJoinRows));
  cfg.blockDim = dim3(few ? 1024 : 256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return from_cuda(few ? cudaLaunchKernelEx(&cfg, join_kernel<D, BF16, 4>, a) : cudaLaunchKernelEx(&cfg, join_kernel<D, BF16, 1>, a));
}

template <int D, bool BF16>
qnre_status_t launch_size(const PrefixArgs& a, bool scored, int sms, cudaStream_t stream) {
  // only D = 128 has a use for the short tables
  const int blocks = (a.n + a.unit_members - 1) / a.unit_members;
  if (D == 128 && a.n <= kSmallRequests && a.n_groups <= kSmallGroups && blocks <= kSmallBlocks) {
    return scored ? launch_prefix<D, BF16, D == 128, true>(a, sms, stream)
                  : launch_prefix<D, BF16, D == 128, false>(a, sms, stream);
  }
  return scored ? launch_prefix<D, BF16, false, true>(a, sms, stream) : launch_prefix<D, BF16, false, false>(a, sms, stream);
}

// The workspace: words of requests and units, the parts of the CTAs' runs, and a place of its own for each row's part over
// its own tokens and, where rows may share, over the common ones.
struct Layout {
  uint64_t requests, row_units, group_units, ml, o, bytes;
  int64_t own_rows, group_rows;
};

Layout layout_of(int64_t n, int64_t nodes, int64_t Hq, int64_t Hk, int D, bool groups) {
  const int64_t unit_nodes = std::min<int64_t>(nodes, kTile / (Hq / Hk)), tiles = (nodes + unit_nodes - 1) / unit_nodes;
  const int64_t slots = 2ll * kMaxCtas * 128, rows = (n * nodes * Hq + 7) / 8 * 8;
  Layout l;
  auto up = [](uint64_t x) { return (x + 15) / 16 * 16; };
  l.requests = 0;
  l.row_units = up(n * sizeof(int2));
  l.group_units = l.row_units + up(n * Hk * tiles * sizeof(Desc));
  l.ml = l.group_units + (groups ? up(n * Hk * tiles * sizeof(Desc)) : 0);
  l.own_rows = slots;
  l.group_rows = slots + rows;
  l.o = l.ml + (slots + (groups ? 2 : 1) * rows) * sizeof(float4);
  l.bytes = l.o + static_cast<uint64_t>(slots + (groups ? 2 * rows : 0)) * D * 4;
  return l;
}

// ------------------------------------------------------------------ the common tokens of groups
constexpr int kSpan = 256;  // blocks of a row that a warp compares at a time

__global__ void __launch_bounds__(1024) shared_prefix_kernel(CacheView c, const int32_t* rows, int n, const int32_t* groups,
                                                             int32_t* shared) {
  __shared__ int common;  // blocks; the first CTA's of the cluster holds the least
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const uint32_t rank = ptx::cluster_ctarank();
  const int g = blockIdx.x / ncta, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int start = min(max(groups[g], 0), n), members = min(max(groups[g + 1], 0), n) - start;
  if (threadIdx.x == 0) common = INT_MAX;
  __syncthreads();
  if (members > 1) {
    const int row0 = rows[start];
    const bool ok0 = row0 >= 0 && row0 < c.rows;
    const int len0 = ok0 ? min(c.length(row0) / c.page_size, c.max_blocks) : 0;
    if (!ok0 && threadIdx.x == 0) atomicOr(c.status, QNRE_CACHE_BAD_ROW);
    const int32_t* table0 = c.table + static_cast<long long>(ok0 ? row0 : 0) * c.max_blocks;
    const int spans = (len0 + kSpan - 1) / kSpan;
    int least = len0;
    // (member, span) pairs over the cluster's warps; the first member's spans find its own missing pages
    for (long long at = rank * 32 + warp; at < static_cast<long long>(members) * max(spans, 1); at += ncta * 32) {
      const int member = static_cast<int>(at % members), b0 = static_cast<int>(at / members) * kSpan;
      const int row = rows[start + member];
      const bool ok = row >= 0 && row < c.rows;
      if (!ok && lane == 0) atomicOr(c.status, QNRE_CACHE_BAD_ROW);
      const int blocks = ok ? min(min(c.length(row) / c.page_size, c.max_blocks), len0) : 0;
      least = min(least, blocks);
      const int32_t* table = c.table + static_cast<long long>(ok ? row : 0) * c.max_blocks;
      int mine[kSpan / 32], first[kSpan / 32];
#pragma unroll
      for (int k = 0; k < kSpan / 32; ++k) {
        const int b = b0 + k * 32 + lane;
        mine[k] = first[k] = -1;
        if (b < blocks) {
          mine[k] = table[b];
          first[k] = table0[b];
        }
      }
#pragma unroll
      for (int k = 0; k < kSpan / 32; ++k) {
        const int b = b0 + k * 32 + lane;
        if (b < blocks && (mine[k] != first[k] || mine[k] < 0 || mine[k] >= c.pages)) least = min(least, b);
      }
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);
    if (lane == 0) atomicMin(&common, least);
  }
  __syncthreads();
  ptx::cluster_sync();
  if (threadIdx.x == 0 && rank != 0 && members > 1)
    asm volatile("red.shared::cluster.min.s32 [%0], %1;" ::"r"(ptx::mapa_shared(ptx::smem_addr(&common), 0)), "r"(common)
                 : "memory");
  __syncwarp();
  ptx::cluster_sync();
  if (threadIdx.x == 0 && rank == 0) shared[g] = members > 1 ? common * c.page_size : 0;
}

}  // namespace

extern "C" {

qnre_status_t qnre_cache_shared_prefix(const qnre_cache_t* cache, const int32_t* rows, int n, const int32_t* groups,
                                       int n_groups, int32_t* shared, qnre_stream_t stream) {
  const qnre_status_t st = check_cache(cache, n);
  if (st != QNRE_OK) return st;
  if (n_groups < 0) return QNRE_ERR_INVALID_ARG;
  if (n_groups > QNRE_MAX_CALL_ROWS) return QNRE_ERR_CAPACITY;
  if (n_groups == 0) return QNRE_OK;
  if ((rows == nullptr && n > 0) || groups == nullptr || shared == nullptr) return QNRE_ERR_INVALID_ARG;
  if (!aligned(rows, 4) || !aligned(groups, 4) || !aligned(shared, 4)) return QNRE_ERR_ALIGNMENT;
  const ByteRange w = span(shared, static_cast<uint64_t>(n_groups) * 4);
  const ByteRange in[] = {span(rows, static_cast<uint64_t>(n) * 4), span(groups, (static_cast<uint64_t>(n_groups) + 1) * 4),
                          span(cache->block_table, static_cast<uint64_t>(cache->rows) * cache->max_blocks * 4),
                          span(cache->seq_lens, static_cast<uint64_t>(cache->rows) * 4),
                          span(cache->page_refs, static_cast<uint64_t>(cache->pages) * 4), span(cache->status, 4),
                          span(cache->scratch, scratch_bytes(cache)),
                          span(cache->k, pool_bytes(cache)), span(cache->v, pool_bytes(cache))};
  for (const ByteRange& r : in)
    if (overlaps(w, r)) return QNRE_ERR_ALIAS;
  cudaLaunchConfig_t cfg{};
  // few groups: several CTAs each, about as many as one a SM
  unsigned cluster = 8;
  while (cluster > 1 && n_groups * cluster > 152) cluster /= 2;
  cfg.gridDim = dim3(n_groups * cluster);
  cfg.blockDim = dim3(1024);
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
  return from_cuda(cudaLaunchKernelEx(&cfg, shared_prefix_kernel, view_of(cache), rows, n, groups, shared));
}

qnre_status_t qnre_prefix_attention_workspace_bytes(int n, int nodes, int q_heads, int kv_heads, int head_dim, int n_groups,
                                                    uint64_t* bytes) {
  if (bytes == nullptr || n < 0 || nodes < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || n_groups < 0)
    return QNRE_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || q_heads / kv_heads > kTile) return QNRE_ERR_UNSUPPORTED;
  if (n > QNRE_MAX_CALL_ROWS || nodes > QNRE_MAX_NODES || q_heads > 65535) return QNRE_ERR_CAPACITY;
  *bytes = layout_of(n, std::max(nodes, 1), q_heads, kv_heads, head_dim, n_groups > 0).bytes;
  return QNRE_OK;
}

qnre_status_t qnre_prefix_attention(const qnre_tensor4_t* q, const qnre_cache_t* cache, int layer, const int32_t* rows,
                                    const int32_t* groups, int n_groups, const int32_t* shared, const uint64_t* mask,
                                    const int32_t* depths, const int32_t* counts, float scale, float softcap,
                                    const float* slopes, void* out, float* lse, void* workspace, uint64_t workspace_bytes,
                                    qnre_stream_t stream) {
  if (q == nullptr) return QNRE_ERR_INVALID_ARG;
  qnre_tensor4_t own = *q;
  alignas(16) static char nothing[16];
  const bool empty = own.shape[0] == 0 || own.shape[1] == 0;
  if (own.data == nullptr && empty) own.data = nothing;
  ByteRange rq;
  qnre_status_t st = check_view(&own, &rq);
  if (st == QNRE_OK) st = check_cache(cache, static_cast<int>(std::min<int64_t>(own.shape[0], 0x7FFFFFFF)));
  if (st != QNRE_OK) return st;
  if (own.dtype != cache->dtype || own.shape[3] != cache->head_dim || own.shape[2] % cache->heads != 0 || layer < 0 ||
      layer >= cache->layers || !(scale > 0.f) || !std::isfinite(scale) || !(softcap >= 0.f) || !std::isfinite(softcap) ||
      n_groups < 0)
    return QNRE_ERR_INVALID_ARG;
  if (softcap > 0.f && !(softcap >= 1e-30f && std::isfinite(scale / softcap))) return QNRE_ERR_UNSUPPORTED;
  if (own.shape[2] / cache->heads > kTile) return QNRE_ERR_UNSUPPORTED;
  if (own.shape[1] > QNRE_MAX_NODES || own.shape[2] > 65535 || n_groups > QNRE_MAX_CALL_ROWS) return QNRE_ERR_CAPACITY;
  if (!rows_vectorisable(&own, 2)) return QNRE_ERR_ALIGNMENT;
  if (empty) return QNRE_OK;
  if (rows == nullptr || out == nullptr || workspace == nullptr || (n_groups > 0 && (groups == nullptr || shared == nullptr)))
    return QNRE_ERR_INVALID_ARG;
  if (!aligned(rows, 4) || !aligned(groups, 4) || !aligned(shared, 4) || !aligned(counts, 4) || !aligned(depths, 4) ||
      !aligned(slopes, 4) || !aligned(mask, 8) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
    return QNRE_ERR_ALIGNMENT;
  const int n = static_cast<int>(own.shape[0]), nodes = static_cast<int>(own.shape[1]), Hq = static_cast<int>(own.shape[2]);
  const Layout l = layout_of(n, nodes, Hq, cache->heads, cache->head_dim, n_groups > 0);
  if (workspace_bytes < l.bytes) return QNRE_ERR_CAPACITY;
  const uint64_t tokens = static_cast<uint64_t>(n) * nodes, out_rows = tokens * Hq;
  auto words = [](const void* p, uint64_t bytes) { return p != nullptr ? span(p, bytes) : ByteRange{0, 0}; };
  const ByteRange writes[] = {span(out, out_rows * cache->head_dim * 2), words(lse, out_rows * 4), span(workspace, l.bytes)};
  const ByteRange reads[] = {rq,
                             span(cache->k, pool_bytes(cache)),
                             span(cache->v, pool_bytes(cache)),
                             span(rows, static_cast<uint64_t>(n) * 4),
                             n_groups > 0 ? words(groups, (static_cast<uint64_t>(n_groups) + 1) * 4) : ByteRange{0, 0},
                             n_groups > 0 ? words(shared, static_cast<uint64_t>(n_groups) * 4) : ByteRange{0, 0},
                             words(mask, tokens * 8),
                             words(depths, tokens * 4),
                             words(counts, static_cast<uint64_t>(n) * 4),
                             words(slopes, static_cast<uint64_t>(Hq) * 4),
                             span(cache->block_table, static_cast<uint64_t>(cache->rows) * cache->max_blocks * 4),
                             span(cache->seq_lens, static_cast<uint64_t>(cache->rows) * 4),
                             span(cache->page_refs, static_cast<uint64_t>(cache->pages) * 4),
                             span(cache->status, 4),
                             span(cache->scratch, scratch_bytes(cache))};
  for (int i = 0; i < 3; ++i) {
    for (const ByteRange& r : reads)
      if (overlaps(writes[i], r)) return QNRE_ERR_ALIAS;
    if (overlaps(writes[i], writes[(i + 1) % 3])) return QNRE_ERR_ALIAS;
  }

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QNRE_ERR_CUDA;
  if (!own_memory(cache->k, dev) || !own_memory(cache->v, dev)) return QNRE_ERR_INVALID_ARG;

  PrefixArgs a{};
  a.c = view_of(cache);
  a.layer = layer;
  a.n = n;
  a.n_groups = n_groups;
  a.nodes = nodes;
  a.Hq = Hq;
  a.Hk = cache->heads;
  a.G = a.Hq / a.Hk;
  a.unit_nodes = std::min(nodes, kTile / a.G);
  a.row_tiles = (nodes + a.unit_nodes - 1) / a.unit_nodes;
  a.unit_members = a.row_tiles > 1 ? 1 : std::max(1, kTile / a.G / nodes);
  a.warp_members = std::max(1, 32 / (a.G * a.unit_nodes));
  a.by_page = Divisor::of(cache->page_size);
  a.by_G = Divisor::of(a.G);
  a.by_nodes = Divisor::of(a.unit_nodes);
  a.by_members = Divisor::of(a.unit_members);
  a.by_tiles = Divisor::of(a.row_tiles);
  // CTAs of a cluster: the units that a group of average size has for a K head
  const int members = n_groups > 0 ? (n + n_groups - 1) / n_groups : 0;
  const int units = (members + a.unit_members - 1) / a.unit_members * a.row_tiles;
  a.cl = std::min(std::max(units, 1), kMaxCluster);
  a.by_cl = Divisor::of(a.cl);
  const int64_t tiles = (static_cast<int64_t>(cache->max_blocks) * cache->page_size + kTile - 1) / kTile + kUnitCost;
  if (2 * a.n * tiles * a.Hk * a.row_tiles > 0x7FFFFFFF || static_cast<int64_t>(out_rows) > 0x7FFFFF00) return QNRE_ERR_CAPACITY;
  a.box = std::min(a.cl > 1 ? kTile / kMaxCluster : kTile, cache->page_size & -cache->page_size);
  a.rows = rows;
  a.groups = groups;
  a.shared = shared;
  a.counts = counts;
  a.depths = depths;
  a.mask = mask;
  a.slopes = slopes;
  a.backward = slopes != nullptr;
  a.out = static_cast<char*>(out);
  a.lse = lse;
  char* ws = static_cast<char*>(workspace);
  a.requests = reinterpret_cast<int2*>(ws + l.requests);
  a.row_units = reinterpret_cast<Desc*>(ws + l.row_units);
  a.group_units = reinterpret_cast<Desc*>(ws + l.group_units);
  a.part_ml = reinterpret_cast<float4*>(ws + l.ml);
  a.part_o = reinterpret_cast<float4*>(ws + l.o);
  a.own_rows = l.own_rows;
  a.group_rows = l.group_rows;
  a.scale_log2 = scale * kLog2e;
  a.cap_log2 = softcap * kLog2e;
  a.cap_in = softcap > 0.f ? scale / softcap : 0.f;
  constexpr double kNear[3] = {-0.33332663774490356, 0.1329982578754425, -0.04914848133921623};
  a.cap_near = 0.35f;
  double power = 1.0;
  for (int i = 0; i < 3; ++i) {
    power *= static_cast<double>(a.cap_in) * a.cap_in;
    a.cap_poly[i] = static_cast<float>(kNear[i] * power);
    if (!std::isnormal(a.cap_poly[i])) a.cap_near = -1.f;  // (a cap of a millionth, or of thousands)
  }
  const bool bf16 = cache->dtype == QNRE_DTYPE_BF16;
  const uint64_t D = cache->head_dim, ps = cache->page_size, H = cache->heads;
  const uint64_t dims[4] = {D, ps, H, static_cast<uint64_t>(cache->layers) * cache->pages};
  const uint64_t strides[3] = {D * 2, ps * D * 2, H * ps * D * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(a.box), 1, 1};
  const uint64_t q_dims[4] = {D, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.nodes), static_cast<uint64_t>(a.n)};
  const uint64_t q_strides[3] = {static_cast<uint64_t>(own.stride[2]) * 2, static_cast<uint64_t>(own.stride[1]) * 2,
                                 static_cast<uint64_t>(own.stride[0]) * 2};
  const uint32_t q_box[4] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(a.unit_nodes),
                             static_cast<uint32_t>(a.unit_members)};
  if (!encode_tiled_16bit(&a.tq, own.data, bf16, 4, q_dims, q_strides, q_box) ||
      !encode_tiled_16bit(&a.tk, cache->k, bf16, 4, dims, strides, box) ||
      !encode_tiled_16bit(&a.tv, cache->v, bf16, 4, dims, strides, box))
    return QNRE_ERR_CUDA;
  const bool scored = softcap > 0.f || slopes != nullptr;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) return bf16 ? launch_size<128, true>(a, scored, sms, s) : launch_size<128, false>(a, scored, sms, s);
  return bf16 ? launch_size<64, true>(a, scored, sms, s) : launch_size<64, false>(a, scored, sms, s);
}

}  // extern "C"
