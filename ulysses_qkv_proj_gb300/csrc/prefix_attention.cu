// prefix_attention.cu -- attention over a paged cache whose rows share their leading pages (samples, drafts or requests
// of one prompt): the common tokens are read once for the whole group.  Scores may be capped by a tanh and get a bias
// that falls with distance.
//
//   o = sum_x p_x v_x,  p = softmax(cap tanh(scale q.k_x / cap) + slope (pos_x - pos_q)) over the tokens a node sees
//
// A softmax over two sets of tokens is the join of two softmaxes, so each row has two parts: its group's common tokens,
// where all members' nodes and query heads of a K head are rows of one matrix product (128 to a unit, several units
// to a cluster that fetches K and V for all of them by multicast), and its own tokens behind them.  Both are cut into units and
// tiles as in tree_attention.cu and dealt out in equal runs; whole clusters take one kind or the other, in the
// proportion of their tiles, so that both kinds run side by side in one launch.  A second kernel joins a row's parts: the
// group's, in the order of its tiles, then its own.  Everything is found from lengths in device memory by each CTA itself
// (the number of common tokens too), so a captured call follows them, and the order of sums depends on them alone.
//
// In a CTA the roles are those of tree_attention.cu: two TMA warps, two threads that issue the products, eight softmax
// warps of which two threads share a row of 128.  Few rows leave lanes idle, which costs nothing where HBM is the limit.
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
constexpr int kSmall = 64;    // requests whose table is short enough for a third V tile at D = 128
constexpr int kSmallLen = 1 << 24;
constexpr float kLog2e = 1.4426950408889634f;

// Where a unit's results are: `parts` runs of it from CTA `cta` on; 0: one piece, in the rows' own places; -1: in the output.
struct Desc {
  int cta, parts;
};

struct PrefixArgs {
  CUtensorMap tk, tv, tq_group, tq_row;
  CacheView c;
  const int32_t *rows, *groups, *shared, *counts, *depths;
  const uint64_t* mask;
  const float* slopes;
  char* out;
  float* lse;
  int* first_of;      // [n]: the first request of the group whose common tokens a request reads, or -1
  Desc* row_units;    // [n][Hk][row_tiles]
  Desc* group_units;  // [n][Hk][row_tiles], by the first request of the unit
  float2* part_ml;    // [2 kMaxCtas 128 + rows of both kinds]: maximum (base 2), sum
  float4* part_o;     // the same rows of D, laid out by piece_of
  long long own_rows, group_rows;  // where the rows' own places begin, for each kind
  float scale_log2, cap_in, cap_log2;  // capped: 2 log2(e) scale / cap, cap log2(e)
  int layer, n, n_groups, nodes, Hq, Hk, G, box, cl;
  int unit_nodes, unit_members, row_tiles;  // nodes and members of a unit; tiles of one request's nodes
};

// Eight rows' pieces of 16 bytes lie side by side, so that the threads that write, a row each, fill whole lines.
template <int D>
__device__ __forceinline__ long long piece_of(long long row, int i) {
  return ((row >> 3) * (D / 4) + i) * 8 + (row & 7);
}

// Shared memory: as many tiles of K and V in flight as fit.
template <int D, bool SMALL>
struct Smem {
  static constexpr int kRequests = SMALL ? kSmall : QNRE_MAX_CALL_ROWS;
  static constexpr int kKStages = D == 128 ? 3 : 5;
  static constexpr int kVStages = D == 128 ? (SMALL ? 3 : 2) : 5;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kTileBytes;
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kMl = kV + kVStages * kTileBytes;   // float [2][2][128]
  static constexpr int kItems = kMl + 2048;                // int2 [kRequests]
  static constexpr int kExtra = kItems + kRequests * 8;    // int [kRequests] (SMALL: in the items)
  static constexpr int kPre = kExtra + (SMALL ? 0 : kRequests * 4);  // int [kRequests + 1]
  static constexpr int kBars = (kPre + (kRequests + 1) * 4 + 7) / 8 * 8;
  static constexpr int kWords = kBars + 8 * (2 * kKStages + 2 * kVStages + 13);
  static constexpr int kBytes = kWords + 32;
  static_assert(kBytes <= 232448, "one CTA's shared memory");
  static_assert(6 * (QNRE_MAX_CALL_ROWS + 1) * 4 <= kKStages * kTileBytes, "the first tables lie where K will");
};

struct Words {
  unsigned long long bad_nodes[3];  // drafts with non-finite V elements, segments in turn
  uint32_t tmem, abort;
};

struct Bars {
  uint32_t kfull, kempty, vfull, vempty, qfull, qempty, sfull, sfree, pready, pvdone, ofree, drain, drain2;
};

// One unit's part of a CTA's run.
struct Seg {
  int item, kvh, rt, t0, t1;
  int base, len, total;  // its tokens: context [base, len), drafts up to total
  int start, members;    // of a group
  int begin;             // the run's place of its first tile
  bool whole;
  int slot;
};

// A CTA's run over the units of its kind.
template <bool SMALL>
struct Cursor {
  const int* pre;
  const int2* items;
  const int* extra;
  int cur, end, item, cl, rank, row_tiles, unit_members, index, count, quot, rem;  // run `index` of `count`
  bool group;

  __device__ __forceinline__ static int tiles_of(int tokens) { return tokens > 0 ? (tokens + kTile - 1) / kTile : 1; }
  __device__ __forceinline__ static int clusters_of(int members, int unit_members, int row_tiles, int cl) {
    return ((members + unit_members - 1) / unit_members * row_tiles + cl - 1) / cl;
  }
  __device__ __forceinline__ int start_of(int c) const { return c * quot + c * rem / count; }
  __device__ __forceinline__ bool next(Seg& s) {
    while (cur < end) {
      while (cur >= pre[item + 1]) ++item;
      const int2 it = items[item];
      s.item = item;
      if (group) {
        s.base = 0;
        s.start = it.x >> 16;
        s.members = it.x & 0xFFFF;
        s.len = s.total = it.y;
      } else {
        s.base = it.x;
        s.len = SMALL ? it.y >> 7 : it.y;
        s.total = s.len + (SMALL ? it.y & 127 : extra[item]);
        s.start = item;
        s.members = 1;
      }
      const int tiles = tiles_of(s.total - s.base), per = tiles + kUnitCost;
      const int off = cur - pre[item];
      const int unit = off / per, o = off - unit * per;
      const int take = min(per - o, end - cur);
      s.begin = cur - o + kUnitCost;
      cur += take;
      s.t0 = max(0, o - kUnitCost);
      s.t1 = max(0, o + take - kUnitCost);
      if (s.t0 == s.t1) continue;  // the unit's cost falls to this CTA, its tiles to the next
      const int per_head = group ? clusters_of(s.members, unit_members, row_tiles, cl) : row_tiles;
      s.kvh = unit / per_head;
      s.rt = (unit - s.kvh * per_head) * cl + rank;
      s.whole = s.t0 == 0 && s.t1 == tiles;
      // a CTA goes on with one unit at most, and leaves one unfinished at most
      s.slot = 2 * static_cast<int>(blockIdx.x) + (s.t0 == 0 ? 1 : 0);
      return true;
    }
    return false;
  }
};

// What row `ur` of a unit stands for.
struct UnitRow {
  int request, node, head;
  bool there;
};
__device__ __forceinline__ UnitRow unit_row(const PrefixArgs& a, const Seg& s, bool group, int ur) {
  const int q = ur / a.G;
  UnitRow r;
  if (group) {
    const int tile = s.rt / a.row_tiles, block = s.rt - tile * a.row_tiles;
    const int mi = q / a.unit_nodes, member = tile * a.unit_members + mi;
    r.node = block * a.unit_nodes + q - mi * a.unit_nodes;
    r.request = s.start + member;
    r.there = mi < a.unit_members && member < s.members && r.node < a.nodes;
  } else {
    r.node = s.rt * a.unit_nodes + q;
    r.request = s.item;
    r.there = q < a.unit_nodes && r.node < a.nodes;
  }
  r.head = s.kvh * a.G + ur - q * a.G;
  return r;
}

// Among the softmax threads.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }

// ------------------------------------------------------------------ TMA warps
// One warp brings Q and K, another V.  With `share` each CTA of the cluster fetches its share of a tile's boxes for all.
template <typename L, int D, bool SMALL>
__device__ void run_producer(const PrefixArgs& a, const Bars& bars, uint32_t smem, Cursor<SMALL> cur, Seg s, bool more,
                             int kv, bool share, volatile uint32_t* abort_flag) {
  constexpr int kHalves = D / 64;
  const int lane = threadIdx.x % 32;
  const int chunk = lane / kHalves, half = lane % kHalves;
  const bool active = chunk < kTile / a.box && (!share || lane % a.cl == cur.rank);
  const int ps = a.c.page_size, step = kTile / ps, step_off = kTile - step * ps;
  const int none = a.c.layers * a.c.pages;  // past the end: the box is filled with zeros
  const uint16_t everyone = static_cast<uint16_t>((1u << a.cl) - 1u);
  const CUtensorMap* map = kv ? &a.tv : &a.tk;
  const CUtensorMap* q_map = cur.group ? &a.tq_group : &a.tq_row;
  const uint32_t dst = smem + (kv ? L::kV : L::kK) + half * (kTile * 128) + chunk * a.box * 128;
  const uint32_t q_bytes = static_cast<uint32_t>(D * 2 * a.G * a.unit_nodes * (cur.group ? a.unit_members : 1));
  const uint32_t full = kv ? bars.vfull : bars.kfull, empty = kv ? bars.vempty : bars.kempty;
  const uint32_t stages = kv ? L::kVStages : L::kKStages;
  uint32_t slot = 0, phase = 1;
  auto settle = [] {  // stop: what is in flight lands in microseconds; the kernel's end waits for it
    const uint64_t t0 = ptx::global_timer_ns();
    while (ptx::global_timer_ns() - t0 < 50000) {
    }
  };
  for (uint32_t seg = 0; more; ++seg, more = cur.next(s)) {
    const int row = a.rows[s.start];
    const bool fetches = active && row >= 0 && row < a.c.rows;
    const int32_t* table = a.c.table + static_cast<long long>(fetches ? row : 0) * a.c.max_blocks;
    int pos = s.base + s.t0 * kTile + chunk * a.box;
    int block = pos / ps, off = pos - block * ps;
    auto look = [&]() -> int { return fetches && pos < s.total && block < a.c.max_blocks ? __ldg(table + block) : -1; };
    int entry = look();
    if (kv == 0) {  // the unit's Q rows (one buffer: the last unit's scores are done)
      if (!wait(bars.qempty, (seg & 1u) ^ 1u, abort_flag, a.c.status)) return settle();
      if (lane == 0) ptx::mbar_arrive_expect_tx(bars.qfull, q_bytes);
      __syncwarp();
      const int tile = cur.group ? s.rt / a.row_tiles : 0;
      const int node = (s.rt - tile * a.row_tiles) * a.unit_nodes, request = s.start + tile * a.unit_members;
      if (lane < kHalves)
        tma_load_4d(smem + L::kQ + lane * (kTile * 128), q_map, bars.qfull, lane * 64, s.kvh * a.G, node, request);
    }
    for (int t = s.t0; t < s.t1; ++t) {
      const bool there = entry >= 0 && entry < a.c.pages;
      if (fetches && !there && pos < s.total) atomicOr(a.c.status, QNRE_CACHE_BAD_PAGE);
      const int page = there ? a.layer * a.c.pages + entry : none, at = off;
      pos += kTile;
      block += step;
      off += step_off;
      if (off >= ps) {
        off -= ps;
        ++block;
      }
      entry = look();  // on its way while this tile's place is waited for
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
template <typename L, int D, bool BF16, bool SMALL>
__device__ void run_scores(const PrefixArgs& a, const Bars& bars, uint32_t smem, uint32_t tmem, Cursor<SMALL> cur, Seg s,
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

// O += P V, tile after tile; names the places of the units begun here for the join.
template <typename L, int D, bool BF16, bool SMALL>
__device__ void run_outputs(const PrefixArgs& a, const Bars& bars, uint32_t smem, uint32_t tmem, Cursor<SMALL> cur, Seg s,
                            bool more, bool share, volatile uint32_t* abort_flag) {
  constexpr uint32_t kFmt = BF16 ? (1u << 7 | 1u << 10) : 0u;
  constexpr uint32_t kIdesc =
      (1u << 4) | kFmt | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24);
  const uint64_t ring0 = ptx::smem_desc_sw128(smem + L::kV, kTile * 128, 1024);
  const uint16_t everyone = static_cast<uint16_t>((1u << a.cl) - 1u);
  uint32_t g = 0, slot = 0, phase = 0;
  for (uint32_t seg = 0; more; ++seg, more = cur.next(s)) {
    if (s.t0 == 0) {
      int parts = !cur.group && s.base == 0 ? -1 : 0;
      if (!s.whole) {
        const int last = s.begin + Cursor<SMALL>::tiles_of(s.total - s.base) - 1;
        int lo = cur.index, hi = cur.count - 1;  // the last run that starts by the last tile
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (cur.start_of(mid) <= last) lo = mid; else hi = mid - 1;
        }
        parts = lo - cur.index + 1;
      }
      const Desc d{static_cast<int>(blockIdx.x), parts};
      const int tile = cur.group ? s.rt / a.row_tiles : 0, block = s.rt - tile * a.row_tiles;
      const int request = s.start + tile * a.unit_members;
      if (tile * a.unit_members < s.members)
        (cur.group ? a.group_units : a.row_units)[(request * a.Hk + s.kvh) * a.row_tiles + block] = d;
    }
    for (int t = s.t0; t < s.t1; ++t, ++g) {
      const uint32_t b = g & 1u;
      const bool first = t == s.t0;
      if (!wait(bars.vfull + 8 * slot, phase, abort_flag, a.c.status) ||
          (first && !wait(bars.ofree, (seg & 1u) ^ 1u, abort_flag, a.c.status)) ||
          !wait(bars.pready + 8 * b, (g >> 1) & 1u, abort_flag, a.c.status))
        return drain_mma(bars.drain2);
      ptx::tc_fence_after_sync();
      const uint64_t v = desc_at(ring0, slot * L::kTileBytes);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk)
        umma_f16_ts(tmem + kTmemO, tmem + kTmemP + b * 64 + kk * 8, desc_at(v, kk * 2048), kIdesc,
                    (t > s.t0 || kk > 0) ? 1u : 0u);
      ptx::umma_commit(bars.pvdone + 8 * b);
      release(bars.vempty + 8 * slot, share, everyone);
      if (++slot == L::kVStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

// ------------------------------------------------------------------ softmax warps
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two threads a row, half a tile each.  SCORED: scores are capped or biased, and come out in base 2; else the scale is
// applied with the maximum.
template <typename L, int D, bool BF16, bool SMALL, bool SCORED>
__device__ void run_softmax(const PrefixArgs& a, const Bars& bars, char* smem_base, uint32_t tmem, Cursor<SMALL> cur,
                            Seg next, bool more, volatile uint32_t* abort_flag, unsigned long long* bad_nodes) {
  constexpr int kCols = kTile / 2, kOut = D / 2;  // tokens of a tile, columns of O this thread has
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int ur = tid % 128, copy = tid / 128, c0 = copy * kCols, o0 = copy * kOut;
  const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
  float* ml = reinterpret_cast<float*>(smem_base + L::kMl);
  const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
  const int room = a.c.max_blocks * a.c.page_size;

  // what this thread's row of a segment is
  struct RowInfo {
    UnitRow at;
    bool row_ok;    // of a node that sees anything
    uint64_t bits;  // the drafts it sees
    int place;      // its position
    float slope;    // in base 2
  };
  auto row_info = [&](const Seg& s) {
    RowInfo r{unit_row(a, s, cur.group, ur), false, 0, 0, 0.f};
    if (!r.at.there) return r;
    const int i = r.at.request;
    r.row_ok = a.counts == nullptr || r.at.node < a.counts[i];
    if (!cur.group)
      r.bits = a.mask != nullptr ? a.mask[static_cast<long long>(i) * a.nodes + r.at.node] : (2ull << r.at.node) - 1;
    if (SCORED && a.slopes != nullptr) {
      r.slope = a.slopes[r.at.head] * kLog2e;
      const int row = cur.group ? a.rows[i] : 0;
      const int len = cur.group ? (row >= 0 && row < a.c.rows ? min(a.c.length(row), room) : 0) : s.len;
      r.place = len + (a.depths != nullptr ? a.depths[static_cast<long long>(i) * a.nodes + r.at.node] : r.at.node);
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
    const int slots = s.total - s.len;  // drafts that have a place
    const uint64_t bits = slots < 64 ? row.bits & ((1ull << slots) - 1) : row.bits;
    const int table_row = a.rows[s.start];
    float m = -INFINITY, l = 0.f;
    for (int t = s.t0; t < s.t1; ++t, ++g) {
      const uint32_t b = g & 1u;
      const int pos0 = s.base + t * kTile;
      uint32_t v[kCols / 32][32];
      wait(bars.pvdone + 8 * b, ((g >> 1) & 1u) ^ 1u, abort_flag, a.c.status);
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

      const bool tail = pos0 + kTile > s.len;
      if (SCORED) {
        if (a.cap_log2 > 0.f) {  // tanh x = 1 - 2 / (1 + e^2x): to 2^-23 of the cap, however large the score
#pragma unroll
          for (int i = 0; i < kCols; ++i) {
            const float e = exp2_fast(__uint_as_float(v[i / 32][i % 32]) * a.cap_in);
            v[i / 32][i % 32] = __float_as_uint(fmaf(rcp_fast(e + 1.f), -2.f * a.cap_log2, a.cap_log2));
          }
        } else {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            v[i / 32][i % 32] = __float_as_uint(__uint_as_float(v[i / 32][i % 32]) * a.scale_log2);
        }
        if (a.slopes != nullptr) {
          const int d0 = pos0 + c0;
          const float at0 = row.slope * static_cast<float>(d0 - row.place);
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            v[i / 32][i % 32] = __float_as_uint(__uint_as_float(v[i / 32][i % 32]) + fmaf(row.slope, static_cast<float>(i), at0));
          if (tail && a.depths != nullptr && !cur.group) {  // a draft lies at its depth, not at its slot
#pragma unroll 1
            for (int j = max(s.len - d0, 0); j < min(s.total - d0, kCols); ++j) {
              const int node = d0 + j - s.len;
              const float off = row.slope * static_cast<float>(a.depths[static_cast<long long>(s.item) * a.nodes + node] - node);
#pragma unroll
              for (int i = 0; i < kCols; ++i)
                if (i == j) v[i / 32][i % 32] = __float_as_uint(__uint_as_float(v[i / 32][i % 32]) + off);
            }
          }
        }
      }
      if (tail) {
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j) {
          const uint32_t see = seen_word(pos0 + c0 + 32 * j - s.len, bits);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(see & (1u << i))) v[j][i] = 0xFF800000u;
        }
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < kCols / 32; ++j)
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          mx0 = max3(mx0, __uint_as_float(v[j][i]), __uint_as_float(v[j][i + 1]));
          mx1 = max3(mx1, __uint_as_float(v[j][i + 2]), __uint_as_float(v[j][i + 3]));
        }
      float mx = fmaxf(mx0, mx1) * (SCORED ? 1.f : a.scale_log2);
      {  // with the other half's; two buffers, as the next tile's may be written before this is read
        float* at = ml + b * 256 + ur;
        at[copy * 128] = mx;
        pair_sync(warp % 4);
        mx = fmaxf(mx, at[(copy ^ 1) * 128]);
      }
      mx -= kLift<BF16>;  // m: the row's maximum less the lift, which leaves O / l and m + log2 l as they are
      const bool grow = mx > m + kRescale;
      if (t == s.t0) {
        m = mx;
      } else if (__any_sync(0xFFFFFFFFu, grow)) {
        const uint32_t last = g - 1;
        wait(bars.pvdone + 8 * (last & 1u), (last >> 1) & 1u, abort_flag, a.c.status);
        __syncwarp();
        ptx::tc_fence_after_sync();
        const float f = grow ? exp2_fast(m - mx) : 1.f;
        if (grow) m = mx;
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
      const float ms = m == -INFINITY ? 0.f : m;
      const uint64_t neg = pair(-ms, -ms);
      uint32_t p[kCols / 2];
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) {
        float e0, e1;
        const uint64_t x = pair(__uint_as_float(v[i / 16][(2 * i) % 32]), __uint_as_float(v[i / 16][(2 * i + 1) % 32]));
        unpair(SCORED ? add2(x, neg) : fma2(x, scale2, neg), e0, e1);
        e0 = exp2_fast(e0);
        e1 = exp2_fast(e1);
        sum[i & 1] = add2(sum[i & 1], pair(e0, e1));
        p[i] = pack2<BF16>(e0, e1);
      }
      {
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      tmem_st_x32(tmem + lane_base + kTmemP + b * 64 + c0 / 2, p);
      if (tail) {
        const uint32_t slot = g % L::kVStages;
        wait(bars.vfull + 8 * slot, (g / L::kVStages) & 1u, abort_flag, a.c.status);
        const int x = tid % 128, pos = pos0 + x;
        constexpr int kPieces = D / 16;
        if (pos >= s.len && clean_v_row<D, BF16>(smem_base + L::kV + slot * L::kTileBytes + x * 128, pos < s.total,
                                                 copy * kPieces, (copy + 1) * kPieces))
          atomicOr(bad_nodes + seg % 3, 1ull << (pos - s.len));
        __syncwarp();
      }
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
    ml[(g & 1u) * 256 + tid] = l;  // (the buffer that the last tile did not use)
    const uint32_t last = g - 1;
    wait(bars.pvdone + 8 * (last & 1u), (last >> 1) & 1u, abort_flag, a.c.status);
    soft_sync();
    ptx::tc_fence_after_sync();
    // every warp has read the word of the segment before, and none uses it again before the next segment's end
    if (tid == 0) bad_nodes[(seg + 2) % 3] = 0;
    const uint64_t bad = row_ok ? bad_nodes[seg % 3] & bits : 0;
    l += ml[(g & 1u) * 256 + (tid ^ 128)];
    pair_sync(warp % 4);  // read by both before the next tile's maxima go there
    const bool done = s.whole && !cur.group && s.base == 0;  // no other part of these rows
    const float inv = !done ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
    const long long token = static_cast<long long>(row.at.request) * a.nodes + row.at.node;
    const long long orow = token * a.Hq + row.at.head;
    const int head = row.at.head - s.kvh * a.G;
    const long long prow =
        s.whole ? (cur.group ? a.group_rows : a.own_rows) +
                      (static_cast<long long>(s.kvh) * a.n * a.nodes + token) * a.G + head
                : static_cast<long long>(s.slot) * 128 + ur;
#pragma unroll 1
    for (int c = o0; c < o0 + kOut; c += 32) {
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
      if (__any_sync(0xFFFFFFFFu, row_ok && odd0 + odd1 != 0.f)) {  // (NaN compares unequal)
        const Kinds k = search_context<BF16>(a.c, a.layer, table_row, s.kvh, s.base + s.t0 * kTile,
                                             min(s.base + s.t1 * kTile, s.len), c);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t bit = 1u << i;
          if ((k.plus | k.minus | k.nan) & bit)
            x[i] = (k.nan | (k.plus & k.minus)) & bit ? NAN : (k.plus & bit ? INFINITY : -INFINITY);
        }
      }
      if (bad != 0) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          x[i] = add_nonfinite<BF16>(a.c, a.layer, table_row, s.kvh, s.len, s.base + s.t0 * kTile, s.base + s.t1 * kTile,
                                     bad, c + i, x[i]);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = row_ok ? x[i] * inv : 0.f;
      if (in_out && done) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack2<BF16>(x[2 * e], x[2 * e + 1]);
        uint4* dst = reinterpret_cast<uint4*>(a.out + (orow * D + c) * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      } else if (in_out) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          a.part_o[piece_of<D>(prow, c / 4 + i)] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
      __syncwarp();
    }
    if (in_out && copy == 0) {
      if (!done)
        a.part_ml[prow] = make_float2(m, l);
      else if (a.lse != nullptr)
        a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
}

// Running sums (or maxima) of x[1 .. n], by one warp.
template <bool MAXIMUM>
__device__ __forceinline__ void scan_table(int* x, int n) {
  const int lane = threadIdx.x % 32;
  int carry = 0;
  for (int base = 0; base < n; base += 32) {
    int v = base + lane < n ? x[base + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v = MAXIMUM ? max(v, u) : v + u;
    }
    v = MAXIMUM ? max(v, carry) : v + carry;
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
  int* pre = reinterpret_cast<int*>(smem_base + L::kPre);
  int2* items = reinterpret_cast<int2*>(smem_base + L::kItems);
  int* extra = reinterpret_cast<int*>(smem_base + L::kExtra);
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
  if (warp == kSoftWarps) ptx::tmem_alloc(ptx::smem_addr(&words->tmem), 512);
  if (warp == kSoftWarps + 1 && lane == 0) {
    words->abort = 0;
    words->bad_nodes[0] = words->bad_nodes[1] = words->bad_nodes[2] = 0;
    ptx::prefetch_tensormap(&a.tk);
    ptx::prefetch_tensormap(&a.tv);
    ptx::prefetch_tensormap(&a.tq_group);
    ptx::prefetch_tensormap(&a.tq_row);
  }
  // Lengths, common tokens, and the first tile of each item in the two concatenated runs; the tables lie where K will.
  constexpr int kMost = QNRE_MAX_CALL_ROWS + 1;
  int* starts = reinterpret_cast<int*>(smem_base + L::kK);
  int* common = starts + kMost;  // tokens of each group
  int* lens = common + kMost;
  int* drafts = lens + kMost;
  int* row_pre = drafts + kMost;
  int* group_pre = row_pre + kMost;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ps = a.c.page_size, room = a.c.max_blocks * ps;
  for (int g = tid; g <= a.n_groups; g += kThreads) {
    starts[g] = a.n_groups > 0 ? min(max(a.groups[g], 0), a.n) : 0;
    common[g] = g < a.n_groups ? min(max(a.shared[g], 0), room) / ps * ps : 0;
  }
  for (int i = tid; i < a.n; i += kThreads) {
    const int row = a.rows[i];
    int len = 0, cnt = 0;
    if (row >= 0 && row < a.c.rows) {
      len = min(a.c.length(row), room);
      cnt = a.counts != nullptr ? min(max(a.counts[i], 0), a.nodes) : a.nodes;
    } else if (blockIdx.x == 0) {
      atomicOr(a.c.status, QNRE_CACHE_BAD_ROW);
    }
    lens[i] = len;
    drafts[i] = min(len + cnt, room) - len;
  }
  __syncthreads();
  if (warp == 0) scan_table<true>(starts, a.n_groups + 1);  // (ascending, whatever is given)
  __syncthreads();
  auto group_of = [&](int i) {  // the last group that starts by i, or -1 where it ends before i
    int lo = -1, hi = a.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (starts[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo >= 0 && i < starts[lo + 1] ? lo : -1;
  };
  if (a.n_groups > 0) {
    for (int i = tid; i < a.n; i += kThreads) {  // no more than every member has
      const int g = group_of(i);
      if (g >= 0) atomicMin(&common[g], starts[g + 1] - starts[g] > 1 ? lens[i] / ps * ps : 0);
    }
    __syncthreads();
  }
  using Run = Cursor<SMALL>;
  for (int i = tid; i < a.n; i += kThreads) {
    const int g = a.n_groups > 0 ? group_of(i) : -1;
    const int base = g >= 0 ? common[g] : 0;
    row_pre[i + 1] = (Run::tiles_of(lens[i] + drafts[i] - base) + kUnitCost) * a.Hk * a.row_tiles;
    if (blockIdx.x == 0) a.first_of[i] = base > 0 ? starts[g] : -1;
  }
  for (int g = tid; g < a.n_groups; g += kThreads) {
    const int members = starts[g + 1] - starts[g];
    group_pre[g + 1] = members > 0 && common[g] > 0
                           ? (Run::tiles_of(common[g]) + kUnitCost) * a.Hk *
                                 Run::clusters_of(members, a.unit_members, a.row_tiles, a.cl)
                           : 0;
  }
  if (tid == 0) row_pre[0] = group_pre[0] = 0;
  __syncthreads();
  if (warp == 0) scan_table<false>(row_pre + 1, a.n);
  if (warp == 1) scan_table<false>(group_pre + 1, a.n_groups);
  __syncthreads();

  // The clusters that take groups: in proportion to the tiles, so that the longest run of either kind is the shortest.
  const int W_rows = row_pre[a.n], W_groups = group_pre[a.n_groups];
  const int clusters = static_cast<int>(gridDim.x) / a.cl;
  int for_groups = 0;
  if (W_groups > 0) {
    const float wide = static_cast<float>(W_groups) * a.cl;
    const int low = static_cast<int>(clusters * (wide / (wide + W_rows)));
    auto longest = [&](int c) {
      return c < 1 || c >= clusters ? 3e38f
                                    : fmaxf(static_cast<float>(W_groups) / c,
                                            static_cast<float>(W_rows) / static_cast<float>((clusters - c) * a.cl));
    };
    for_groups = longest(low) <= longest(low + 1) ? low : low + 1;
    for_groups = min(max(for_groups, 1), clusters - 1);
  }
  const int cluster = static_cast<int>(blockIdx.x) / a.cl;
  Run cur;
  cur.group = cluster < for_groups;
  const bool share = cur.group && a.cl > 1;
  cur.pre = pre;
  cur.items = items;
  cur.extra = extra;
  cur.cl = cur.group ? a.cl : 1;
  cur.rank = share ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  cur.row_tiles = a.row_tiles;
  cur.unit_members = a.unit_members;
  const int W = cur.group ? W_groups : W_rows;
  cur.index = cur.group ? cluster : static_cast<int>(blockIdx.x) - for_groups * a.cl;
  cur.count = min(cur.group ? for_groups : (clusters - for_groups) * a.cl, W);
  cur.quot = W / cur.count;
  cur.rem = W - cur.quot * cur.count;
  cur.cur = cur.index < cur.count ? cur.start_of(cur.index) : 0;
  cur.end = cur.index < cur.count ? cur.start_of(cur.index + 1) : 0;
  const int n_items = cur.group ? a.n_groups : a.n;
  for (int i = tid; i <= n_items; i += kThreads) {
    pre[i] = cur.group ? group_pre[i] : row_pre[i];
    if (i == n_items) break;
    if (cur.group) {
      items[i] = make_int2(starts[i] << 16 | (starts[i + 1] - starts[i]), common[i]);
    } else {
      const int g = a.n_groups > 0 ? group_of(i) : -1;
      const int base = g >= 0 ? common[g] : 0;
      items[i] = make_int2(base, SMALL ? lens[i] << 7 | drafts[i] : lens[i]);
      if (!SMALL) extra[i] = drafts[i];
    }
  }
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
  ptx::fence_proxy_async_smem();  // the tables were there before K is
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (a.cl > 1) ptx::cluster_sync();  // every CTA's barriers stand, and its tables are read, before another sends to it
  ptx::tc_fence_after_sync();
  const uint32_t tmem = words->tmem;
  int lo = 0, hi = n_items - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (pre[mid] <= cur.cur) lo = mid; else hi = mid - 1;
  }
  cur.item = lo;
  Seg first;  // found once for all roles
  const bool more = cur.next(first);

  if (warp < kSoftWarps) {
    run_softmax<L, D, BF16, SMALL, SCORED>(a, bars, smem_base, tmem, cur, first, more, &words->abort, words->bad_nodes);
  } else if (warp == kSoftWarps || warp == kSoftWarps + 3) {
    run_producer<L, D, SMALL>(a, bars, smem, cur, first, more, warp == kSoftWarps ? 0 : 1, share, &words->abort);
  } else if (warp == kSoftWarps + 1) {
    if (lane == 0) run_scores<L, D, BF16, SMALL>(a, bars, smem, tmem, cur, first, more, share, &words->abort);
  } else if (lane == 0) {
    run_outputs<L, D, BF16, SMALL>(a, bars, smem, tmem, cur, first, more, share, &words->abort);
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
struct JoinArgs {
  const int* first_of;
  const Desc *row_units, *group_units;
  const float2* part_ml;
  const float4* part_o;
  char* out;
  float* lse;
  long long own_rows, group_rows, rows;  // rows: of the output
  int n, nodes, Hq, Hk, G, cl, unit_nodes, unit_members, row_tiles;
};

// A thread has four columns of a row, a warp eight rows' (whole lines of the parts).  Rows go by K head, request, node, head.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) join_kernel(const JoinArgs a) {
  constexpr int kWarps = D / 16;  // that share eight rows
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long rr = (static_cast<long long>(blockIdx.x) * (8 / kWarps) + warp / kWarps) * 8 + lane % 8;
  const int i4 = warp % kWarps * 4 + lane / 8;
  if (rr >= a.rows) return;
  const int per_head = a.n * a.nodes * a.G;  // (below 2^31 / Hk)
  const int kvh = static_cast<int>(rr / per_head), in_head = static_cast<int>(rr - static_cast<long long>(kvh) * per_head);
  const int token = in_head / a.G, h = in_head - token * a.G;
  const int i = token / a.nodes, node = token - i * a.nodes;
  const int block = node / a.unit_nodes, in_block = node - block * a.unit_nodes;
  const Desc own = a.row_units[(i * a.Hk + kvh) * a.row_tiles + block];
  if (own.parts < 0) return;
  const int first = a.first_of[i];
  const int own_parts = max(own.parts, 1), own_ur = in_block * a.G + h;
  Desc group{0, 0};
  int group_parts = 0, group_ur = 0;
  if (first >= 0) {
    const int mi = (i - first) % a.unit_members;
    group = a.group_units[((i - mi) * a.Hk + kvh) * a.row_tiles + block];
    group_parts = max(group.parts, 1);
    group_ur = (mi * a.unit_nodes + in_block) * a.G + h;
  }
  const int parts = group_parts + own_parts;
  auto row_of = [&](int p) -> long long {
    if (p < group_parts)
      return group.parts == 0 ? a.group_rows + rr : static_cast<long long>(2 * (group.cta + p * a.cl) + (p == 0 ? 1 : 0)) * 128 + group_ur;
    p -= group_parts;
    return own.parts == 0 ? a.own_rows + rr : static_cast<long long>(2 * (own.cta + p) + (p == 0 ? 1 : 0)) * 128 + own_ur;
  };
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < parts; p0 += 4) {  // four parts' loads at once
    float2 ml[4];
    float4 v[4];
    float mx = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool there = p0 + k < parts;
      const long long row = row_of(there ? p0 + k : p0);
      ml[k] = a.part_ml[row];
      v[k] = a.part_o[piece_of<D>(row, i4)];
      if (!there) ml[k].x = -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) mx = fmaxf(mx, ml[k].x);
    const float f = M == -INFINITY ? 0.f : part_weight(M - mx);
    M = mx;
    l *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (p0 + k >= parts) break;
      const float w = ml[k].x == -INFINITY ? 0.f : part_weight(ml[k].x - M);
      l = fmaf(ml[k].y, w, l);
      acc.x = fmaf(v[k].x, w, acc.x);
      acc.y = fmaf(v[k].y, w, acc.y);
      acc.z = fmaf(v[k].z, w, acc.z);
      acc.w = fmaf(v[k].w, w, acc.w);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const long long orow = static_cast<long long>(token) * a.Hq + kvh * a.G + h;
  *reinterpret_cast<uint2*>(a.out + (orow * D + 4 * i4) * 2) =
      make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
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
  const JoinArgs j{a.first_of, a.row_units, a.group_units, a.part_ml, a.part_o, a.out, a.lse, a.own_rows, a.group_rows,
                   static_cast<long long>(a.n) * a.nodes * a.Hq, a.n, a.nodes, a.Hq, a.Hk, a.G, a.cl, a.unit_nodes,
                   a.unit_members, a.row_tiles};
  constexpr int kJoinRows = 1024 / D;  // a block
  cfg.gridDim = dim3(static_cast<unsigned>((j.rows + kJoinRows - 1) / kJoinRows));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return from_cuda(cudaLaunchKernelEx(&cfg, join_kernel<D, BF16>, j));
}

template <int D, bool BF16>
qnre_status_t launch_size(const PrefixArgs& a, bool scored, int sms, cudaStream_t stream) {
  // only D = 128 has a use for the shorter table
  const bool small = D == 128 && a.n <= kSmall && a.n_groups <= kSmall && a.c.max_blocks * a.c.page_size < kSmallLen;
  if (small) {
    return scored ? launch_prefix<D, BF16, D == 128, true>(a, sms, stream)
                  : launch_prefix<D, BF16, D == 128, false>(a, sms, stream);
  }
  return scored ? launch_prefix<D, BF16, false, true>(a, sms, stream) : launch_prefix<D, BF16, false, false>(a, sms, stream);
}

// The workspace: words of requests and units, the parts of the CTAs' runs, and, where rows may share, a place of its own for
// each row's part of either kind.
struct Layout {
  uint64_t first_of, row_units, group_units, ml, o, bytes;
  int64_t own_rows, group_rows;
};

Layout layout_of(int64_t n, int64_t nodes, int64_t Hq, int64_t Hk, int D, bool groups) {
  const int64_t unit_nodes = std::min<int64_t>(nodes, kTile / (Hq / Hk)), tiles = (nodes + unit_nodes - 1) / unit_nodes;
  const int64_t slots = 2ll * kMaxCtas * 128, rows = groups ? (n * nodes * Hq + 7) / 8 * 8 : 0;
  Layout l;
  auto up = [](uint64_t x) { return (x + 15) / 16 * 16; };
  l.first_of = 0;
  l.row_units = up(n * 4);
  l.group_units = l.row_units + up(n * Hk * tiles * sizeof(Desc));
  l.ml = l.group_units + (groups ? up(n * Hk * tiles * sizeof(Desc)) : 0);
  l.own_rows = slots;
  l.group_rows = slots + rows;
  l.o = l.ml + (slots + 2 * rows) * 8;
  l.bytes = l.o + static_cast<uint64_t>(slots + 2 * rows) * D * 4;
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
          mine[k] = __ldg(table + b);
          first[k] = __ldg(table0 + b);
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
                             words(slopes, static_cast<uint64_t>(Hq) * 4)};
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
  // CTAs of a cluster: the units that a group of average size has for a K head
  const int members = n_groups > 0 ? (n + n_groups - 1) / n_groups : 0;
  const int units = (members + a.unit_members - 1) / a.unit_members * a.row_tiles;
  a.cl = std::min(std::max(units, 1), kMaxCluster);
  const int64_t tiles = (static_cast<int64_t>(cache->max_blocks) * cache->page_size + kTile - 1) / kTile + kUnitCost;
  if (a.n * tiles * a.Hk * a.row_tiles > 0x7FFFFFFF || static_cast<int64_t>(out_rows) > 0x7FFFFFFF) return QNRE_ERR_CAPACITY;
  a.box = std::min(a.cl > 1 ? kTile / kMaxCluster : kTile, cache->page_size & -cache->page_size);
  a.rows = rows;
  a.groups = groups;
  a.shared = shared;
  a.counts = counts;
  a.depths = depths;
  a.mask = mask;
  a.slopes = slopes;
  a.out = static_cast<char*>(out);
  a.lse = lse;
  char* ws = static_cast<char*>(workspace);
  a.first_of = reinterpret_cast<int*>(ws + l.first_of);
  a.row_units = reinterpret_cast<Desc*>(ws + l.row_units);
  a.group_units = reinterpret_cast<Desc*>(ws + l.group_units);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part_o = reinterpret_cast<float4*>(ws + l.o);
  a.own_rows = l.own_rows;
  a.group_rows = l.group_rows;
  a.scale_log2 = scale * kLog2e;
  a.cap_log2 = softcap * kLog2e;
  a.cap_in = softcap > 0.f ? 2.f * kLog2e * scale / softcap : 0.f;
  const bool bf16 = cache->dtype == QNRE_DTYPE_BF16;
  const uint64_t D = cache->head_dim, ps = cache->page_size, H = cache->heads;
  const uint64_t dims[4] = {D, ps, H, static_cast<uint64_t>(cache->layers) * cache->pages};
  const uint64_t strides[3] = {D * 2, ps * D * 2, H * ps * D * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(a.box), 1, 1};
  const uint64_t q_dims[4] = {D, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.nodes), static_cast<uint64_t>(a.n)};
  const uint64_t q_strides[3] = {static_cast<uint64_t>(own.stride[2]) * 2, static_cast<uint64_t>(own.stride[1]) * 2,
                                 static_cast<uint64_t>(own.stride[0]) * 2};
  uint32_t q_box[4] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(a.unit_nodes), 1};
  if (!encode_tiled_16bit(&a.tq_row, own.data, bf16, 4, q_dims, q_strides, q_box)) return QNRE_ERR_CUDA;
  q_box[3] = static_cast<uint32_t>(a.unit_members);
  if (!encode_tiled_16bit(&a.tq_group, own.data, bf16, 4, q_dims, q_strides, q_box) ||
      !encode_tiled_16bit(&a.tk, cache->k, bf16, 4, dims, strides, box) ||
      !encode_tiled_16bit(&a.tv, cache->v, bf16, 4, dims, strides, box))
    return QNRE_ERR_CUDA;
  const bool scored = softcap > 0.f || slopes != nullptr;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) return bf16 ? launch_size<128, true>(a, scored, sms, s) : launch_size<128, false>(a, scored, sms, s);
  return bf16 ? launch_size<64, true>(a, scored, sms, s) : launch_size<64, false>(a, scored, sms, s);
}

}  // extern "C"
