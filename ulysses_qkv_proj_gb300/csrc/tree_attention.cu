// tree_attention.cu -- attention of drafted tree nodes (or of one new token) over a
// paged K/V cache, on the sm_103a tensor cores.
//
//   o = sum_x p_x v_x,  p = softmax(scale q.k_x) over the tokens a node sees
//
// Work is cut into units (request, K head, up to 128 rows of (node, query head of the group)) and
// each unit into tiles of 128 cached tokens; the concatenated tiles of all units, with a fixed cost
// for each unit's start and end, are dealt out in equal consecutive runs, one to a CTA, so batches
// of any raggedness load every SM alike.  Each CTA takes the lengths from device memory and finds its own run.  A unit that spans
// CTAs leaves an unnormalised (m, l, O) in the workspace from each, joined by combine_kernel in
// CTA order: the result depends on the lengths alone, never on timing.
//
// In a CTA: one warp brings K tiles and Q by TMA, one V tiles (a page's tokens of one head are one run of
// memory; boxes of the largest power of two that divides the page, the page numbers fetched a tile ahead); one
// thread issues S = Q K^T (tcgen05.mma, fp32 S in tensor memory, two buffers), another O += P V (P from tensor
// memory), so that neither waits behind the other; the softmax warps make one pass over S with a running
// maximum and sum in base 2.  P is rounded to the inputs' type, as the second product's operands have one type (relative
// 2^-8 for bf16, 2^-11 for fp16; its sum is kept of the unrounded values in fp32); O is rescaled only when a row's maximum
// grows by more than 2^8.  fp16 has few exponents: P is formed 2^7 times larger there (kLift), so that it stays below
// 2^15 and is normal down to 2^-21 of the row's maximum; smaller weights are off by at most 2^-32 of the maximum's.
// Without that the share of 10^5 tokens under one strong score 17.5 nats above them was lost whole.
//
// Units of few rows would leave lanes idle: with up to 32 (64) rows they are laid out REP = 4 (2) times, copy
// c looking at its own 128 / REP tokens of each tile.  P is zero outside that block, so one O accumulator of 128
// rows holds REP independent partial results, joined at the end through shared memory; the tensor work is
// the same and each softmax thread has 1 / REP of the exponentials.  With more rows two threads share a row,
// half a tile each.  Row tiles of one head (more than 128 rows) run as a cluster of up to four CTAs that
// fetch K and V for one another by multicast.
//
// Slots that a row does not see must not reach it, whatever they hold: scores are replaced before use; V rows of
// slots past the drafts are zeroed in shared memory, and non-finite V elements of drafted nodes (which
// some rows see and others do not) are zeroed there and added to the rows that see them at the end.  Every row sees the
// context, whose V stays as it is; but an infinite element meets zeros of P in the other copies of a row (or where a weight
// rounds to nothing), and 0 inf is NaN.  So when a row's sum is not finite the context is searched, and a channel that
// holds non-finite elements gets their sum: infinity, or NaN for a NaN or for both signs.  Each warp votes on its own rows and
// searches alone: a vote of all softmax warps would be a barrier more for every unit (16 trees of 32 nodes +1.5 %).
//
// Bound: HBM up to 128 rows; above, the bytes that enter an SM (64 KB of K and V a tile of 1024 cycles of
// tensor work, at 34 bytes a cycle and SM).  Measured (device time): 64 requests of 130..32000 tokens, 64 heads on 8,
// D = 128 bf16: 234 us, 6.68 TB/s; 16 trees of 32 nodes over 900..16001 tokens: 84 us, 1.10 PFLOP/s; 6 trees of 61
// nodes, D = 64 fp16: 37 us; one request of 4097 tokens, 32 heads on 8: 13 us, of which the join is three.  Steps, in
// that order: first form 431 / 229 / 270 / 20.6; Q by TMA, scores of the next unit before the last product, masks as
// words, a unit's cost in the split 258 / 147 / 50 / 17; two issuing threads, descriptors by one add 239 / 142 / 50 /
// 17; multicast, page numbers ahead - / 109 / 48 / 15.3; three tiles of K and of V in flight 237 / 100 / 48 / 15.2;
// cheaper unit ends, a unit's cost four tiles (2: 102 / 53, 8: 100 / 48 cold) 234 / 91 / 37 / 14.3; eight warps a row in
// the join of few rows, its parts counted beforehand 234 / 87 / 37 / 13.2; parts of more than 64 rows written eight
// rows to a line - / 84 / - / -; the vote on non-finite sums 230 / 84 / 36.8 / 13.0, from 230 / 84 / 36.7 / 12.8 on the same
// machine.  Tried and left: Q in tensor memory with P over S (108) or one P buffer (106), the pass
// with a standing maximum 32 columns at a time (101), a CTA pair multiplying as one (98), two row tiles a CTA on the same
// K and V (117: P lies in S's place, so each tile is product, scores, softmax in a row, 4170 cycles for the two).
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
#include <cstdint>

namespace {

using namespace qnre;
using namespace qnre::api;
using namespace qnre::attention;

// Softmax warps: with REP = 1 two threads share a row, each half of a tile's tokens.  Else one thread a row and copy,
// and at D = 64, where a tile's bytes arrive faster than four warps finish its softmax (1400 cycles against 1800), two
// groups of four warps that take alternate tiles, each with an O of its own (at D = 128 tensor memory has no room for a
// second, and a tile's bytes take 2800 cycles).  32 requests of 130..16000 tokens, 64 heads on 8: 45.2 us against 48.6
// with one group, 4 trees of 40 nodes, 14 heads: 32.3 against 37.0, one request of 4097 tokens 11.1 against 10.9; at
// REP = 1 two groups are slower (16 trees of 32 nodes, 32 heads on 8: 45.5 against 43.3).  Then the K and V TMA warps
// and the warps that issue S and O products.
template <int D, int REP>
constexpr int kGroups = D == 64 && REP > 1 ? 2 : 1;
template <int D, int REP>
constexpr int kSoftThreads = REP == 1 ? 256 : 128 * kGroups<D, REP>;
template <int D, int REP>
constexpr int kThreads = kSoftThreads<D, REP> + 128;
constexpr int kMaxCtas = 152;  // one a SM
constexpr int kTmemS = 0, kTmemO = 256, kTmemP = 384;  // columns: S 2 x 128, O D or 2 x 64, P 2 x 64
constexpr int kMaxCluster = 4;  // row tiles that share K and V
constexpr int kUnitCost = 4;  // a unit's start and end, in tiles

// A unit that spans clusters c0 .. c0 + parts - 1, written by its second one for combine_kernel.
struct Desc {
  int parts, req, kvh, rt, c0, pad[3];
};

struct AttnArgs {
  CUtensorMap tk, tv, tq;
  CacheView c;
  const int32_t* rows;
  const int32_t* counts;
  const uint64_t* mask;
  char* out;
  float* lse;
  Desc* desc;
  float* part_ml;  // [2 * kMaxCtas][128][2]: maximum (base 2), sum
  float* part_o;   // [2 * kMaxCtas] of 128 rows of D, laid out by part_at
  float scale_log2;
  int layer, n, nodes, Hq, Hk, G, unit_nodes, row_groups, box, cl;  // cl: CTAs a cluster, row tiles a group
};

// Shared memory.  Loads take about 2900 cycles from request to use when every SM loads, a tile of scores or of
// outputs some 1200, so three tiles of K and of V are wanted: at D = 128 they fit next to Q when one row tile needs
// no join (REP = 1) and the batch's lengths are few (SMALL: 64 requests); else V has two.
template <int D, int REP, bool SMALL>
struct Smem {
  static constexpr int kRequests = SMALL ? 64 : QNRE_MAX_CALL_ROWS;
  static constexpr int kKStages = D == 128 ? 3 : 5;
  static constexpr int kVStages = D == 128 ? (REP == 1 && SMALL ? 3 : 2) : 5;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kTileBytes;
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kSoft = kSoftThreads<D, REP>;
  static constexpr int kJoin = kV + kVStages * kTileBytes;               // REP > 1: float [kSoft][33]
  static constexpr int kMl = kJoin + (REP > 1 ? kSoft * 33 * 4 : 0);     // float [kSoft][2]; REP = 1: [2][2][128]
  static constexpr int kLen = kMl + (REP > 1 ? kSoft * 2 * 4 : 2048);    // int2 [kRequests]
  static constexpr int kPre = kLen + kRequests * 8;                      // int [kRequests + 1]
  static constexpr int kBars = (kPre + (kRequests + 1) * 4 + 15) / 16 * 16;
  static constexpr int kWords = kBars + 8 * (2 * kKStages + 2 * kVStages + 13);
  static constexpr int kBytes = kWords + 32;
  static_assert(kBytes <= 232448, "one CTA's shared memory");
};

// Words shared by the roles.
struct Words {
  unsigned long long bad_nodes[3];  // drafts with non-finite V elements, segments in turn
  uint32_t tmem, abort;
};

struct Bars {
  uint32_t kfull, kempty, vfull, vempty, qfull, qempty, sfull, sfree, pready, pvdone, ofree, drain, drain2;
};

// One unit's part of a CTA's run.
struct Seg {
  int req, kvh, rt, t0, t1, len, total;
  bool whole;
  int slot;
};

struct Cursor {
  const int* pre;
  const int2* lens;
  int cur, end, req, row_groups, cl, rank;
  __device__ __forceinline__ static int tiles_of(int total) { return total > 0 ? (total + kTile - 1) / kTile : 1; }
  __device__ __forceinline__ bool next(Seg& s) {
    while (cur < end) {
      while (cur >= pre[req + 1]) ++req;
      s.req = req;
      s.len = lens[req].x;
      s.total = lens[req].y;
      const int tiles = tiles_of(s.total), per = tiles + kUnitCost;
      const int off = cur - pre[req];
      const int unit = off / per, o = off - unit * per;
      const int take = min(per - o, end - cur);
      cur += take;
      s.t0 = max(0, o - kUnitCost);
      s.t1 = max(0, o + take - kUnitCost);
      if (s.t0 == s.t1) continue;  // the unit's cost falls to this CTA, its tiles to the next
      s.kvh = unit / row_groups;
      s.rt = (unit - s.kvh * row_groups) * cl + rank;
      s.whole = s.t0 == 0 && s.t1 == tiles;
      // a CTA goes on with one unit at most, and leaves one unfinished at most
      s.slot = 2 * static_cast<int>(blockIdx.x) + (s.t0 == 0 ? 1 : 0);
      return true;
    }
    return false;
  }
};

// Among the softmax threads; among the two warps that share 32 rows.
template <int THREADS>
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}
// ------------------------------------------------------------------ TMA warps
// One warp brings Q and K, another V.  With MC each CTA of the cluster fetches its share of a tile's boxes for
// all of them.
template <typename L, int D, int REP, bool MC>
__device__ void run_producer(const AttnArgs& a, const Bars& bars, uint32_t smem, Cursor cur, Seg s, bool more, int kv,
                             volatile uint32_t* abort_flag) {
  constexpr int kHalves = D / 64;
  const int lane = threadIdx.x % 32;
  const int chunk = lane / kHalves, half = lane % kHalves;
  const bool active = chunk < kTile / a.box && (!MC || lane % a.cl == cur.rank);
  const int ps = a.c.page_size, step = kTile / ps, step_off = kTile - step * ps;
  const int none = a.c.layers * a.c.pages;  // past the end: the box is filled with zeros
  const uint16_t everyone = static_cast<uint16_t>((1u << a.cl) - 1u);
  const CUtensorMap* map = kv ? &a.tv : &a.tk;
  const uint32_t dst = smem + (kv ? L::kV : L::kK) + half * (kTile * 128) + chunk * a.box * 128;
  const int q_nodes = min(a.unit_nodes, a.nodes);
  const uint32_t q_bytes = static_cast<uint32_t>(REP * D * 2 * a.G * q_nodes);
  const uint32_t full = kv ? bars.vfull : bars.kfull, empty = kv ? bars.vempty : bars.kempty;
  const uint32_t stages = kv ? L::kVStages : L::kKStages;
  uint32_t slot = 0, phase = 1;
  auto settle = [] {  // stop: what is in flight lands in microseconds; the kernel's end waits for it
    const uint64_t t0 = ptx::global_timer_ns();
    while (ptx::global_timer_ns() - t0 < 50000) {
    }
  };
  for (uint32_t seg = 0; more; ++seg, more = cur.next(s)) {
    const int row = a.rows[s.req];
    const bool fetches = active && row >= 0 && row < a.c.rows;
    const int32_t* table = a.c.table + static_cast<long long>(fetches ? row : 0) * a.c.max_blocks;
    int pos = s.t0 * kTile + chunk * a.box;
    int block = pos / ps, off = pos - block * ps;
    // (a plain load, not a read-only one: the kernel starts beside the launch that writes the table)
    auto look = [&]() -> int { return fetches && block < a.c.max_blocks ? table[block] : -1; };
    int entry = look();
    if (kv == 0) {  // the unit's Q rows, REP times
      // (one buffer: the last unit's results are still being written when its last scores are done)
      if (!wait(bars.qempty, (seg & 1u) ^ 1u, abort_flag, a.c.status)) return settle();
      if (lane == 0) ptx::mbar_arrive_expect_tx(bars.qfull, q_bytes);
      __syncwarp();
      if (lane < REP * kHalves)
        tma_load_4d(smem + L::kQ + (lane % kHalves) * (kTile * 128) + (lane / kHalves) * (kTile / REP) * 128, &a.tq,
                    bars.qfull, (lane % kHalves) * 64, s.kvh * a.G, s.rt * a.unit_nodes, s.req);
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
        if (MC)
          tma_load_4d_multicast(dst + slot * L::kTileBytes, map, full + 8 * slot, half * 64, at, s.kvh, page,
                                everyone);
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
// S = Q K^T, tile after tile, across units: two ahead of the softmax as far as S's two buffers allow.
template <typename L, int D, bool BF16, bool MC>
__device__ void run_scores(const AttnArgs& a, const Bars& bars, uint32_t smem, uint32_t tmem, Cursor cur, Seg s,
                           bool more, volatile uint32_t* abort_flag) {
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
      if (MC)
        umma_commit_multicast(bars.kempty + 8 * slot, everyone);
      else
        ptx::umma_commit(bars.kempty + 8 * slot);
      if (t + 1 == s.t1) ptx::umma_commit(bars.qempty);
      if (++slot == L::kKStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

// O += P V, tile after tile; with two groups of softmax warps even and odd tiles each have an O.
template <typename L, int D, bool BF16, bool MC, int GROUPS>
__device__ void run_outputs(const AttnArgs& a, const Bars& bars, uint32_t smem, uint32_t tmem, Cursor cur, Seg s,
                            bool more, volatile uint32_t* abort_flag) {
  constexpr uint32_t kFmt = BF16 ? (1u << 7 | 1u << 10) : 0u;
  constexpr uint32_t kIdesc =
      (1u << 4) | kFmt | (1u << 16) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24);
  const uint64_t ring0 = ptx::smem_desc_sw128(smem + L::kV, kTile * 128, 1024);
  const uint16_t everyone = static_cast<uint16_t>((1u << a.cl) - 1u);
  uint32_t g = 0, slot = 0, phase = 0;
  for (uint32_t seg = 0; more; ++seg, more = cur.next(s)) {
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
        umma_f16_ts(tmem + kTmemO + (GROUPS == 2 ? b * 64 : 0), tmem + kTmemP + b * 64 + kk * 8, desc_at(v, kk * 2048),
                    kIdesc, (t - s.t0 >= GROUPS || kk > 0) ? 1u : 0u);
      ptx::umma_commit(bars.pvdone + 8 * b);
      if (MC)
        umma_commit_multicast(bars.vempty + 8 * slot, everyone);
      else
        ptx::umma_commit(bars.vempty + 8 * slot);
      if (++slot == L::kVStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
}

// ------------------------------------------------------------------ softmax warps
template <typename L, int D, bool BF16, int REP>
__device__ void run_softmax(const AttnArgs& a, const Bars& bars, char* smem_base, uint32_t smem, uint32_t tmem,
                            Cursor cur, Seg next, bool more, volatile uint32_t* abort_flag,
                            unsigned long long* bad_nodes) {
  constexpr bool kSplit = REP == 1;    // two threads a row, one maximum and one O
  constexpr int kCols = kSplit ? 64 : kTile / REP;  // tokens of a tile this thread looks at
  constexpr int kRows = 128 / REP;     // unit rows
  constexpr int kOut = kSplit ? D / 2 : D;  // columns of O this thread scales and writes
  constexpr int kTwo = kGroups<D, REP> == 2, kSoft = kSoftThreads<D, REP>;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t group = kTwo ? tid / 128 : 0;  // of alternate tiles
  const int ur = tid % kRows, copy = (kSplit ? tid : tid % 128) / kRows, c0 = copy * kCols;
  const int part = tid / kRows;  // of a row's results
  const int o0 = kSplit ? copy * kOut : 0;
  const uint32_t o_at = kTmemO + group * 64;
  const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
  float* join = reinterpret_cast<float*>(smem_base + L::kJoin);
  float* ml = reinterpret_cast<float*>(smem_base + L::kMl);
  const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);

  if (REP > 1) {  // P outside this copy's tokens stays zero
    uint32_t zero[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) zero[i] = 0;
#pragma unroll
    for (int c = 0; c < (kTwo ? 64 : 128); c += 32) tmem_st_x32(tmem + lane_base + kTmemP + group * 64 + c, zero);
    tmem_st_wait();
  }
  const int ur_node = ur / a.G, ur_head = ur - ur_node * a.G;

  // what this thread's row of a segment is
  struct RowInfo {
    int node, head;
    bool in_out, row_ok;  // a row of the output; of a node that sees anything
    uint64_t bits;        // the drafts it sees
  };
  auto row_info = [&](const Seg& s) {
    RowInfo r{s.rt * a.unit_nodes + ur_node, s.kvh * a.G + ur_head, false, false, 0};
    r.in_out = ur_node < a.unit_nodes && r.node < a.nodes;
    r.row_ok = r.in_out && (a.counts == nullptr || r.node < a.counts[s.req]);
    if (r.in_out)
      r.bits = a.mask != nullptr ? a.mask[static_cast<long long>(s.req) * a.nodes + r.node] : (2ull << r.node) - 1;
    return r;
  };

  uint32_t g = 0;
  Seg s;
  RowInfo row{}, next_row{};
  if (more) next_row = row_info(next);
  for (uint32_t seg = 0; more; ++seg) {
    s = next;
    row = next_row;
    const int node = row.node, head = row.head;
    const bool in_out = row.in_out, row_ok = row.row_ok;
    const int slots = s.total - s.len;  // drafts that have a place
    const uint64_t bits = slots < 64 ? row.bits & ((1ull << slots) - 1) : row.bits;
    float m = -INFINITY, l = 0.f;
    for (int t = s.t0; t < s.t1; ++t, ++g) {
      const uint32_t b = g & 1u;
      if (kTwo && b != group) continue;
      uint32_t v[kCols / 32][32];
      // P's buffer is free once the product two tiles back is done (long ago, by now; with two groups, this
      // group's last: waiting for it only before P is stored changes nothing)
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

      const bool tail = (t + 1) * kTile > s.len;
      if (tail) {
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j) {
          const uint32_t see = seen_word(t * kTile + c0 + 32 * j - s.len, bits);
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
      float mx = fmaxf(mx0, mx1) * a.scale_log2;
      if (kSplit) {  // with the other half's; two buffers, as the next tile's may be written before this is read
        float* at = ml + b * 256 + ur;
        at[copy * 128] = mx;
        pair_sync(warp % 4);
        mx = fmaxf(mx, at[(copy ^ 1) * 128]);
      }
      mx -= kLift<BF16>;  // m: the row's maximum less the lift, which leaves O / l and m + log2 l as they are
      const bool grow = mx > m + kRescale;
      if (t - s.t0 < (kTwo ? 2 : 1)) {
        m = mx;
      } else if (__any_sync(0xFFFFFFFFu, grow)) {
        if (!kTwo) {  // (else O's last product was two tiles back)
          const uint32_t last = g - 1;
          wait(bars.pvdone + 8 * (last & 1u), (last >> 1) & 1u, abort_flag, a.c.status);
          __syncwarp();
          ptx::tc_fence_after_sync();
        }
        const float f = grow ? exp2_fast(m - mx) : 1.f;
        if (grow) m = mx;
        l *= f;
#pragma unroll 1
        for (int c = o0; c < o0 + kOut; c += 32) {
          uint32_t o[32];
          ptx::tmem_ld_32x32b_x32(tmem + lane_base + o_at + c, o);
          ptx::tmem_ld_wait();
          tmem_fence_regs(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st_x32(tmem + lane_base + o_at + c, o);
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
        unpair(fma2(pair(__uint_as_float(v[i / 16][(2 * i) % 32]), __uint_as_float(v[i / 16][(2 * i + 1) % 32])), scale2,
                    neg), e0, e1);
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
      const uint32_t pt = tmem + lane_base + kTmemP + b * 64 + c0 / 2;
      if (kCols == 64) {
        tmem_st_x32(pt, p);
      } else {
        tmem_st_x16(pt, p);
      }
      if (tail) {
        const uint32_t slot = g % L::kVStages;
        wait(bars.vfull + 8 * slot, (g / L::kVStages) & 1u, abort_flag, a.c.status);
        const int x = tid % 128, pos = t * kTile + x, pieces = D / 8 / (kSplit ? 2 : 1);
        if (pos >= s.len && clean_v_row<D, BF16>(smem_base + L::kV + slot * L::kTileBytes + x * 128, pos < s.total,
                                                 kSplit ? copy * pieces : 0, (kSplit ? copy * pieces : 0) + pieces))
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
    if (kSplit) {
      ml[(g & 1u) * 256 + tid] = l;  // (the buffer that the last tile did not use)
    } else {
      ml[2 * tid] = m;
      ml[2 * tid + 1] = l;
    }
    // this group's last product of the segment (a segment of one tile leaves the other group none)
    const uint32_t last = kTwo && ((g - 1) & 1u) != group ? g - 2 : g - 1;
    const bool any = !kTwo || last + (s.t1 - s.t0) + 1 > g;
    if (any) wait(bars.pvdone + 8 * (last & 1u), (last >> 1) & 1u, abort_flag, a.c.status);
    soft_sync<kSoft>();
    ptx::tc_fence_after_sync();
    // every warp has read the word of the segment before, and none uses it again before the next segment's end
    if (tid == 0) bad_nodes[(seg + 2) % 3] = 0;
    const uint64_t bad = row_ok ? bad_nodes[seg % 3] & bits : 0;
    float f = 1.f;  // of this copy's part
    if (kSplit) {
      l += ml[(g & 1u) * 256 + (tid ^ 128)];
      pair_sync(warp % 4);  // read by both before the next tile's maxima go there
    } else {
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int c = 0; c < kSoft / kRows; ++c) M = fmaxf(M, ml[2 * (c * kRows + ur)]);
#pragma unroll
      for (int c = 0; c < kSoft / kRows; ++c) {
        const float mc = ml[2 * (c * kRows + ur)];
        sum += ml[2 * (c * kRows + ur) + 1] * (mc == -INFINITY ? 0.f : exp2_fast(mc - M));
      }
      f = m == -INFINITY ? 0.f : exp2_fast(m - M);
      m = M;
      l = sum;
    }
    const float inv = !s.whole ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
    const long long orow = (static_cast<long long>(s.req) * a.nodes + node) * a.Hq + head;
    const long long prow = static_cast<long long>(s.slot) * 128 + ur;
    constexpr int kPer = kSplit ? 32 : 32 / (kSoft / kRows);  // columns of a block of 32 this thread writes, from jc on
    const int jc = kSplit ? 0 : part * kPer;
#pragma unroll 1
    for (int c = o0; c < o0 + kOut; c += 32) {
      uint32_t o[32];
      ptx::tmem_ld_32x32b_x32(tmem + lane_base + o_at + c, o);
      ptx::tmem_ld_wait();
      tmem_fence_regs(o);
      if (c + 32 == o0 + kOut) {
        ptx::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.ofree);
      }
      float x[kPer];
      if (REP == 1) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = __uint_as_float(o[i]);
      } else {  // the copies of a row lie in different warps
#pragma unroll
        for (int i = 0; i < 32; ++i) join[tid * 33 + i] = any ? __uint_as_float(o[i]) * f : 0.f;
        soft_sync<kSoft>();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          x[i] = 0.f;
#pragma unroll
          for (int k = 0; k < kSoft / kRows; ++k) x[i] += join[(k * kRows + ur) * 33 + jc + i];
        }
        soft_sync<kSoft>();
      }
      uint64_t odd = 0;  // 0 x is 0 for every finite x
#pragma unroll
      for (int i = 0; i < kPer; i += 2) odd = fma2(pair(x[i], x[i + 1]), 0, odd);
      float odd0, odd1;
      unpair(odd, odd0, odd1);
      if (__any_sync(0xFFFFFFFFu, row_ok && odd0 + odd1 != 0.f)) {  // (NaN compares unequal)
        const Kinds k = search_context<BF16>(a.c, a.layer, a.rows[s.req], s.kvh, s.t0 * kTile, min(s.t1 * kTile, s.len), c);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t bit = 1u << (jc + i);
          if ((k.plus | k.minus | k.nan) & bit)
            x[i] = (k.nan | (k.plus & k.minus)) & bit ? NAN : (k.plus & bit ? INFINITY : -INFINITY);
        }
      }
      if (bad != 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          x[i] = add_nonfinite<BF16>(a.c, a.layer, a.rows[s.req], s.kvh, s.len, s.t0 * kTile, s.t1 * kTile, bad, c + jc + i, x[i]);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = row_ok ? x[i] * inv : 0.f;
      if (in_out && s.whole) {
        uint32_t w[kPer / 2];
#pragma unroll
        for (int e = 0; e < kPer / 2; ++e) w[e] = pack2<BF16>(x[2 * e], x[2 * e + 1]);
        char* dst = a.out + (orow * D + c + jc) * 2;
        if constexpr (kPer >= 8) {
#pragma unroll
          for (int i = 0; i < kPer / 8; ++i)
            reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
          *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        }
      } else if (in_out) {
        float4* dst = reinterpret_cast<float4*>(a.part_o);
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i)
          dst[part_at<D, REP == 1>(s.slot, ur, (c + jc) / 4 + i)] =
              make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
      __syncwarp();
    }
    if (in_out && part == 0) {
      if (!s.whole)
        reinterpret_cast<float2*>(a.part_ml)[prow] = make_float2(m, l);
      else if (a.lse != nullptr)
        a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
}

template <int D, bool BF16, int REP, bool MC, bool SMALL>
__global__ void __launch_bounds__(kThreads<D, REP>, 1) attention_kernel(const __grid_constant__ AttnArgs a) {
  using L = Smem<D, REP, SMALL>;
  extern __shared__ __align__(1024) char smem_base[];
  const uint32_t smem = ptx::smem_addr(smem_base);
  Words* words = reinterpret_cast<Words*>(smem_base + L::kWords);
  constexpr int kSoftWarps = kSoftThreads<D, REP> / 32;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int* pre = reinterpret_cast<int*>(smem_base + L::kPre);
  int2* lens = reinterpret_cast<int2*>(smem_base + L::kLen);
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
    for (int i = 0; i < L::kKStages; ++i) {
      ptx::mbar_init(bars.kfull + 8 * i, 1);
      ptx::mbar_init(bars.kempty + 8 * i, a.cl);
    }
    for (int i = 0; i < L::kVStages; ++i) {
      ptx::mbar_init(bars.vfull + 8 * i, 1);
      ptx::mbar_init(bars.vempty + 8 * i, a.cl);
    }
    ptx::mbar_init(bars.qfull, 1);
    ptx::mbar_init(bars.qempty, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars.sfull + 8 * i, 1);
      ptx::mbar_init(bars.sfree + 8 * i, kSoftWarps / kGroups<D, REP>);
      ptx::mbar_init(bars.pready + 8 * i, kSoftWarps / kGroups<D, REP>);
      ptx::mbar_init(bars.pvdone + 8 * i, 1);
    }
    ptx::mbar_init(bars.ofree, kSoftWarps);
    ptx::mbar_init(bars.drain, 1);
    ptx::mbar_init(bars.drain2, 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&a.tk);
    ptx::prefetch_tensormap(&a.tv);
    ptx::prefetch_tensormap(&a.tq);
  }
  // the rows' lengths, and the first tile of each request in the concatenated run
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int units = a.Hk * a.row_groups;
  const int room = a.c.max_blocks * a.c.page_size;
  for (int i = tid; i < a.n; i += kThreads<D, REP>) {
    const int row = a.rows[i];
    int len = 0, cnt = 0;
    if (row >= 0 && row < a.c.rows) {
      len = min(a.c.length(row), room);
      cnt = a.counts != nullptr ? min(max(a.counts[i], 0), a.nodes) : a.nodes;
    } else if (blockIdx.x == 0) {
      atomicOr(a.c.status, QNRE_CACHE_BAD_ROW);
    }
    const int total = min(len + cnt, room);
    lens[i] = make_int2(len, total);
    pre[i + 1] = (Cursor::tiles_of(total) + kUnitCost) * units;
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    if (lane == 0) pre[0] = 0;
    for (int base = 0; base < a.n; base += 32) {
      int v = base + lane < a.n ? pre[base + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
      }
      if (base + lane < a.n) pre[base + lane + 1] = carry + v;
      carry += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (MC) ptx::cluster_sync();  // every CTA's barriers stand before another arrives on them
  ptx::tc_fence_after_sync();
  const uint32_t tmem = words->tmem;
  // this cluster's run of the W tiles: clusters get equal runs, in 32-bit arithmetic
  const int rank = MC ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int cluster = MC ? static_cast<int>(blockIdx.x) / a.cl : static_cast<int>(blockIdx.x);
  const int W = pre[a.n];
  const int clusters = min(static_cast<int>(gridDim.x) / a.cl, W);
  const int quot = W / clusters, rem = W - quot * clusters;
  auto start_of = [&](int c) { return c * quot + c * rem / clusters; };
  Cursor cur;
  cur.pre = pre;
  cur.lens = lens;
  cur.row_groups = a.row_groups;
  cur.cl = a.cl;
  cur.rank = rank;
  cur.cur = cluster < clusters ? start_of(cluster) : 0;
  cur.end = cluster < clusters ? start_of(cluster + 1) : 0;
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (pre[mid] <= cur.cur) lo = mid; else hi = mid - 1;
  }
  cur.req = lo;
  // The first unit's part is found here, once for all roles: the roles' own copies of this code start with an empty
  // instruction cache (1700 cycles to the first part; one request 13.8 us, so 13.5).
  Seg first;
  const bool more = cur.next(first);

  if (warp < kSoftWarps) {
    run_softmax<L, D, BF16, REP>(a, bars, smem_base, smem, tmem, cur, first, more, &words->abort, words->bad_nodes);
  } else if (warp == kSoftWarps || warp == kSoftWarps + 3) {
    run_producer<L, D, REP, MC>(a, bars, smem, cur, first, more, warp == kSoftWarps ? 0 : 1, &words->abort);
  } else if (warp == kSoftWarps + 1) {
    if (lane == 0) run_scores<L, D, BF16, MC>(a, bars, smem, tmem, cur, first, more, &words->abort);
  } else if (lane == 0) {
    // does this run go on with a unit that the one before it began?  Then name it for the join
    Desc d{};
    const Seg& s = first;
    if (more && s.t0 > 0) {
      const int tiles = Cursor::tiles_of(s.total);
      const int begin = pre[s.req] + (s.kvh * a.row_groups + s.rt / a.cl) * (tiles + kUnitCost) + kUnitCost;
      if (begin >= start_of(cluster - 1)) {
        int lo = cluster, hi = clusters - 1;  // the last cluster whose run starts by its last tile
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (start_of(mid) <= begin + tiles - 1) lo = mid; else hi = mid - 1;
        }
        d = Desc{lo - cluster + 2, s.req, s.kvh, s.rt, cluster - 1, {0, 0, 0}};
      }
    }
    a.desc[blockIdx.x] = d;
    run_outputs<L, D, BF16, MC, kGroups<D, REP>>(a, bars, smem, tmem, cur, first, more, &words->abort);
  }
  __syncwarp();
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  if (warp == kSoftWarps) {
    ptx::tmem_relinquish_alloc_permit();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (MC) {
    __syncwarp();
    ptx::cluster_sync();  // none leaves while another may still write to it
  }
}

// Joins the parts of the units that span CTAs: block x is the unit's second CTA.
// Up to 64 rows: WARPS warps a row, each with every WARPS-th part, so that a row of many parts (few rows of a long
// context) costs one round of loads.
template <int D, bool BF16, int WARPS>
__global__ void __launch_bounds__(256) combine_few_kernel(const Desc* desc, const float* part_ml, const float* part_o,
                                                          char* out, float* lse, int nodes, int Hq, int G,
                                                          int unit_nodes, int cl) {
  constexpr int kPer = D / 32;
  __shared__ float join[WARPS > 1 ? WARPS : 1][D + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Desc d = desc[blockIdx.x];
  if (d.parts == 0) return;
  const int lane = threadIdx.x % 32, sub = threadIdx.x / 32 % WARPS;
  const int r = blockIdx.y * (8 / WARPS) + threadIdx.x / 32 / WARPS;  // with WARPS = 8 the same for a whole block
  const int node = d.rt * unit_nodes + r / G, head = d.kvh * G + r % G;
  if (r >= unit_nodes * G || node >= nodes) return;
  const int rank = blockIdx.x % cl;
  auto row_of = [&](int i) { return static_cast<long long>(2 * ((d.c0 + i) * cl + rank) + (i == 0 ? 1 : 0)) * 128 + r; };
  float M = -INFINITY;
  for (int i = lane; i < d.parts; i += 32) M = fmaxf(M, part_ml[2 * row_of(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float acc[kPer] = {}, l = 0.f;
#pragma unroll 8
  for (int i = sub; i < d.parts; i += WARPS) {
    const long long at = row_of(i);
    const float2 ml = reinterpret_cast<const float2*>(part_ml)[at];
    const float w = ml.x == -INFINITY ? 0.f : part_weight(ml.x - M);
    const float* o = part_o + at * D + lane * kPer;
    l = fmaf(ml.y, w, l);
    if (kPer == 4) {
      const float4 v = *reinterpret_cast<const float4*>(o);
      acc[0] = fmaf(v.x, w, acc[0]);
      acc[1] = fmaf(v.y, w, acc[1]);
      acc[kPer - 2] = fmaf(v.z, w, acc[kPer - 2]);
      acc[kPer - 1] = fmaf(v.w, w, acc[kPer - 1]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(o);
      acc[0] = fmaf(v.x, w, acc[0]);
      acc[1] = fmaf(v.y, w, acc[1]);
    }
  }
  if (WARPS > 1) {  // the warps' sums, in their order
#pragma unroll
    for (int e = 0; e < kPer; ++e) join[sub][e * 32 + lane] = acc[e];
    if (lane == 0) join[sub][D] = l;
    __syncthreads();
    if (sub != 0) return;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      l += join[k][D];
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += join[k][e * 32 + lane];
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const long long orow = (static_cast<long long>(d.req) * nodes + node) * Hq + head;
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + (orow * D + lane * kPer) * 2);
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) dst[i] = pack2<BF16>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (lse != nullptr && lane == 0) lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

// More rows: a thread has four columns of a row, a warp eight rows' (one line of a part each load and four columns).
template <int D, bool BF16>
__global__ void __launch_bounds__(256) combine_kernel(const Desc* desc, const float* part_ml, const float* part_o,
                                                      char* out, float* lse, int nodes, int Hq, int G, int unit_nodes,
                                                      int cl) {
  constexpr int kWarps = D / 16;  // that share eight rows
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Desc d = desc[blockIdx.x];
  if (d.parts == 0) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int r = (blockIdx.y * (8 / kWarps) + warp / kWarps) * 8 + lane % 8, i4 = warp % kWarps * 4 + lane / 8;
  const int node = d.rt * unit_nodes + r / G, head = d.kvh * G + r % G;
  if (r >= unit_nodes * G || node >= nodes) return;
  const int rank = blockIdx.x % cl;
  auto slot_of = [&](int i) { return 2 * ((d.c0 + i) * cl + rank) + (i == 0 ? 1 : 0); };
  const float2* mls = reinterpret_cast<const float2*>(part_ml);
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < d.parts; i0 += 4) {  // four parts' loads at once
    float2 ml[4];
    float4 v[4];
    float mx = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool there = i0 + k < d.parts;
      const int slot = slot_of(there ? i0 + k : i0);
      ml[k] = mls[slot * 128 + r];
      v[k] = reinterpret_cast<const float4*>(part_o)[part_at<D, true>(slot, r, i4)];
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
      if (i0 + k >= d.parts) break;
      const float w = ml[k].x == -INFINITY ? 0.f : part_weight(ml[k].x - M);
      l = fmaf(ml[k].y, w, l);
      acc.x = fmaf(v[k].x, w, acc.x);
      acc.y = fmaf(v[k].y, w, acc.y);
      acc.z = fmaf(v[k].z, w, acc.z);
      acc.w = fmaf(v[k].w, w, acc.w);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  const long long orow = (static_cast<long long>(d.req) * nodes + node) * Hq + head;
  *reinterpret_cast<uint2*>(out + (orow * D + 4 * i4) * 2) =
      make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  if (lse != nullptr && i4 == 0) lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

constexpr uint64_t kDescBytes = 152 * sizeof(Desc);
constexpr uint64_t kMlBytes = 2ull * kMaxCtas * 128 * 2 * 4;

template <int D, bool BF16, int REP, bool MC, bool SMALL>
qnre_status_t launch_attention(const AttnArgs& a, int sms, cudaStream_t stream) {
  const auto kernel = attention_kernel<D, BF16, REP, MC, SMALL>;
  // per device, kept: the raised shared-memory limit, and how many clusters of each size are resident at once
  static std::atomic<uint64_t> ready{0};
  static std::atomic<int> resident[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QNRE_ERR_CUDA;
  dev &= 63;
  if (!(ready.load() >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, REP, SMALL>::kBytes) != cudaSuccess)
      return QNRE_ERR_CUDA;
    ready.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads<D, REP>);
  cfg.dynamicSmemBytes = Smem<D, REP, SMALL>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cl;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MC ? 2 : 1;
  int ctas = std::min(sms, kMaxCtas);
  if (MC) {
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
  cfg.gridDim = dim3(ctas);
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return QNRE_ERR_CUDA;
  const int rows = std::min(a.nodes, a.unit_nodes) * a.G;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  // Up to 32 rows a unit leave the machine room for eight warps a row: one request 13.2 us against 15.2, while units
  // of 61 rows take 42 against 37.  More than 64 rows: parts grouped by eight rows, 16 trees of 32 nodes 84 us against
  // 87, units of 61 rows 38.2 against 37.2.
  const auto join = REP == 4   ? combine_few_kernel<D, BF16, 8>
                    : REP == 2 ? combine_few_kernel<D, BF16, 1>
                               : combine_kernel<D, BF16>;
  constexpr int kJoinRows = REP == 4 ? 1 : (REP == 2 ? 8 : 1024 / D);  // a block
  cfg.gridDim = dim3(ctas, (rows + kJoinRows - 1) / kJoinRows);
  return from_cuda(cudaLaunchKernelEx(&cfg, join, static_cast<const Desc*>(a.desc),
                                      static_cast<const float*>(a.part_ml), static_cast<const float*>(a.part_o), a.out,
                                      a.lse, a.nodes, a.Hq, a.G, a.unit_nodes, a.cl));
}

template <int D, bool BF16, bool SMALL>
qnre_status_t launch_rep(const AttnArgs& a, int sms, cudaStream_t stream) {
  const int rows = std::min(a.nodes, a.unit_nodes) * a.G;
  if (a.cl > 1) return launch_attention<D, BF16, 1, true, SMALL>(a, sms, stream);
  if (rows > 64) return launch_attention<D, BF16, 1, false, SMALL>(a, sms, stream);
  if (rows > 32) return launch_attention<D, BF16, 2, false, false>(a, sms, stream);
  return launch_attention<D, BF16, 4, false, false>(a, sms, stream);
}

template <int D, bool BF16>
qnre_status_t launch_size(const AttnArgs& a, int sms, cudaStream_t stream) {
  // only REP = 1 at D = 128 has a use for the smaller table
  return D == 128 && a.n <= 64 ? launch_rep<D, BF16, D == 128>(a, sms, stream) : launch_rep<D, BF16, false>(a, sms, stream);
}

}  // namespace

extern "C" {

qnre_status_t qnre_tree_attention_workspace_bytes(int head_dim, uint64_t* bytes) {
  if (bytes == nullptr) return QNRE_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return QNRE_ERR_UNSUPPORTED;
  *bytes = kDescBytes + kMlBytes + 2ull * kMaxCtas * 128 * head_dim * 4;
  return QNRE_OK;
}

qnre_status_t qnre_tree_attention(const qnre_tensor4_t* q, const qnre_cache_t* cache, int layer, const int32_t* rows,
                                  const uint64_t* mask, const int32_t* counts, float scale, void* out, float* lse,
                                  void* workspace, uint64_t workspace_bytes, qnre_stream_t stream) {
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
      layer >= cache->layers || !(scale > 0.f) || !std::isfinite(scale))
    return QNRE_ERR_INVALID_ARG;
  if (own.shape[2] / cache->heads > kTile) return QNRE_ERR_UNSUPPORTED;
  if (own.shape[1] > QNRE_MAX_NODES || own.shape[2] > 65535) return QNRE_ERR_CAPACITY;
  if (!rows_vectorisable(&own, 2)) return QNRE_ERR_ALIGNMENT;
  uint64_t need = 0;
  qnre_tree_attention_workspace_bytes(cache->head_dim, &need);
  if (empty) return QNRE_OK;
  if (rows == nullptr || out == nullptr || workspace == nullptr) return QNRE_ERR_INVALID_ARG;
  if (!aligned(rows, 4) || !aligned(counts, 4) || !aligned(mask, 8) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return QNRE_ERR_ALIGNMENT;
  if (workspace_bytes < need) return QNRE_ERR_CAPACITY;
  const int64_t out_rows = own.shape[0] * own.shape[1] * own.shape[2];
  const ByteRange ro = span(out, static_cast<uint64_t>(out_rows) * cache->head_dim * 2), rw = span(workspace, need);
  const ByteRange rl = lse != nullptr ? span(lse, static_cast<uint64_t>(out_rows) * 4) : ByteRange{0, 0};
  const ByteRange pools[2] = {span(cache->k, pool_bytes(cache)), span(cache->v, pool_bytes(cache))};
  for (const ByteRange& w : {ro, rw, rl})
    for (const ByteRange& r : {rq, pools[0], pools[1]})
      if (overlaps(w, r)) return QNRE_ERR_ALIAS;
  if (overlaps(ro, rw) || overlaps(ro, rl) || overlaps(rw, rl)) return QNRE_ERR_ALIAS;

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return QNRE_ERR_CUDA;
  if (!own_memory(cache->k, dev) || !own_memory(cache->v, dev)) return QNRE_ERR_INVALID_ARG;

  AttnArgs a{};
  a.c = view_of(cache);
  a.layer = layer;
  a.n = static_cast<int>(own.shape[0]);
  a.nodes = static_cast<int>(own.shape[1]);
  a.Hq = static_cast<int>(own.shape[2]);
  a.Hk = cache->heads;
  a.G = a.Hq / a.Hk;
  a.unit_nodes = kTile / a.G;
  const int row_tiles = (a.nodes + a.unit_nodes - 1) / a.unit_nodes;
  a.cl = std::min(row_tiles, kMaxCluster);
  a.row_groups = (row_tiles + a.cl - 1) / a.cl;
  const int64_t tiles = (static_cast<int64_t>(cache->max_blocks) * cache->page_size + kTile - 1) / kTile + kUnitCost;
  if (a.n * tiles * a.Hk * a.row_groups > 0x7FFFFFFF) return QNRE_ERR_CAPACITY;
  a.box = std::min(a.cl > 1 ? kTile / kMaxCluster : kTile, cache->page_size & -cache->page_size);
  a.rows = rows;
  a.counts = counts;
  a.mask = mask;
  a.out = static_cast<char*>(out);
  a.lse = lse;
  a.desc = static_cast<Desc*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + kDescBytes);
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kDescBytes + kMlBytes);
  a.scale_log2 = scale * 1.4426950408889634f;
  const bool bf16 = cache->dtype == QNRE_DTYPE_BF16;
  const uint64_t D = cache->head_dim, ps = cache->page_size, H = cache->heads;
  const uint64_t dims[4] = {D, ps, H, static_cast<uint64_t>(cache->layers) * cache->pages};
  const uint64_t strides[3] = {D * 2, ps * D * 2, H * ps * D * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(a.box), 1, 1};
  const uint64_t q_dims[4] = {D, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.nodes), static_cast<uint64_t>(a.n)};
  const uint64_t q_strides[3] = {static_cast<uint64_t>(own.stride[2]) * 2, static_cast<uint64_t>(own.stride[1]) * 2,
                                 static_cast<uint64_t>(own.stride[0]) * 2};
  const uint32_t q_box[4] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(std::min(a.nodes, a.unit_nodes)), 1};
  if (!encode_tiled_16bit(&a.tq, own.data, bf16, 4, q_dims, q_strides, q_box) ||
      !encode_tiled_16bit(&a.tk, cache->k, bf16, 4, dims, strides, box) ||
      !encode_tiled_16bit(&a.tv, cache->v, bf16, 4, dims, strides, box))
    return QNRE_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) return bf16 ? launch_size<128, true>(a, sms, s) : launch_size<128, false>(a, sms, s);
  return bf16 ? launch_size<64, true>(a, sms, s) : launch_size<64, false>(a, sms, s);
}

}  // extern "C"
