// kv_window_attn and kv_prefix_attn: causal attention of packed new tokens on
// tcgen05 tensor cores.
//
//   out[t,h,:] = sum_{j in A(t)} softmax_j(q[t,h].K_j / sqrt(d)) V_j
// with A(t) the sink and the newest `local` tokens up to t's own position, or
// a shared prefix and everything up to t's own position behind it.
//
// Rows.  The queries of a KV head's group share its keys, so the rows of one
// product are (token, head of the group): 256 rows, two 128-row tiles, are an
// item's queries.  Keys come in tiles of 128 tokens; an item walks the tiles
// that some row of it attends to (prefix, sink, window), one pass, with the
// running maximum and sum of every row in registers:
//   S = Q K^T        128 x 128, K = d        operands in shared memory
//   P = exp2(S c - m c) in bf16, written over S in TMEM
//   O += P V         128 x d, K = tokens     P from TMEM, V read MN-major
// O stays in TMEM; it is rescaled only when a row's maximum has grown by more
// than 2^8 since the exponents were last based (the factor cancels in the
// final division, and fp32 and bf16 hold 2^8 as well as 1).  P is rounded to
// bf16, the type that its product with V takes (at most 2^-8 of each weight, the
// size of the bf16 output's own rounding; on random values the two together are
// 1.35 times the rounding alone); the sum that divides takes the unrounded fp32
// values, so lse is as exact as fp32.
//
// Work.  Two schedules, chosen by the numbers of rows and tiles (attn_schedule):
//   whole  many items, or short ones: each CTA takes one of every round of G
//          items whole, from the batch's end to its beginning (a sequence's last
//          query tiles attend to the most keys; different sequences are not
//          weighed against each other), every other round in reverse (items of
//          128 rows where those of 256 are few, and those in twos where there are
//          several to an SM).
//   split  few items: the tiles of all items are laid end to end and every CTA
//          takes an equal range of that line; an item that several CTAs share
//          leaves partial (max, sum, O) rows in the workspace and kv_merge_kernel
//          joins them.  With a shared prefix its queries are one sequence of
//          their own (all tokens of the batch, 256 rows to an item), so that
//          the prefix is read once per 256 rows and not once per sequence (from
//          HBM once for all: see tile_of).
// The line is planned on the device from the lengths, of which the host knows
// nothing: by a warp of every CTA for itself, or by kv_plan_kernel for a batch
// whose plan does not fit beside the tiles.  Whole items of single tokens need no
// plan.
//
// Roles (384 threads):
//   warps 0-3, 4-7  softmax: group s owns accumulators S_s and O_s, thread r
//            row r.  An item of more than 128 rows gives each group a query
//            tile (pair); a smaller one gives the groups alternate key tiles
//            (parity), each with its own statistics and O, joined by group 0 or
//            (of a share) by the merge; or two such items, of neighbouring KV
//            heads, get a group each (dual), which hides the start and end of
//            short items behind each other.
//   warp 8   K loads, warp 9  V loads (TMA, 64-row boxes: a page holds at least
//            64 tokens, so a box never leaves its page).  Boxes that no row
//            attends to are not loaded.  One ring of five tiles, in the order of
//            use.
//   warp 10  MMA issue.
//   warp 11  the plan, the CTA's shares (handed to the others through a queue of
//            four) and their query loads.
// Rows of V that no row of the item attends to may hold anything (0 x NaN is
// NaN): the softmax threads zero them in shared memory.
//
// Bounds.  Prefill: the tensor cores.  4 d FLOP per query row and key; S has both
// operands in shared memory, 128 bytes a cycle, all that there is.  One tile of
// two query tiles takes 2048 cycles at their full rate and 3100 to 3300 here:
// what is left are the waits between softmax and products (a row's softmax takes
// 1100 cycles to its first half, 1500 to its second, and each group's products
// 1024).  Measured among others of its kind, the power cap active: 8192 causal
// tokens, 64 heads: 715 to 765 us, 1440 to 1540 TFLOP/s (75 to 80 % of cuBLAS's burst
// rate, 84 to 89 % of its sustained one); 32768 tokens, 32 heads, a window of
// 4096: 1370 to 1400 us, 1480 to 1510 TFLOP/s of useful products (3 % more are
// computed at the window's edges).  The comparisons beside the code were timed
// in short runs, in which the first of these takes 660 to 680 us.  ncu (4096
// tokens): tensor pipe 63 % of its active peak, special functions 32 %, issue 42
// %, DRAM 7 %.
// Decode: HBM.  64 sequences, a window of 4096, 8 KV heads (0.99 GB): 149 to 154 us,
// 6.5 TB/s (97 % of a copy's rate); one sequence of 131072 tokens (0.54 GB): 87 us.
// ncu: 382 MB read where 373 are needed.
// Few tokens: latency.  4 sequences' 260 tokens: 8.9 us on the GPU: the
// first item takes 1.1, its first key 1.7, a tile 0.7 to 1.4 (and a plan, where
// one is needed, 0.6).  16 ragged sequences of 1 to 64 tokens, up to 1400 cached: 16 us with items of 128
// rows, joined in the block; with 256-row items and a join by the merge 30.
// A shared prefix: 128 sequences over 131072 tokens, 32 heads: 252 to 268 us.
#include <cuda.h>

#include <algorithm>
#include <climits>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace qasc {
namespace {

constexpr int kTile = 128;                    // tokens of a key tile, rows of a query tile
constexpr int kItemRows = 2 * kTile;
constexpr int kHalf = kTile * 128;            // 128 rows x 64 bf16 columns
constexpr int kTileBytes = 2 * kHalf;
constexpr int kBox = 64;                      // rows of a K / V box
constexpr int kBoxBytes = kBox * 128;
constexpr int kSlots = 5;                     // ring of K and V tiles
constexpr int kKWarp = 8, kVWarp = 9, kMmaWarp = 10, kQWarp = 11;
constexpr int kThreads = 384;
// Registers: 384 threads start with 168 each (64512); the softmax warpgroups
// take 200 and the third keeps 104, the same sum.
constexpr int kSoftRegs = 200, kOtherRegs = 104;
constexpr int kTmemCols = 512;                // S_0, S_1, O_0, O_1
constexpr int kMaxSeq = 2048 + 1;             // sequences of the plan (the shared prefix is one)
constexpr int kMaxEnt = 4608;                 // items per KV head of a split plan (see may_split)
constexpr int kPlanWords = 320;               // of the plan that fit into shared memory beside the ring
constexpr int kQueue = 4;                     // pieces handed out ahead
constexpr int kPieceReaders = 11;             // warps that take them: K, V, MMA, softmax
// Places of an item on the line: kItemCost for what it costs beside its tiles
// (queries, the first tile's latency, the output), then one per tile, or two
// of a pair item.  Measured at one, two, three places: 128 sequences over a 128K
// prefix 250, 237, 254 us, over a 4K prefix 42, 43, 47; 8 over 8K 20.1, 19.5, 18.5.
constexpr int kItemCost = 2;
constexpr int kChunks = kD / 4;               // 16-byte chunks of a partial row
// log2(e) / sqrt(128): logits in base-2 units.
constexpr float kScale = 1.4426950408889634f * 0.08838834764831845f;
constexpr float kRebase = 8.0f;               // growth of a row's maximum (log2) that rescales O

struct Args {
  KvAttnArgs a;
  int B, Hq, Hkv, gsh;      // gsh = log2(Hq / Hkv)
  int64_t n_cap;
  int item_rows;            // query rows of an item: 256, or 128 (whole only)
  int dual;                 // whole items (of 128 rows) in twos: a unit is two neighbouring KV heads
  int uniform;              // whole items of single tokens: one per sequence and KV head, no plan
  int once;                 // keys are read by one item, or two
  int split, pre;           // pre: the shared prefix is sequence 0 of the plan (split only)
  int slot_rows;            // partial rows a CTA may add to an item (split)
  float4* part_o;           // [rows][32] of a share: element (row, chunk) at chunk * rows + row
  float2* part_ml;          // [rows] (max in log2 units, sum)
  int32_t* ent_base;        // [kMaxSeq + 1] the plan in global memory: written by kv_plan_kernel, or by
  int32_t* line;            // [kMaxEnt + 1] CTA 0 for the merge
  int4* info;               // [kMaxEnt] per entry: first token of the sequence, first row, rows, sequence (< 0: prefix)
  int max_ent;              // entries that T tokens of B sequences can make (malformed cu_q is cut to it)
  int plan_global;          // the plan is too large for shared memory
  unsigned* err;
};

// A CTA's share of an item, as its roles take it: key tiles k0 .. k0 + n - 1.
struct alignas(16) Piece {
  int tok0, rows;     // first query token, rows
  int g, b;           // KV head, sequence (< 0: the shared prefix)
  int p0, p1;         // positions of the first and last row
  int lo, hi;         // own tokens attended by some row: [0, min(sink, hi + 1)) and [lo, hi]
  int np, ns, w0;     // tiles of the prefix; boxes of the sink in front of the window, first box of the window
  int k0, n;          // n < 0: no more pieces
  int flags;
  int64_t part;       // first partial row
};
constexpr int kPair = 1;    // two query tiles, one per group; else the groups take alternate key tiles of one
constexpr int kWhole = 2;   // every tile of the item: the output is written, not a partial
constexpr int kTurn = 4;    // the first tile of a parity piece is group 1's
constexpr int kDual = 8;    // the items of KV heads g and g + 1, one per group: their tiles alternate in the ring

struct Smem {
  uint8_t q[2][kTileBytes];
  uint8_t kv[kSlots][kTileBytes];
  Piece piece[kQueue];
  uint64_t pc_full[kQueue], pc_empty[kQueue];
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[2], p_full[2][2], o_full[2];   // p_full: the first and last 64 tokens
  uint64_t x_full, x_empty;                      // group 1's part of a whole parity item is there, is taken
  float2 x_ml[kTile];                            // its rows' (max in log2 units, sum)
  uint32_t tmem_base;
  int32_t plan[kPlanWords];
  uint64_t mma_done;                             // every product of the CTA is complete (where a wait ran out)
  uint4 last[3];                                 // what the loaders (K, V, queries) issued last
  int32_t failed;                                // a wait ran out
};

static_assert(sizeof(Smem) <= 232448, "shared memory of a block");

// ent_base[s]: items per KV head before sequence s (split).  line: places
// before entry e, all KV heads (split); items before sequence s (whole).
struct Plan {
  const int32_t* ent_base;
  const int32_t* line;
  int entries;
};

struct Seq {
  int q0, ql, len, b;   // first token, tokens, cached tokens; b < 0: the shared prefix
};

__device__ __forceinline__ int clampi(int64_t v, int64_t lo, int64_t hi) {
  return static_cast<int>(v < lo ? lo : (v > hi ? hi : v));
}

__device__ __forceinline__ Seq seq_of(const Args& p, int s) {
  const Batch& bt = p.a.bt;
  Seq r;
  if (p.pre && s == 0) {
    r.b = -1;
    r.q0 = bt.cu_q ? clampi(__ldg(bt.cu_q), 0, bt.T) : 0;
    r.ql = (bt.cu_q ? clampi(__ldg(bt.cu_q + bt.B), r.q0, bt.T) : static_cast<int>(bt.T)) - r.q0;
    r.len = static_cast<int>(p.a.n_prefix);
    return r;
  }
  r.b = s - p.pre;
  if (bt.cu_q) {
    r.q0 = clampi(__ldg(bt.cu_q + r.b), 0, bt.T);
    r.ql = clampi(__ldg(bt.cu_q + r.b + 1), r.q0, bt.T) - r.q0;
  } else {
    r.q0 = r.b;
    r.ql = 1;
  }
  r.len = clampi(__ldg(bt.lens + r.b), 0, p.n_cap);
  return r;
}

// Query rows r0 .. r0 + rows - 1 of a sequence for a KV head, and the key
// tiles that they attend to: np of the prefix, ns of the sink in front of the
// window, then those of the window from w0 on.
struct Item {
  Seq s;
  int r0, rows;
  int p0, p1;         // positions of the first and last row
  int lo, hi;         // own tokens attended by some row: [0, min(sink, hi + 1)) and [lo, hi]
  int np, ns, w0, cnt;
};

__device__ __forceinline__ int ceil_tiles(int64_t n) { return static_cast<int>((n + kTile - 1) / kTile); }

__device__ __forceinline__ Item make_item(const Args& p, const Seq& s, int qt) {
  Item it;
  it.s = s;
  it.r0 = qt * p.item_rows;
  it.rows = min(p.item_rows, (s.ql << p.gsh) - it.r0);
  it.ns = 0;
  it.w0 = 0;
  it.p0 = s.len - s.ql + (it.r0 >> p.gsh);
  it.p1 = s.len - s.ql + ((it.r0 + it.rows - 1) >> p.gsh);
  it.lo = 0;
  it.hi = -1;
  if (s.b < 0) {
    it.np = ceil_tiles(p.a.n_prefix);
    it.cnt = it.np;
    return it;
  }
  it.np = p.pre ? 0 : ceil_tiles(p.a.n_prefix);
  it.cnt = it.np;
  if (it.p1 >= 0) {
    const int64_t lo = static_cast<int64_t>(it.p0) - p.a.local + 1;
    it.lo = static_cast<int>(lo > 0 ? lo : 0);
    it.hi = it.p1;
    it.w0 = it.lo / kBox;
    it.ns = min(min(p.a.sink, it.hi + 1) / kBox + (min(p.a.sink, it.hi + 1) % kBox > 0), it.w0);
    // With an odd number of boxes an empty one stands behind the sink's, not at
    // the end: the window's tiles are then likely to be attended to in full.
    if (it.ns < it.w0 && it.ns > 0 && ((it.ns + it.hi / kBox - it.w0 + 1) & 1)) --it.w0;
    it.cnt += (it.ns + it.hi / kBox - it.w0 + 2) / 2;
  }
  return it;
}

// The i-th key tile of a piece of n.  A share of the prefix begins at its tile
// w0 and goes around: a tile comes up at the same time in every share that holds
// it, those of the prefix's other items, so that it is read from HBM once (128
// sequences of 4 rows a KV head over a 128K prefix: 237 us, 255 without; 256 of
// them 383 and 422).
template <bool kSplit>
__device__ __forceinline__ int tile_of(const Piece& pc, int i, int n) {
  if (kSplit && pc.b < 0) {
    i += pc.w0;
    if (i >= n) i -= n;
  }
  return pc.k0 + i;
}

// Key tile k of an item is two boxes of 64 tokens: the first token of one, and
// whether it is of the prefix.  An item's own boxes are those of the sink, then
// those of the window, so that a sink of a few tokens takes half a tile (a box
// behind the last one begins behind hi).
__device__ __forceinline__ int box_token(const Piece& pc, int k, int half, bool* prefix) {
  *prefix = k < pc.np;
  const int b = 2 * (k < pc.np ? k : k - pc.np) + half;
  return (k < pc.np || b < pc.ns ? b : pc.w0 + b - pc.ns) * kBox;
}

// Token j (of a prefix tile or an own one) is attended by some row of the item.
__device__ __forceinline__ bool any_row_sees(const Args& p, const Piece& pc, bool prefix, int j) {
  if (prefix) return j < p.a.n_prefix;
  return j <= pc.hi && (j >= pc.lo || j < p.a.sink);
}
// The same for any token of [j, j + kBox).
__device__ __forceinline__ bool any_row_sees_box(const Args& p, const Piece& pc, bool prefix, int j) {
  if (prefix) return j < p.a.n_prefix;
  return j <= pc.hi && (j + kBox > pc.lo || j < p.a.sink);
}

__device__ __forceinline__ int tile_weight(int rows) { return rows > kTile ? 2 : 1; }
// Place of an item's first and last tile on its span (an empty item: its last place).
__device__ __forceinline__ int first_place(int span) { return min(kItemCost, span - 1); }
__device__ __forceinline__ int last_place(int span, int w) { return span > kItemCost ? span - w : span - 1; }

// A line of U places over G <= 2^15 CTAs: CTA c has the places
// [c U / G, (c + 1) U / G).  In 32 bits, with U = q G + r.
struct Ranges {
  unsigned U, G, q, r;
  __device__ __forceinline__ Ranges(int places, int grid) {
    U = places;
    G = min(grid, places);
    q = U / G;
    r = U - q * G;
  }
  __device__ __forceinline__ int start(unsigned c) const { return static_cast<int>(c * q + c * r / G); }
  // The CTA that holds place x.
  __device__ __forceinline__ int cta(int x) const {
    int c = min(static_cast<int>(__fdividef(static_cast<float>(x) * static_cast<float>(G), static_cast<float>(U))),
                static_cast<int>(G) - 1);
    while (start(c) > x) --c;
    while (start(c + 1) <= x) ++c;
    return c;
  }
};

// Last i in [0, n) with arr[i] <= x (arr ascending, arr[0] <= x).
__device__ __forceinline__ int find_last(const int32_t* arr, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (arr[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int q_tiles(const Args& p, const Seq& s) {
  if (p.a.skip_empty && s.len == 0) return 0;
  return ((s.ql << p.gsh) + p.item_rows - 1) / p.item_rows;
}

// Exclusive prefix sums of f(0) .. f(n - 1) into arr[0 .. n], by a warp or
// (kBlock) a block, whose first warp does the adding.
template <bool kBlock, class F>
__device__ __forceinline__ void plan_scan(int32_t* arr, int n, F&& f) {
  const int lane = threadIdx.x & 31;
  if (kBlock) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) arr[i] = f(i);
    __syncthreads();
  }
  if (!kBlock || threadIdx.x < 32) {
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane, v = i < n ? (kBlock ? arr[i] : f(i)) : 0;
      int inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += w;
      }
      if (i < n) arr[i] = carry + inc - v;
      carry += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) arr[n] = carry;
  }
  if (kBlock) __syncthreads();
  else __syncwarp();
}

__device__ __forceinline__ void check_lens(const Args& p, int first, int step) {
  for (int b = first; b < p.B; b += step) {
    const int v = __ldg(p.a.bt.lens + b);
    if (v < 0 || v > p.n_cap) record_error(p.err, kErrBadPage);
  }
}

// The plan in shared memory, by a warp or a block: ent_base [NS + 1] and line
// [entries + 1].  Places are counted in 32 bits: an item has at most 2 n_cap / 128
// + 6 of its own tiles, and with B Hkv n_cap < 2^31 and n_cap < 2^24, which every
// call checks, the last items of the sequences have below 2^26 together, all
// others of a split (may_split) below 2^29; those of a prefix have below 2^29 +
// 2^25 with T Hq n_prefix < 2^43, which its call checks.  `publish`: the copies in global memory (for the merge, and
// for a batch whose plan the attention's CTAs cannot hold), and the check of
// the lengths.
template <bool kBlock>
__device__ __forceinline__ int make_plan(const Args& p, int32_t* ent_base, int32_t* line, bool publish) {
  const int NS = p.B + p.pre, first = kBlock ? threadIdx.x : threadIdx.x & 31, step = kBlock ? blockDim.x : 32;
  if (publish) check_lens(p, first, step);
  if (!p.split) {
    plan_scan<kBlock>(line, NS, [&](int s) { return q_tiles(p, seq_of(p, s)) * (p.Hkv >> p.dual); });
    if (kBlock)
      for (int s = first; s <= NS; s += step) p.line[s] = line[s];
    return NS;
  }
  plan_scan<kBlock>(ent_base, NS, [&](int s) { return q_tiles(p, seq_of(p, s)); });
  const int entries = min(ent_base[NS], p.max_ent);
  plan_scan<kBlock>(line, entries, [&](int e) {
    const int s = find_last(ent_base, NS, e);
    const Item it = make_item(p, seq_of(p, s), e - ent_base[s]);
    if (publish) p.info[e] = make_int4(it.s.q0, it.r0, it.rows, it.s.b);
    return (it.cnt * tile_weight(it.rows) + kItemCost) * p.Hkv;
  });
  if (publish) {
    for (int e = first; e <= entries; e += step) p.line[e] = line[e];
    for (int s = first; s < NS; s += step) p.ent_base[s] = min(ent_base[s], entries);
    if (first == 0) p.ent_base[NS] = entries;
  }
  return entries;
}

// First partial row of an item's share of CTA c.  Two rows of the area belong
// to every query row (each group leaves one of a parity item), ordered as the
// line is; each CTA crossed adds slot_rows, the most rows of one share, so that
// no two shares overlap.
__device__ __forceinline__ int64_t part_row(const Args& p, const Item& it, int g, int cta) {
  const int64_t fam = p.pre && it.s.b >= 0 ? p.a.bt.T * p.Hq : 0;   // the prefix's shares stand first
  const int64_t row = fam + static_cast<int64_t>(it.s.q0) * p.Hq + static_cast<int64_t>(it.r0) * p.Hkv +
                      static_cast<int64_t>(g) * it.rows;
  return 2 * row + static_cast<int64_t>(cta) * p.slot_rows;
}

// The group of a parity piece's first tile.  Of a split they go on alternating
// from piece to piece: while one group writes a short piece's rows the other has
// the next piece's tile.
template <bool kSplit>
__device__ __forceinline__ int first_group(const Piece& pc) {
  return kSplit && (pc.flags & (kTurn | kDual)) == kTurn ? 1 : 0;
}

// The shares of this CTA in order.
template <bool kSplit>
struct Walk {
  int pos, end, n;   // split: place on the line, its end; whole: round
  int e, s;          // split: current entry and its sequence
  __device__ __forceinline__ int units(const Args& p, const Plan& S) const {
    return !kSplit && p.uniform ? n * (p.Hkv >> p.dual) : S.line[n];
  }
  __device__ __forceinline__ void init(const Args& p, const Plan& S) {
    n = S.entries;
    pos = end = 0;
    if (n == 0) return;
    const int U = units(p, S);
    if (kSplit) {
      const Ranges line(U, gridDim.x);
      if (blockIdx.x >= line.G) return;
      pos = line.start(blockIdx.x);
      end = line.start(blockIdx.x + 1);
      e = find_last(S.line, n, pos);
      s = find_last(S.ent_base, p.B + p.pre, e);
    } else {
      end = (U + gridDim.x - 1) / gridDim.x;
    }
  }
  __device__ __forceinline__ bool next(const Args& p, const Plan& S, Piece& pc) {
    Item it;
    int g;
    if (kSplit) {
      int off, take, span, w;
      while (true) {
        if (pos >= end) return false;
        while (S.line[e + 1] <= pos) ++e;
        while (S.ent_base[s + 1] <= e) ++s;
        span = (S.line[e + 1] - S.line[e]) / p.Hkv;
        const int rem = pos - S.line[e];
        g = rem / span;
        off = rem - g * span;
        take = min(span - off, end - pos);
        pos += take;
        it = make_item(p, seq_of(p, s), e - S.ent_base[s]);
        w = tile_weight(it.rows);
        if (off + take > first_place(span) && off <= last_place(span, w)) break;   // not the item's cost alone
      }
      // a tile belongs to the share that holds its first place
      pc.k0 = (max(0, off - kItemCost) + w - 1) / w;
      pc.n = (max(0, off + take - kItemCost) + w - 1) / w - pc.k0;
      const bool pair = it.rows > kTile;
      const bool all = off <= first_place(span) && off + take > last_place(span, w);
      pc.flags = (pair ? kPair : 0) | (pair && !p.pre && all ? kWhole : 0);
      pc.part = part_row(p, it, g, blockIdx.x);
      if (!pair && all && it.cnt > 0 && g + 1 < p.Hkv && end - pos >= span) {   // the next head's item as well
        pc.flags |= kDual;
        pos += span;
      }
    } else {
      const int U = n > 0 ? units(p, S) : 0;
      int u;
      do {
        if (pos >= end) return false;
        // rounds alternate direction, so that a CTA with a heavy item gets a light one next
        u = pos * static_cast<int>(gridDim.x) +
            ((pos & 1) ? static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
        ++pos;
      } while (u >= U);
      const int x = U - 1 - u;   // late query tiles attend to the most keys
      const int heads = p.Hkv >> p.dual;
      const int sq = p.uniform ? x / heads : find_last(S.line, n, x), rem = x - (p.uniform ? sq * heads : S.line[sq]);
      it = make_item(p, seq_of(p, sq), rem / heads);
      g = (rem % heads) << p.dual;
      pc.k0 = 0;
      pc.n = it.cnt;
      pc.flags = (it.rows > kTile ? kPair : 0) | kWhole | p.dual * kDual;
      pc.part = 0;
    }
    pc.tok0 = it.s.q0 + (it.r0 >> p.gsh);
    pc.rows = it.rows;
    pc.g = g;
    pc.b = it.s.b;
    pc.p0 = it.p0;
    pc.p1 = it.p1;
    pc.lo = it.lo;
    pc.hi = it.hi;
    pc.np = it.np;
    pc.ns = it.ns;
    pc.w0 = it.w0;
    if (kSplit && it.s.b < 0) {
      // the first tile in the share of which a CTA's places on an item's span begin a multiple of a share's length
      const Ranges line(S.line[n], gridDim.x);
      const int w = tile_weight(it.rows);
      const unsigned m = static_cast<unsigned>((static_cast<uint64_t>(pc.k0) * w * line.G + line.U - 1) / line.U);
      const int first = (line.start(m) + w - 1) / w - pc.k0;
      pc.w0 = first > 0 && first < pc.n ? first : 0;
    }
    return true;
  }
};

// Places of K_i and V_i of a piece of n tiles in the ring: `ahead` K tiles
// stand in front, then V_k and K_{k + ahead} in turn.
__device__ __forceinline__ uint32_t k_place(int i, int ahead) { return i < ahead ? i : 2 * i - ahead + 1; }
__device__ __forceinline__ uint32_t v_place(int i, int n, int ahead) { return min(n, i + ahead) + i; }

// 3-D tiled tensor copy: x innermost (elements), y, z.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// 32 columns of this thread's TMEM lane, from registers r[0 .. 32).
#define KV_TMEM_LD32(addr, r)                                                                                         \
  asm volatile(                                                                                                       \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"       \
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                                              \
      : "=f"((r)[0]), "=f"((r)[1]), "=f"((r)[2]), "=f"((r)[3]), "=f"((r)[4]), "=f"((r)[5]), "=f"((r)[6]),             \
        "=f"((r)[7]), "=f"((r)[8]), "=f"((r)[9]), "=f"((r)[10]), "=f"((r)[11]), "=f"((r)[12]), "=f"((r)[13]),         \
        "=f"((r)[14]), "=f"((r)[15]), "=f"((r)[16]), "=f"((r)[17]), "=f"((r)[18]), "=f"((r)[19]), "=f"((r)[20]),      \
        "=f"((r)[21]), "=f"((r)[22]), "=f"((r)[23]), "=f"((r)[24]), "=f"((r)[25]), "=f"((r)[26]), "=f"((r)[27]),      \
        "=f"((r)[28]), "=f"((r)[29]), "=f"((r)[30]), "=f"((r)[31])                                                    \
      : "r"(addr))
#define KV_TMEM_ST32(addr, r)                                                                                         \
  asm volatile(                                                                                                       \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"    \
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),                                   \
      "r"((r)[0]), "r"((r)[1]), "r"((r)[2]), "r"((r)[3]), "r"((r)[4]), "r"((r)[5]), "r"((r)[6]), "r"((r)[7]),         \
      "r"((r)[8]), "r"((r)[9]), "r"((r)[10]), "r"((r)[11]), "r"((r)[12]), "r"((r)[13]), "r"((r)[14]),                 \
      "r"((r)[15]), "r"((r)[16]), "r"((r)[17]), "r"((r)[18]), "r"((r)[19]), "r"((r)[20]), "r"((r)[21]),               \
      "r"((r)[22]), "r"((r)[23]), "r"((r)[24]), "r"((r)[25]), "r"((r)[26]), "r"((r)[27]), "r"((r)[28]),               \
      "r"((r)[29]), "r"((r)[30]), "r"((r)[31])                                                                       \
      : "memory")
// Wait for this thread's TMEM loads; r[0 .. 32) may be used from here on (an
// asm statement that names them, so that no use moves in front of the wait).
#define KV_TIE16(r)                                                                                                   \
  asm volatile(""                                                                                                     \
               : "+f"((r)[0]), "+f"((r)[1]), "+f"((r)[2]), "+f"((r)[3]), "+f"((r)[4]), "+f"((r)[5]), "+f"((r)[6]),    \
                 "+f"((r)[7]), "+f"((r)[8]), "+f"((r)[9]), "+f"((r)[10]), "+f"((r)[11]), "+f"((r)[12]),               \
                 "+f"((r)[13]), "+f"((r)[14]), "+f"((r)[15]))
#define KV_TIE32(r)     \
  do {                  \
    KV_TIE16(r);        \
    KV_TIE16((r) + 16); \
  } while (0)
#define KV_TMEM_WAIT32(r) \
  do {                    \
    tmem_wait_ld();       \
    KV_TIE32(r);          \
  } while (0)
#define KV_TMEM_ST16(addr, r)                                                                                         \
  asm volatile(                                                                                                       \
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::    \
          "r"(addr),                                                                                                  \
      "f"((r)[0]), "f"((r)[1]), "f"((r)[2]), "f"((r)[3]), "f"((r)[4]), "f"((r)[5]), "f"((r)[6]), "f"((r)[7]),         \
      "f"((r)[8]), "f"((r)[9]), "f"((r)[10]), "f"((r)[11]), "f"((r)[12]), "f"((r)[13]), "f"((r)[14]), "f"((r)[15])   \
      : "memory")
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bounded wait of a whole warp.  All lanes try and vote, so that the warp
// never diverges: a wait by one lane, or a loop that lanes leave one by one,
// costs the product pipeline more than the tries do (8192 causal tokens of 64
// heads: 888 us with one lane waiting, 742 with a loop per lane, 710 so).  The
// tries without a suspend-time hint wake sooner (745 us with one).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity,
                                          unsigned long long limit_ns = kWaitTimeoutNs) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) return false;
  return true;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Behind the roles, where a wait ran out, of any warp: the issuers wait for the
// loads and products that they have in flight (otherwise the warp that uses
// them has), so that nothing writes into shared or tensor memory that is the
// next block's by then.  Of the ring's five tiles at most four are one loader's.
// (A call of its own, since the code of the roles is sensitive to what stands
// behind them: inlined, 128 sequences over a 128K prefix took 264 us, 258 so; as
// unconditional waits in the roles it cost decoding 1.3 %.)
__device__ __noinline__ void finish_issued(Smem& S, int warp) {
  if (warp == kKWarp || warp == kVWarp) {
    const uint4 at = S.last[warp - kKWarp];   // places + 1
    auto done = [&](uint32_t x) {
      if (x > 0) wait_warp(&S.full[(x - 1) % kSlots], ((x - 1) / kSlots) & 1u);
    };
    done(at.x);
    done(at.y);
    done(at.z);
    done(at.w);
  } else if (warp == kQWarp) {
    const uint4 n = S.last[2];
    if (n.x > 0) wait_warp(&S.q_full[0], (n.x - 1) & 1u);
    if (n.y > 0) wait_warp(&S.q_full[1], (n.y - 1) & 1u);
  } else if (warp == kMmaWarp) {
    if (elect_one()) mma_commit(&S.mma_done);   // the lane that issued
    wait_warp(&S.mma_done, 0);
  }
}

// Bits [0, n) of a word, n any integer.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// Three kernels, since the code of one schedule costs the others: with the join
// of whole parity items in the split's kernel 128 sequences over a 128K prefix
// took 297 us, without it 262; 608 sequences of one 36-token item a KV head take
// 97 us in a kernel of twos alone, 108 in one that also holds whole pair items.
enum Mode { kModeSplit, kModeWhole, kModeTwos };

// kTest: the waits give up after p.a.wait_ns, and the tile at place p.a.stall of
// the ring never comes (the failure path of every role, without a fault).
template <Mode kMode, bool kTest = false>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attn_kernel(const Args p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  constexpr bool kSplit = kMode == kModeSplit;
  auto is_pair = [](const Piece& pc) { return kMode != kModeTwos && (pc.flags & kPair) != 0; };
  auto is_dual = [](const Piece& pc) {   // 0, 1
    return kMode == kModeTwos || (kMode == kModeSplit && (pc.flags & kDual)) ? 1 : 0;
  };
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem_raw) & 1023u) {   // the tiles' swizzle counts from here; the whole block leaves
    record_error(p.err, kErrInternal);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&S.pc_full[i], 1);
      mbar_init(&S.pc_empty[i], kPieceReaders);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i][0], 4);
      mbar_init(&S.p_full[i][1], 4);
      mbar_init(&S.o_full[i], 1);
    }
    mbar_init(&S.x_full, 4);
    mbar_init(&S.x_empty, 4);
    mbar_init(&S.mma_done, 1);
    S.failed = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == kMmaWarp) tmem_alloc(&S.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  pdl_wait();
  uint32_t ring = 0;     // K and V tiles of the CTA so far: slot ring mod kSlots
  uint32_t pieces = 0;   // pieces taken
  uint32_t uses[2] = {0, 0};   // of the query buffers
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (dead) return;
    if (!wait_warp(bar, parity, kTest ? p.a.wait_ns : kWaitTimeoutNs)) {
      record_error(p.err, kErrTimeout);
      dead = true;
    }
  };
  Piece pc;
  // The next piece, copied; false behind the last.
  auto take = [&]() {
    const uint32_t i = pieces % kQueue;
    wait(&S.pc_full[i], (pieces / kQueue) & 1u);
    if (dead) return false;
    pc = S.piece[i];
    ++pieces;
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.pc_empty[i]);
    return pc.n >= 0;
  };
  // Query buffer of a parity piece (they alternate, so that the next piece's
  // queries load while this one's are in use); a pair's tiles have both.
  auto q_buffer = [&]() { return (uses[0] + uses[1]) & 1u; };
  if (warp >= kKWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kKWarp || warp == kVWarp) {
      // ---- K loads, V loads: lanes 0-3 issue the two 64-column halves of the two boxes
      const bool is_k = warp == kKWarp;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      const int h = (lane >> 1) & 1, half = lane & 1;
      // Where a sequence has few rows its keys are read once: they are the first
      // to leave L2 (32 sequences over a 32K prefix: 45 us, 50 without
      // the hint; 54 with tiles prefetched into L2 ahead of the ring).  Whole
      // items share their keys (677 against 667 us with the hint).
      const uint64_t once = policy_evict_first();
      uint32_t mine[4] = {0, 0, 0, 0};   // places + 1 of this warp's newest loads
      while (take()) {
        const int dual = is_dual(pc), n = pc.n << dual, ahead = is_pair(pc) ? 1 : 2;
        int64_t row = -1;   // of lane's box of 16 tiles from tile i on; -1: no row attends to the box
        for (int i = 0; i < n; ++i) {
          if ((i & 15) == 0) {
            const int j = i + (lane >> 1), k = tile_of<kSplit>(pc, j >> dual, pc.n);
            row = -1;
            if (j < n) {
              bool prefix;
              const int tok = box_token(pc, k, lane & 1, &prefix);
              if (any_row_sees_box(p, pc, prefix, tok)) {
                row = cache_row(prefix ? p.a.pm_prefix : p.a.pm, prefix ? 0 : pc.b, pc.g + (j & dual), p.Hkv, p.n_cap, tok);
                if (row < 0) {
                  record_error(p.err, kErrBadPage);
                  row = 0;
                }
              }
            }
          }
          const int64_t row0 = __shfl_sync(0xffffffffu, row, 2 * (i & 15));
          const int64_t row1 = __shfl_sync(0xffffffffu, row, 2 * (i & 15) + 1);
          const uint32_t at = ring + (is_k ? k_place(i, ahead) : v_place(i, n, ahead)), slot = at % kSlots;
          wait(&S.empty[slot], ((at / kSlots) & 1u) ^ 1u);
          if (kTest && at >= p.a.stall) dead = true;
          if (dead) break;
          if (lane == 0) mbar_arrive_expect_tx(&S.full[slot], ((row0 >= 0) + (row1 >= 0)) * 2 * kBoxBytes);
          __syncwarp();
          const int64_t y = h ? row1 : row0;
          if (lane < 4 && y >= 0) {
            uint8_t* dst = S.kv[slot] + half * kHalf + h * kBoxBytes;
            if (p.once) tma_load_2d_hint(dst, tm, half * 64, static_cast<int32_t>(y), &S.full[slot], once);
            else tma_load_2d(dst, tm, half * 64, static_cast<int32_t>(y), &S.full[slot]);
          }
          mine[3] = mine[2];
          mine[2] = mine[1];
          mine[1] = mine[0];
          mine[0] = at + 1;
        }
        ring += 2 * n;
      }
      if (lane == 0) S.last[warp - kKWarp] = make_uint4(mine[0], mine[1], mine[2], mine[3]);
    } else if (warp == kQWarp) {
      // ---- the plan, the pieces, and their queries
      Plan plan;
      const bool uniform = !kSplit && p.uniform;
      if (uniform) {
        plan.entries = p.B;
      } else if (p.plan_global) {
        plan.ent_base = p.ent_base;
        plan.line = p.line;
        plan.entries = kSplit ? p.ent_base[p.B + p.pre] : p.B;
      } else {
        int32_t* line = S.plan + (kSplit ? p.B + p.pre + 1 : 0);
        plan.ent_base = S.plan;
        plan.line = line;
        plan.entries = make_plan<false>(p, S.plan, line, blockIdx.x == 0);
      }
      Walk<kSplit> walk;
      walk.init(p, plan);
      const int half = lane & 1;
      bool more = true;
      int turn = 0;
      while (more && !dead) {
        more = walk.next(p, plan, pc);
        pc.flags |= turn;
        if (kSplit && !is_pair(pc) && !is_dual(pc)) turn ^= (pc.n & 1) * kTurn;
        const uint32_t i = pieces % kQueue;
        wait(&S.pc_empty[i], ((pieces / kQueue) & 1u) ^ 1u);
        if (dead) break;
        if (lane == 0) {
          if (!more) pc.n = -1;
          S.piece[i] = pc;
          mbar_arrive(&S.pc_full[i]);
        }
        ++pieces;
        if (!more || pc.n == 0) continue;
        const int next_head = is_dual(pc), next_row = is_pair(pc) ? kTile : 0;
        const bool both = next_head || next_row;
        const uint32_t b0 = both ? 0 : q_buffer(), nb = both ? 2 : 1;
        for (uint32_t t = 0; t < nb; ++t) {
          const uint32_t b = b0 + t;
          wait(&S.q_empty[b], (uses[b] & 1u) ^ 1u);
          if (dead) break;
          if (lane == 0) mbar_arrive_expect_tx(&S.q_full[b], kTileBytes);
          __syncwarp();
          if (lane < 2)
            tma_load_3d(S.q[b] + half * kHalf, &tm_q, half * 64, (pc.g + static_cast<int>(t) * next_head) << p.gsh,
                        pc.tok0 + ((static_cast<int>(t) * next_row) >> p.gsh), &S.q_full[b]);
          ++uses[b];
        }
      }
      if (uniform && blockIdx.x == 0) check_lens(p, lane, 32);
      if (lane == 0) S.last[2] = make_uint4(uses[0], uses[1], 0, 0);
    } else if (warp == kMmaWarp) {
      // ---- MMA issue.  The whole warp walks and waits, and one elected lane
      // issues: in code that only one lane runs every operand of an MMA is moved
      // to the uniform registers for itself, and the issue falls behind the
      // tensor cores (85-130 cycles per MMA of 64).  One warp issues for both
      // groups: with a warp each, their products interleave and each group's
      // arrive later (909 against 807 us at 8192 causal tokens, 64 heads).
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = mma_idesc(128, 128);
      constexpr uint32_t idesc_o = mma_idesc(128, 128) | (1u << 16);   // B (V) MN-major
      constexpr uint32_t kStep = kTileBytes >> 4;                      // of a descriptor, from slot to slot
      const uint32_t tS = __shfl_sync(0xffffffffu, tmem, 0), tO = tS + 256;
      const uint64_t qd = sw128_desc(smem_u32(S.q[0])), kd = sw128_desc(smem_u32(S.kv[0]));
      const uint64_t vd = sw128_mn_desc(smem_u32(S.kv[0]), kHalf, 1024);
      uint32_t np = 0;   // bit s: phase of the probabilities of group s
      // A wait that ran out ends the loop over the tiles.  The tile's own products
      // may still be computed, on what is there (a test at each of them costs 1.7 %
      // of a prompt's time), but no tile is handed back to its loader any more: one
      // that never came still belongs to the copy in flight.
      // Waits for the next tile of the ring; its slot.
      auto next_tile = [&]() {
        const uint32_t slot = ring % kSlots;
        wait(&S.full[slot], (ring / kSlots) & 1u);
        ++ring;
        return slot;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) mma_commit(bar);
      };
      auto qk = [&](uint32_t s, uint32_t qtile, uint32_t slot) {   // S_s = Q_qtile K^T
        tc_fence_after();
        const uint64_t ad = qd + qtile * kStep, bd = kd + slot * kStep;
        if (leader) {
  #pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
            mma_bf16(tS + kTile * s, ad + off, bd + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          mma_commit(&S.s_full[s]);
        }
      };
      auto pv = [&](uint32_t s, uint32_t slot, bool first) {   // O_s (+)= P_s V
        const uint64_t bd = vd + slot * kStep;
  #pragma unroll
        for (int h = 0; h < 2; ++h) {
          wait(&S.p_full[s][h], (np >> s) & 1u);
          tc_fence_after();
          if (leader) {
  #pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_bf16_ta(tO + kTile * s, tS + kTile * s + 8 * kk, bd + (kk * 2048 >> 4), idesc_o,
                          (kk > 0 || !first) ? 1u : 0u);
          }
        }
        np ^= 1u << s;
      };
      while (take()) {
        const int dual = __shfl_sync(0xffffffffu, is_dual(pc), 0);
        const int n = __shfl_sync(0xffffffffu, pc.n, 0) << dual;
        if (n == 0) continue;
        if (is_pair(pc)) {
          // Tile k's S is issued behind tile k - 1's O of the same group.  The
          // waits for the next tiles' V and K (some 200 cycles each, even when
          // the data is there) stand around group 1's O, where the tensor cores
          // have work meanwhile; six other orders measured 680 to 706 us against
          // 677 (8192 causal tokens, 64 heads).
          uint32_t kslot = next_tile(), vslot = 0;
          wait(&S.q_full[0], uses[0] & 1u);
          wait(&S.q_full[1], uses[1] & 1u);
          ++uses[0];
          ++uses[1];
          for (int k = -1; k < n && !dead; ++k) {
            const bool has_k = k + 1 < n;
            if (k >= 0) pv(0, vslot, k == 0);
            if (has_k) qk(0, 0, kslot);
            else commit(&S.o_full[0]);
            uint32_t vnext = 0, knext = 0;
            if (has_k) vnext = next_tile();
            if (k >= 0) pv(1, vslot, k == 0);
            if (k + 2 < n) knext = next_tile();
            if (has_k) qk(1, 1, kslot);
            else commit(&S.o_full[1]);
            if (dead) break;
            if (k >= 0) commit(&S.empty[vslot]);
            if (has_k) commit(&S.empty[kslot]);
            if (k + 1 == n - 1) {
              commit(&S.q_empty[0]);
              commit(&S.q_empty[1]);
            }
            vslot = vnext;
            kslot = knext;
          }
        } else {
          const uint32_t qb = dual ? 0 : q_buffer(), turn = __shfl_sync(0xffffffffu, first_group<kSplit>(pc), 0);
          wait(&S.q_full[qb], uses[qb] & 1u);
          ++uses[qb];
          if (dual) {
            wait(&S.q_full[1], uses[1] & 1u);
            ++uses[1];
          }
          for (int k = -2; k < n && !dead; ++k) {
            const uint32_t s = (k + turn) & 1;   // tile k + 2 is of the same group
            if (k >= 0) {
              const uint32_t slot = next_tile();
              pv(s, slot, k < 2);
              if (dead) break;
              commit(&S.empty[slot]);
              if (k >= n - 2) commit(&S.o_full[s]);
            }
            if (k + 2 < n) {
              const uint32_t slot = next_tile();
              const uint32_t qs = dual ? s : qb;
              if (dead) break;
              qk(s, qs, slot);
              commit(&S.empty[slot]);
              if (k + 2 >= n - 1 - dual) commit(&S.q_empty[qs]);   // its last use
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---- softmax and output: group s = warp / 4, row r of its tile
    const int s = warp >> 2, r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + kTile * s + lane_base, to = tmem + 256 + kTile * s + lane_base;
    uint32_t ns = 0, no = 0;   // accumulators S_s, O_s taken
    uint32_t nx = 0;           // items joined
    bool lent = false;         // group 1: group 0 may still be reading O_1 and x_ml
    while (take()) {
      const bool pair = is_pair(pc);
      const int dual = is_dual(pc), n = pc.n << dual, turn = first_group<kSplit>(pc);
      const uint32_t ring0 = ring;
      ring += 2 * n;
      const int row = pair ? kTile * s + r : r;        // of the item
      const bool warp_rows = (warp & 3) * 32 < pc.rows - (pair ? kTile * s : 0);   // the warp has a row
      const int pos = pc.p0 + (row >> p.gsh);
      // first token of the row's window, and of the last row's
      const int row_first = clampi(static_cast<int64_t>(pos) - p.a.local + 1, 0, INT_MAX);
      const int last_first = clampi(static_cast<int64_t>(pc.p1) - p.a.local + 1, 0, INT_MAX);
      float m = -INFINITY, l = 0.0f;
      int done = 0;
      if (lent) {   // the next product overwrites O_1, the next hand-over x_ml
        wait(&S.x_empty, (nx - 1) & 1u);
        lent = false;
      }
      for (int k = 0; k < n && !dead; ++k) {
        if (!pair && ((k + turn) & 1) != s) continue;
        bool prefix;
        const int tile = tile_of<kSplit>(pc, k >> dual, pc.n);
        const int t0 = box_token(pc, tile, 0, &prefix), t1 = box_token(pc, tile, 1, &prefix);
        // Tokens [0, sink) and [first, end) are attended to: by some row, by every
        // row, by this row.
        const int n_prefix = static_cast<int>(p.a.n_prefix), sink = prefix ? 0 : p.a.sink;
        const int any_first = prefix ? 0 : pc.lo, any_end = prefix ? n_prefix : pc.hi + 1;
        const int all_first = prefix ? 0 : last_first, all_end = prefix ? n_prefix : pc.p0 + 1;
        auto inside = [&](int t, int first, int end) { return t + kBox <= end && (t >= first || t + kBox <= sink); };
        const bool clean = !inside(t0, any_first, any_end) || !inside(t1, any_first, any_end);
        const bool all = inside(t0, all_first, all_end) && inside(t1, all_first, all_end);
        uint32_t keep[4] = {0, 0, 0, 0};   // bits: this row attends to the token
        if (!all) {
          const int first = prefix ? 0 : row_first, end = prefix ? n_prefix : pos + 1;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int t = (w < 2 ? t0 : t1) + 32 * (w & 1);   // the word's first token
            keep[w] = below(end - t) & (~below(first - t) | below(sink - t));
          }
        }
        // Rows of V that nobody attends to are zeroed, by each group before
        // its own product reads them.  (Called behind the wait for S: by then
        // the slot's tile before V is long loaded, and the phase of that load
        // is not mistaken for this one's.)
        auto clean_v = [&]() {
          const uint32_t at = ring0 + v_place(k, n, pair ? 1 : 2), slot = at % kSlots;
          wait(&S.full[slot], (at / kSlots) & 1u);
          if (dead) return;
          // Eight lanes to a row of a half: a store of 512 contiguous bytes (a row
          // to a lane would meet in the same banks 32 times over).
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int v_row = (warp & 3) * 32 + 4 * i + (lane >> 3);
            if (!any_row_sees(p, pc, prefix, (v_row < kBox ? t0 : t1 - kBox) + v_row)) {
              uint4* v0 = reinterpret_cast<uint4*>(S.kv[slot] + v_row * 128) + (lane & 7);
              v0[0] = v0[kHalf / 16] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_async_smem();
        };
        wait(&S.s_full[s], ns & 1u);
        if (dead) break;
        ++ns;
        tc_fence_after();
        if (warp_rows) {
          float z[128];
          KV_TMEM_LD32(ts, z);
          KV_TMEM_LD32(ts + 32, z + 32);
          KV_TMEM_LD32(ts + 64, z + 64);
          KV_TMEM_LD32(ts + 96, z + 96);
          KV_TMEM_WAIT32(z);
          KV_TIE32(z + 32);
          KV_TIE32(z + 64);
          KV_TIE32(z + 96);
          if (!all) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((keep[w] >> c) & 1u)) z[32 * w + c] = -INFINITY;
            }
          }
          float a[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = fmaxf(z[i], z[8 + i]);
#pragma unroll
          for (int c = 16; c < 128; c += 16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = fmaxf(fmaxf(a[i], z[c + i]), z[c + 8 + i]);
          }
          const float mx = fmaxf(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])), fmaxf(fmaxf(a[4], a[5]), fmaxf(a[6], a[7])));
          if (done == 0) {
            m = mx;
          } else {
            const float mn = fmaxf(m, mx);
            const bool grow = (mn - m) * kScale > kRebase;   // also from -inf
            if (__any_sync(0xffffffffu, grow)) {
              const float al = grow ? ex2_approx((m - mn) * kScale) : 1.0f;
              l *= al;
              if (grow) m = mn;
              // S_s complete means that the product before it (O_s) is, too
#pragma unroll 1
              for (int c = 0; c < 128; c += 16) {
                float o[16];
                tmem_ld_cols<16>(to + c, o);
                tmem_wait_ld();
                KV_TIE16(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= al;
                KV_TMEM_ST16(to + c, o);
              }
            }
          }
          const float mc = m == -INFINITY ? 0.0f : m * kScale;
          float2 acc[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t u[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 x = __ffma2_rn(make_float2(z[64 * q + 2 * i], z[64 * q + 2 * i + 1]),
                                          make_float2(kScale, kScale), make_float2(-mc, -mc));
              const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
              acc[i & 1] = __fadd2_rn(acc[i & 1], e);
              u[i] = pack_bf16(e.x, e.y);
            }
            KV_TMEM_ST32(ts + 32 * q, u);
            if (q == 0 && clean) clean_v();
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full[s][q]);
          }
          l += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        } else {
          if (clean) clean_v();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&S.p_full[s][0]);
            mbar_arrive(&S.p_full[s][1]);
          }
        }
        ++done;
      }
      if (dead) break;
      if (done > 0) {
        wait(&S.o_full[s], no & 1u);
        if (dead) break;
        ++no;
        tc_fence_after();
      }
      // The statistics in log2 units.  Of a whole parity item group 0 joins both
      // groups' (every thread has the same row in both) and writes the output;
      // of a share each group leaves its own, since the groups would wait for
      // each other (128 sequences over a 4K prefix: 56 us joined, 49 so).
      const bool whole = !kSplit || (pc.flags & kWhole), join_groups = kMode == kModeWhole && !pair;
      float a0 = 1.0f, a1 = 0.0f;
      m *= kScale;
      if (join_groups) {
        if (s == 1) {
          S.x_ml[r] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.x_full);
          ++nx;
          lent = true;
          continue;
        }
        wait(&S.x_full, nx & 1u);
        if (dead) break;
        ++nx;
        tc_fence_after();
        const float2 v = S.x_ml[r];
        const float mt = fmaxf(m, v.x);
        a0 = l != 0.0f ? ex2_approx(m - mt) : 0.0f;
        a1 = v.y != 0.0f ? ex2_approx(v.x - mt) : 0.0f;
        m = mt;
        l = l * a0 + v.y * a1;
      }
      if (warp_rows) {
        const bool active = row < pc.rows;                // the row exists
        const int64_t part = pc.part + (pair ? 0 : (s << dual) * pc.rows);
        const int g = pc.g + (s & dual);
        const int64_t orow =
            (static_cast<int64_t>(pc.tok0) + (row >> p.gsh)) * p.Hq + (g << p.gsh) + (row & ((1 << p.gsh) - 1));
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        auto store_out = [&](const float* o, int c) {   // 32 columns from c on
          uint4* dst = reinterpret_cast<uint4*>(p.a.out + orow * kD + c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
        };
        if (join_groups) {
          const float b0 = done > 0 ? a0 * inv : 0.0f, b1 = a1 * inv;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            float o[32], y[32];
            KV_TMEM_LD32(to + c, o);   // holds anything where the group had no tile
            KV_TMEM_LD32(to + kTile + c, y);
            KV_TMEM_WAIT32(o);
            KV_TIE32(y);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = (done > 0 ? o[i] * b0 : 0.0f) + (n > 1 ? y[i] * b1 : 0.0f);
            if (active) store_out(o, c);
            __syncwarp();
          }
        } else {
          float o[128];
          if (done > 0) {
            KV_TMEM_LD32(to, o);
            KV_TMEM_LD32(to + 32, o + 32);
            KV_TMEM_LD32(to + 64, o + 64);
            KV_TMEM_LD32(to + 96, o + 96);
            KV_TMEM_WAIT32(o);
            KV_TIE32(o + 32);
            KV_TIE32(o + 64);
            KV_TIE32(o + 96);
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i) o[i] = 0.0f;
          }
          if (active && whole) {
#pragma unroll
            for (int i = 0; i < 128; ++i) o[i] *= inv;
#pragma unroll
            for (int c = 0; c < 128; c += 32) store_out(o + c, c);
          } else if (active && l != 0.0f) {
            // pc.rows rows, chunk-major: 32 lanes store 512 contiguous bytes
            float4* dst = p.part_o + part * kChunks + row;
#pragma unroll
            for (int i = 0; i < 32; ++i) dst[i * pc.rows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
          __syncwarp();
        }
        if (active) {
          if (!whole) {
            p.part_ml[part + row] = make_float2(m, l);
            if (dual) p.part_ml[part + pc.rows + row] = make_float2(-INFINITY, 0.0f);   // the other group's, of this head
          }
          if (whole && p.a.lse) p.a.lse[orow] = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
        tc_fence_before();
      }
      if (join_groups) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.x_empty);
      }
    }
  }
  if (dead) S.failed = 1;
  tc_fence_before();
  __syncthreads();
  pdl_trigger();   // (at the CTA's start: 93 against 88 us for one 128K sequence, decoding)
  if (S.failed) finish_issued(S, warp);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The plan of a batch too large for the attention's shared memory, one block.
__global__ void __launch_bounds__(1024) kv_plan_kernel(const Args p) {
  __shared__ int32_t ent_base[kMaxSeq + 1], line[kMaxEnt + 1];
  pdl_wait();
  make_plan<true>(p, ent_base, line, true);
  pdl_trigger();
}

// Joins the partial rows of the items that more than one share (or group)
// computed: exact log-sum-exp, fp32.  A thread owns one 16-byte chunk of a
// query row in every share; PG thread groups of a block take every PG-th share
// (many shares of few rows).  Rows are counted as (token, head of the group),
// packed over the batch: an entry covers the rows [key, key + rows).
constexpr int kMergeThreads = 256;
constexpr size_t merge_smem(int entries) { return static_cast<size_t>(entries) * 12 + 4; }

// One share's (max, sum, output chunk) into the running ones.  A sum of 0 is a
// share without any token (its output chunk is not written); NaN passes.
__device__ __forceinline__ void join(float& m, float& l, float4& o, const float2 v, const float4 y) {
  if (v.y != 0.0f) {
    const float mn = fmaxf(m, v.x);
    const float a = ex2_approx(m - mn), b = ex2_approx(v.x - mn);
    m = mn;
    l = l * a + v.y * b;
    o = make_float4(o.x * a + y.x * b, o.y * a + y.y * b, o.z * a + y.z * b, o.w * a + y.w * b);
  }
}

template <int PG>
__global__ void __launch_bounds__(kMergeThreads) kv_merge_kernel(const Args p, int grid) {
  constexpr int kPer = kMergeThreads / PG;          // (row, chunk) elements of a unit
  constexpr int kRowsU = kPer / kChunks;
  extern __shared__ int32_t msm[];
  __shared__ float2 ml[PG][kPer];
  __shared__ float4 ov[PG][kPer];
  const int pg = threadIdx.x / kPer, x = threadIdx.x - pg * kPer;
  pdl_wait();
  const int entries = __ldcg(p.ent_base + p.B + p.pre);
  const int pre_n = p.pre ? __ldcg(p.ent_base + 1) : 0;   // entries of the prefix stand first
  int32_t* line = msm;                                    // [entries + 1]
  int32_t* key = line + p.max_ent + 1;                    // [entries]
  int32_t* rows_of = key + p.max_ent;                     // [entries]
  for (int e = threadIdx.x; e <= p.max_ent; e += kMergeThreads) {   // those behind `entries` hold anything
    line[e] = __ldcg(p.line + e);
    if (e < p.max_ent) {
      const int4 info = __ldcg(p.info + e);
      key[e] = (info.x << p.gsh) + info.y;
      rows_of[e] = info.z;
    }
  }
  __syncthreads();
  if (entries == 0) return;
  const Ranges ranges(line[entries], grid);
  const int64_t R = p.a.bt.T << p.gsh;
  const int64_t units = (R + kRowsU - 1) / kRowsU * p.Hkv;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int g = static_cast<int>(u % p.Hkv);
    const int64_t row = u / p.Hkv * kRowsU + x % kRowsU;   // neighbours in a share
    const int chunk = x / kRowsU;
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bool write = false;
    for (int f = p.pre ? 0 : 1; f < 2; ++f) {
      // f = 0: the prefix's item that holds this row, f = 1: its own sequence's
      const int e0 = f == 0 ? 0 : pre_n, e1 = f == 0 ? pre_n : entries;
      if (e0 >= e1 || row >= R) continue;
      const int e = e0 + find_last(key + e0, e1 - e0, static_cast<int>(row));
      const int rr = static_cast<int>(row) - key[e], rows = rows_of[e];
      if (rr < 0 || rr >= rows) continue;    // a token of no sequence
      const int span = (line[e + 1] - line[e]) / p.Hkv;
      const int x0 = line[e] + g * span;
      const int c0 = ranges.cta(x0 + first_place(span)), c1 = ranges.cta(x0 + last_place(span, tile_weight(rows)));
      const bool pair = rows > kTile;
      if (pair && c0 == c1 && !p.pre) continue;   // its share has written the output
      write |= f == 1;
      const int count = pair ? c1 - c0 + 1 : 2 * (c1 - c0 + 1);
      const int64_t base = 2 * ((f == 1 && p.pre ? R * p.Hkv : 0) + static_cast<int64_t>(key[e]) * p.Hkv +
                                static_cast<int64_t>(g) * rows);
      auto share = [&](int i) {
        return base + static_cast<int64_t>(c0 + (pair ? i : i >> 1)) * p.slot_rows + (pair ? 0 : (i & 1) * rows);
      };
      int i = pg;
      for (; i + 3 * PG < count; i += 4 * PG) {
        float2 v[4];
        float4 y[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int64_t part0 = share(i + w * PG);
          v[w] = __ldcg(p.part_ml + part0 + rr);
          y[w] = __ldcg(p.part_o + part0 * kChunks + static_cast<int64_t>(chunk) * rows + rr);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) join(m, l, o, v[w], y[w]);
      }
      for (; i < count; i += PG) {
        const int64_t part0 = share(i);
        const float2 v = __ldcg(p.part_ml + part0 + rr);
        join(m, l, o, v, __ldcg(p.part_o + part0 * kChunks + static_cast<int64_t>(chunk) * rows + rr));
      }
    }
    if (PG > 1) {
      ml[pg][x] = make_float2(m, l);
      ov[pg][x] = o;
      __syncthreads();
      if (pg == 0) {
#pragma unroll
        for (int w = 1; w < PG; ++w) join(m, l, o, ml[w][x], ov[w][x]);
      }
      __syncthreads();
    }
    if (write && pg == 0) {
      const int64_t orow = (row >> p.gsh) * p.Hq + (g << p.gsh) + (row & ((1 << p.gsh) - 1));
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      *reinterpret_cast<uint2*>(p.a.out + orow * kD + 4 * chunk) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
      if (p.a.lse && chunk == 0) p.a.lse[orow] = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  }
  pdl_trigger();
}

// Whether a batch of T tokens may be split, which bounds its workspace and its
// plan: fewer items than 4 per SM, or with a shared prefix short sequences.
// Counted with full tiles only (T Gq / 256 per KV head), which every batch has
// at least.  A split plan has at most T Gq / 256 + B entries (T Gq / 256 + 1
// more for a shared prefix), and with
//   T Gq / 256 Hkv < 4 SMs, or Gq T < 128 B with a shared prefix,
// these are below 2 (1024 + 1) + 2048, of kMaxEnt, on a device of up to 256 SMs.
bool may_split(int64_t T, int B, int Hq, int Hkv, bool prefix, int num_sms) {
  const int64_t gq = Hq / Hkv;
  const int64_t items = (T * gq + kItemRows - 1) / kItemRows * Hkv;
  if (prefix && T * gq < static_cast<int64_t>(kTile) * B) return true;
  return items < 4 * static_cast<int64_t>(num_sms);
}

// Key tiles that any item of `rows` query rows of a window call can have.
int64_t most_tiles(const KvAttnArgs& a, int64_t n_cap, int gq, int rows) {
  const int64_t tokens = a.bt.cu_q ? std::min<int64_t>(a.bt.T, rows / gq) : 1;
  const int64_t span = std::min<int64_t>(n_cap, static_cast<int64_t>(a.local) + tokens - 1);   // of the window
  const int64_t boxes = (span + 2 * kBox - 2) / kBox + (std::min<int64_t>(a.sink, n_cap) + kBox - 1) / kBox;
  return (boxes + 1) / 2;
}

// The schedule of a call, `may` it be split, by the time each would take
// (microseconds, fitted to all three at 1 to 128 sequences of 1 to 2048 new
// tokens, windows of 256 to 16384 tokens and prefixes of 128 to 8000).  Whole
// items take rounds over the SMs: of 256 rows (a tile 1.32 us), or of 128 (0.7
// us, 0.8 on all SMs, 1.1 when each of them reads keys of its own) one by one or
// in twos, which saves a start (152 sequences, 8 KV heads: a window of 32 tokens
// 29.3 us in twos, 41.9 joined, of 500 62 and 67); they walk the prefix too.  A split takes equal shares and the merge, and more for the
// partial rows of 256-row items, the prefix's among them.  The host knows only
// n_cap of the lengths; single tokens' are taken to be 0.7 of it on average,
// since equal shares gain where they differ.  32 heads, 8 KV heads, split and
// whole items of 128 rows: one token, a window of 256 11.5 and 10.5 us, of 4096
// 14.4 and 32; 8 sequences of 64 tokens 30.2 and 13.4, 53 and 36.7; 2048 new
// tokens behind a prefix of 1000 149 and 69, with 256 rows 56; 32 tokens of 32
// sequences behind one of 4000 24 and 59.
struct Schedule {
  bool split;
  int item_rows;
  int dual;
};
Schedule attn_schedule(const KvAttnArgs& a, int B, int gq, int Hkv, int64_t n_cap, int num_sms, bool may) {
  const int64_t rows = a.bt.T * gq;   // of all sequences, for one KV head
  auto items_of = [&](int64_t per) { return static_cast<int64_t>(Hkv) * B * ((rows + per * B - 1) / (per * B)); };
  auto rounds = [&](int64_t items) { return static_cast<double>((items + num_sms - 1) / num_sms); };
  const double prefix = static_cast<double>((a.n_prefix + kTile - 1) / kTile);
  const double tiles = static_cast<double>(most_tiles(a, n_cap, gq, kItemRows));
  const double mean = std::min(tiles, 1.0 + 0.7 * static_cast<double>(n_cap) / kTile);
  const int64_t items = items_of(kItemRows), halves = items_of(kTile);
  const double per_sm = static_cast<double>(items) / num_sms;
  const double pre_per_sm = static_cast<double>((rows + kItemRows - 1) / kItemRows * Hkv) / num_sms;
  const double busy = 0.7 + 0.1 * std::min(1.0, static_cast<double>(halves) / num_sms);
  const double reading = std::min(1.0, static_cast<double>(Hkv) * B / num_sms);
  const bool pair = rows > static_cast<int64_t>(kTile) * B;
  const double full = std::min(1.0, static_cast<double>(rows) / (static_cast<double>(kTile) * B));   // of an item's rows
  const double whole256 = pair ? 7.0 + rounds(items) * (1.32 * (tiles + prefix) + 4.8) : 1e30;
  const double walk = (busy + 0.32 * reading * reading) * tiles + busy * prefix;   // of an item's tiles
  const double joined = rounds(halves) * (walk + 3.3);
  const double dual = Hkv % 2 ? 1e30 : rounds((halves + 1) / 2) * (2.0 * walk + 3.3 + 2.0 * full);
  const double whole128 = 5.0 + std::min(joined, dual);
  const double split = (may ? 0.0 : 1e30) + (a.n_prefix ? pre_per_sm * (2.0 * prefix + 20.0) : 0.0) +
                       (pair ? 20.0 + per_sm * (1.7 * tiles + 20.0) : 13.0 + per_sm * (1.2 * mean + 4.5));
  if (split < whole256 && split < whole128) return {true, kItemRows, 0};
  if (whole256 <= whole128) return {false, kItemRows, 0};
  return {false, kTile, dual < joined ? 1 : 0};
}

struct Layout {
  size_t off_o = 0, off_ml = 0, off_base = 0, off_line = 0, off_info = 0, total = 0;
  int slot_rows = 0;
};

Layout layout_of(int64_t T, int Hq, int Hkv, bool prefix, bool split, int num_sms) {
  Layout L;
  const int64_t most = 2 * T * (Hq / Hkv);
  L.slot_rows = static_cast<int>(most < kItemRows ? most : kItemRows);
  const int64_t rows = split ? 2 * T * Hq * (prefix ? 2 : 1) + static_cast<int64_t>(num_sms) * L.slot_rows : 0;
  L.off_base = 0;
  L.off_line = align_up(L.off_base + (kMaxSeq + 1) * sizeof(int32_t), 256);
  L.off_info = align_up(L.off_line + (kMaxEnt + 1) * sizeof(int32_t), 256);
  L.off_ml = align_up(L.off_info + kMaxEnt * sizeof(int4), 256);
  L.off_o = align_up(L.off_ml + static_cast<size_t>(rows) * sizeof(float2), 256);
  L.total = align_up(L.off_o + static_cast<size_t>(rows) * kChunks * sizeof(float4), 256);
  return L;
}

int encode_q(CUtensorMap* m, const uint16_t* q, int64_t T, int Hq, int gq, EncodeTiledFn enc) {
  const uint64_t gdim[3] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(Hq), static_cast<uint64_t>(T)};
  const uint64_t gstride[2] = {kD * 2, static_cast<uint64_t>(Hq) * kD * 2};
  const unsigned box[3] = {64, static_cast<unsigned>(gq), static_cast<unsigned>(kTile / gq)};
  const unsigned estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(q), gdim, gstride, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

int encode_rows(CUtensorMap* m, const uint16_t* base, int64_t rows, EncodeTiledFn enc) {
  const uint64_t gdim[2] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(rows)};
  const uint64_t gstride[1] = {kD * 2};
  const unsigned box[2] = {64, kBox};
  const unsigned estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(base), gdim, gstride, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

using AttnKernel = void (*)(Args, CUtensorMap, CUtensorMap, CUtensorMap);
AttnKernel kernel_of(Mode mode, bool test) {
  switch (mode) {
    case kModeSplit: return test ? kv_attn_kernel<kModeSplit, true> : kv_attn_kernel<kModeSplit>;
    case kModeWhole: return test ? kv_attn_kernel<kModeWhole, true> : kv_attn_kernel<kModeWhole>;
    default: return test ? kv_attn_kernel<kModeTwos, true> : kv_attn_kernel<kModeTwos>;
  }
}

}  // namespace

// Enough for every batch of at most T tokens (and B sequences): the most tokens
// that may be split take the most, more tokens no partial rows.  For the most
// SMs: a device with fewer splits a subset of these batches.
size_t kv_attn_workspace_bytes(int64_t T, int B, int Hq, int Hkv, bool prefix, int num_sms) {
  const int64_t gq = Hq / Hkv;
  int64_t most = (4 * static_cast<int64_t>(num_sms) - 1) / Hkv * kItemRows / gq;   // the bounds of may_split
  if (prefix) most = std::max(most, (static_cast<int64_t>(kTile) * B - 1) / gq);
  return layout_of(std::min(T, most), Hq, Hkv, prefix, true, num_sms).total;
}

size_t kv_attn_whole_bytes() { return layout_of(0, 1, 1, false, false, 0).total; }

cudaError_t configure_kv_attn_kernels(const DeviceInfo&) {
  cudaError_t e;
  for (const bool test : {false, true})
    for (const Mode mode : {kModeSplit, kModeWhole, kModeTwos})
      if ((e = cudaFuncSetAttribute(kernel_of(mode, test), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(sizeof(Smem)))) != cudaSuccess)
        return e;
  const int merge = static_cast<int>(merge_smem(kMaxEnt));
  if ((e = cudaFuncSetAttribute(kv_merge_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, merge)) != cudaSuccess)
    return e;
  if ((e = cudaFuncSetAttribute(kv_merge_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, merge)) != cudaSuccess)
    return e;
  return cudaFuncSetAttribute(kv_merge_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, merge);
}

int launch_kv_attn(const qasc_shape& s, const KvAttnArgs& a, uint8_t* ws, size_t* ws_bytes, const DeviceInfo& dev,
                   cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return cudaErrorNotSupported;
  const int gq = s.Hq / s.Hkv;
  alignas(64) CUtensorMap tq, tk, tv;
  if (encode_q(&tq, a.q, a.bt.T, s.Hq, gq, enc) != 0 || encode_rows(&tk, a.K, a.cache_rows, enc) != 0 ||
      encode_rows(&tv, a.V, a.cache_rows, enc) != 0)
    return cudaErrorInvalidValue;
  Args p;
  p.a = a;
  p.B = s.B;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.gsh = gq == 8 ? 3 : (gq == 4 ? 2 : (gq == 2 ? 1 : 0));
  p.n_cap = s.n_cap;
  const bool prefix = a.n_prefix > 0;
  const Schedule plan = attn_schedule(a, a.seqs > 0 ? a.seqs : s.B, gq, s.Hkv, s.n_cap, dev.num_sms,
                                      may_split(a.bt.T, s.B, s.Hq, s.Hkv, prefix, dev.num_sms));
  p.split = plan.split;
  p.item_rows = plan.item_rows;
  p.dual = plan.dual;
  p.pre = p.split && prefix;
  p.once = a.bt.T * gq <= static_cast<int64_t>(kItemRows) * s.B && p.pre == prefix;
  const Layout L = layout_of(a.bt.T, s.Hq, s.Hkv, prefix, p.split, dev.num_sms);
  if (*ws_bytes < L.total) {
    *ws_bytes = L.total;
    return kSmallWorkspace;
  }
  p.slot_rows = L.slot_rows;
  p.part_o = reinterpret_cast<float4*>(ws + L.off_o);
  p.part_ml = reinterpret_cast<float2*>(ws + L.off_ml);
  p.ent_base = reinterpret_cast<int32_t*>(ws + L.off_base);
  p.line = reinterpret_cast<int32_t*>(ws + L.off_line);
  p.info = reinterpret_cast<int4*>(ws + L.off_info);
  p.err = dev.err_word;
  // Words of the plan: the most items per KV head that T tokens of B sequences can make.
  const int64_t items = (a.bt.T * gq + kItemRows - 1) / kItemRows;
  const int64_t entries = items + s.B + (p.pre ? items : 0);
  p.max_ent = static_cast<int>(entries < kMaxEnt ? entries : kMaxEnt);
  const int64_t words = p.split ? (s.B + p.pre + 1) + (p.max_ent + 1) : s.B + 1;
  p.uniform = !p.split && !a.bt.cu_q;
  p.plan_global = !p.uniform && words > kPlanWords;
  cudaError_t e;
  if (p.plan_global) {
    e = launch_dependent(kv_plan_kernel, dim3(1), dim3(1024), 0, stream, 1, p);
    if (e != cudaSuccess) return e;
  }
  const auto attn = kernel_of(p.split ? kModeSplit : (p.dual ? kModeTwos : kModeWhole), a.stall >= 0);
  e = launch_dependent(attn, dim3(dev.num_sms), dim3(kThreads), sizeof(Smem), stream, 1, p, tq, tk, tv);
  if (e != cudaSuccess || !p.split) return e;
  // Few rows: several thread groups to an element (one 128K sequence 86.3 us,
  // 32 over a 32K prefix 42.7; with one group from 1024 rows on 43.8, with four
  // up to 4096 rows 64 sequences with a 4K window 159 against 157).
  const int64_t out_rows = a.bt.T * s.Hq;
  const int pg = out_rows <= 512 ? 4 : (out_rows <= 2048 ? 2 : 1), per_unit = kMergeThreads / pg / kChunks;
  const int64_t units = (a.bt.T * gq + per_unit - 1) / per_unit * s.Hkv, most = static_cast<int64_t>(dev.num_sms) * 8;
  const auto merge = pg == 4 ? kv_merge_kernel<4> : (pg == 2 ? kv_merge_kernel<2> : kv_merge_kernel<1>);
  return launch_dependent(merge, dim3(static_cast<unsigned>(units < most ? units : most)),
                          dim3(kMergeThreads), merge_smem(p.max_ent), stream, 1, p, dev.num_sms);
}

}  // namespace qasc
