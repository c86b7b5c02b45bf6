// kv4_window_attn and kv4_sparse_attn: attention over a 4-bit cache (kv4.cuh).
//
//   out[t,h,:] = sum_{j in A(t)} softmax_j(q[t,h].K_j / sqrt(d)) V_j
// with A(t) the sink and the newest `local` tokens up to t's own position, or
// (listed) the sink, the listed and the local tokens of a decode step.
//
// What bounds it.  144 bytes of a token and KV head are read for 512 operations
// per query head: bytes, as long as the codes become operands fast enough.  At
// HBM's rate an SM gets some 22 bytes a cycle, 45 values, which as bf16 take 90
// bytes a cycle to write to shared memory and 90 for tensor cores to read again, of
// 128 that there are: so codes go from shared memory to registers, become fp16
// there, and are the register operand of the product (mma.sync, 16 x 8 x 16); a
// tcgen05 product takes its second operand from shared memory only, and 128 rows
// where there are 1 to 16.  The products take a fourth of mma.sync's rate.  One
// sequence of 32768 tokens, 16 rows: 21 us; over a bf16 copy on tcgen05, which is
// where calls of many rows go (see copy_pays), 70.  (For 17 to 128 rows the reckoning is
// another: 180 of 128 bytes a cycle are 1.4 times HBM's time, less than the passes of 16 rows take here.)
//
// Work.  The queries of a KV head's group share its keys: an item is up to
// 8 kNT rows (token, head of the group) of a sequence and KV head.  Its tokens
// are numbered in tiles of 32: the sink's, then those of the window, each of which
// stands in one page, or a list's without gaps.  The tiles of
// all items are laid end to end, every block takes an equal range of that line and
// every warp of it an equal part of the range: a warp walks its tiles alone, has
// the next two on their way (three with 16 columns), and writes the rows of items
// that are all its own.
// Of an item that it shares it keeps (max, sum, O); the block joins its warps' at
// its end, once, and those that go beyond it are left in the workspace, two places a block
// (the item that it begins with, the one that it ends with), where
// kv4_merge_kernel joins them.  (With the tiles of every item dealt to all warps and
// joined in the block, a third of the instructions were the joins': 64 sequences
// with a 4K window 91 us, 73 so.)  Short items are not shared between blocks: each
// block has items of its own, and there is no merge to wait for (4 sequences, sink and
// 256 tokens: 7.0 us, 11 with them on the line).
// Keys stand as rows of the first product and channels as rows of the second,
// queries as columns of both:
//   S^T = K Q^T      (16 tokens x 8 queries, over d)
//   P = exp2(S c - m) in fp16
//   O^T += V^T P^T   (16 channels x 8 queries, over tokens)
// Which value a lane holds of the dimension that a product sums over is free as
// long as both operands agree: of K a lane takes 16 bytes of a row, 32 values in
// a line, of V a group of 16 channels of four tokens, so that it needs one scale
// for each.  P turns from the first product's layout to the second's by
// movmatrix.
//
// Numbers.  scale * code is exact in fp16 (kv4.cuh).  A query row is scaled by a
// power of two to a largest value of 2^14 to 2^15 and is exact in fp16 but for
// values 2^-28 below that one.  Products, statistics and sums are fp32.  P is
// rounded to fp16 (2^-11 of each weight, an eighth of the bf16 output's own
// rounding); its base is 2^-10 of the row's maximum when it was taken, and moves
// when the maximum grows by more than 2^5: P stays below 2^15, and weights down
// to 2^-24 of the largest keep all their bits.  The sum that divides takes P
// unrounded.
//
// Measured among others of its kind.  64 sequences, 4K window, 8 KV heads (280 MB): 58
// us, 4.8 TB/s (70 % of a copy's rate): 4.3 us until the first tile is there (lengths,
// places, pages, rows: four loads one behind the other), then 231 cycles a tile and SM, of
// which HBM's rate allows 201 and the instructions 150, and 3 us of join and merge.  One
// sequence of 131072 tokens, 64 heads (151 MB): 36.5 us.  Four 128K contexts at 20 %, a
// list a KV head: 38 us; of scattered rows HBM reads 64 bytes for 8 of scales, 134 MB for
// 95, at 6.1 TB/s once the first rows are there (7 us).  ncu, the first case: 279.7 MB
// read, hmma pipe 22 %, ALU pipe 44 %, issue 53 %.  What did not pay: 16 warps of
// two stages (spills), the first product of a tile beside the second of the one before
// (65.9 against 65.7), one loop over items and tiles (66.8 against 62.1), the first tiles' pages
// asked for together (59.7 against 58.5), L2's default fetch of 128 bytes for lists (48 against 40).
#include <algorithm>
#include <climits>

#include "internal.h"
#include "kv4.cuh"

namespace qasc {
namespace {

constexpr int kTile = 32;                      // tokens of a warp's tile
// Of a block, by its items' column tiles: as many warps as the registers allow
// (166 and 243 of a thread).  64 sequences with a 4K window: 12 warps of three stages 66
// us, 8 of four 69, 16 of two, which spill, 67.
constexpr int warps_of(int nt) { return nt == 1 ? 12 : 8; }
constexpr int stages_of(int nt) { return nt == 1 ? 3 : 4; }   // tiles of a warp's ring
constexpr int kTileCodes = kTile * kKv4Codes;  // bytes
constexpr int kTileScales = kTile * kKv4Groups;
constexpr int kStage = 2 * (kTileCodes + kTileScales);
constexpr int kSums = 512;                     // places are summed for as many groups of sequences at most
constexpr int kQueue = 8;                      // items that a warp's loads are ahead of its products, at most
constexpr int kItemCost = 2;                   // places of an item beside its tiles: queries, output (4: 2 % more)
constexpr int kTokensMost = 1 << 24;           // above n_cap, and sink and local as the kernel has them
constexpr int kTilesMost = kTokensMost / kTile;
// Sequences of more rows than this take their keys and values from a bf16 copy and
// go to kv_window_attn's kernel, whose products are tcgen05's: a row block here costs
// what it costs whether the next one needs the same keys or not.  One sequence of
// 32768 tokens, 32 heads, 8 KV heads, here and over a copy: 64 rows 49 and 71 us,
// 128 rows 86 and 76, 256 rows 161 and 85; 32 sequences of 4096, 64 heads, 136 rows: 348 and 241.
constexpr int64_t kCopyRows = 128;
constexpr int kLeast = 8;                      // places that a block takes at least
// Items of more tokens than this may be shared between blocks; with more items than warps those
// of more than the second.  (256 sequences of one token, 8 KV heads, 1000 tokens each: 84 us as whole
// items, 69 shared; 200: 55 and 57; 400 of 260 tokens: 42 and 45.)
constexpr int kWholeTokens = 1024, kWholeMany = 288;
constexpr float kBase = 10.0f;                 // log2 of P at the maximum that the base was taken from
constexpr float kGrow = 5.0f;                  // growth of the maximum that moves the base
// log2(e) / sqrt(128): logits in base-2 units.
constexpr float kScale = 1.4426950408889634f * 0.08838834764831845f;

// Window calls; what they have beside a copy of all sequences of many rows; listed ones.
enum Kind { kWindow, kRest, kListed };

struct Args {
  Kv4AttnArgs a;
  int B, Hq, Hkv, gsh;      // gsh = log2(Hq / Hkv)
  int seqs;                 // sequences of the line: B, or (listed) the KV heads of all
  int64_t n_cap;
  int n, sink_end, local_start;   // listed: tokens of every sequence, its regions
  const int32_t* copied;    // [B] not 0: a sequence that is left out here (NULL: none of these)
  int64_t copy_tokens;      // kRest: sequences of more than kCopyRows rows that see 1 to as many tokens are left out
  int whole;                // items are not shared between blocks
  int ssh;                  // sequences of a sum: 2^ssh
  int ush;                  // tiles of a place: 2^ush, so that the line has fewer than 2^31 places
  float* part_o;            // [grid][2][rows][128]
  float2* part_ml;          // [grid][2][rows] (max in log2 units, sum)
  struct Share* share;      // [grid] the item that a block shares with those behind it
  unsigned* err;
};

// Rows [first, first + rows) of a KV head's (token, head of the group) rows, and the
// last block that has a part of them; rows 0: none.
struct Share {
  int64_t first;
  int rows, g;
  int last, pad;
};

// A warp's part of an item: tiles t0 .. t0 + n - 1 of `tiles`.
struct alignas(16) Piece {
  int tok0, rows;      // first query token, rows
  int b, g;
  int p0, p1;          // positions of the first and last row
  int lo;              // window: token of the slot behind the sink's, a multiple of 32; listed: list's entries
  int head, cnt;       // slots of the sink, of all
  int t0, n, tiles;
  int m0, m1;          // tiles [m0, m1) are attended to as a whole by every row
  int x0;              // its first place on the line
  int64_t base;        // the sequence's first entry of the block table, or the KV head's first row
};

struct Seq {
  int q0, ql, len;
};

// Where a warp's loads stand: item `rem` of sequence b's `items`.
struct Walk {
  int x0;              // the item's first place
  int b, rem, items, span;
  int start, end;      // the warp's places; whole items: its part of each of them and their parts
  int left;            // whole items: items left, this one among them
  int used;            // this item has been handed out
  Seq s;
};

// Part of an item in shared memory: rows [kRows][128] fp32, their chunks of four
// turned by (row / 2) mod 4 (which the products' layout writes without
// bank conflicts), and their (max, sum).
template <int kRows>
struct Part {
  float4 o[kRows][kD / 4];
  float2 ml[kRows];
};

__device__ __forceinline__ int clampi(int64_t v, int64_t lo, int64_t hi) {
  return static_cast<int>(v < lo ? lo : (v > hi ? hi : v));
}

template <bool kList>
__device__ __forceinline__ Seq seq_of(const Args& p, int b) {
  Seq r;
  if (kList) {   // (the line's sequences are KV heads of sequences here, each with a list)
    r.q0 = b / p.Hkv;
    r.ql = 1;
    r.len = p.n;
    return r;
  }
  const Batch& bt = p.a.bt;
  if (bt.cu_q) {
    r.q0 = clampi(__ldg(bt.cu_q + b), 0, bt.T);
    r.ql = clampi(__ldg(bt.cu_q + b + 1), r.q0, bt.T) - r.q0;
  } else {
    r.q0 = b;
    r.ql = 1;
  }
  r.len = clampi(__ldg(bt.lens + b), 0, p.n_cap);
  return r;
}

__device__ __forceinline__ int list_len(const Args& p, int b, int g) {
  if (p.a.sel_len == nullptr) return p.a.K;
  return clampi(__ldg(p.a.sel_len + (p.a.sel_per_kv ? b * p.Hkv + g : b)), 0, p.a.K);
}

// Items of a sequence (row blocks times KV heads) and the places of each: the
// most tiles that any of them has (whole items: one).
template <int kKind, int kRows>
__device__ __forceinline__ int items_of(const Args& p, const Seq& s, int b) {
  if (kKind == kListed) return 1;
  const int64_t rows = static_cast<int64_t>(s.ql) << p.gsh;
  if (kKind == kWindow && p.copied && __ldcg(p.copied + b)) return 0;
  if (kKind == kRest && rows > kCopyRows) {
    int between;
    const int tokens = kv4_tokens_seen(s.len, s.ql, p.a.sink, p.a.local, &between);
    if (tokens > 0 && tokens <= p.copy_tokens) return 0;
  }
  return static_cast<int>((rows + kRows - 1) / kRows) * p.Hkv;
}
template <bool kList, int kRows>
__device__ __forceinline__ int span_of(const Args& p, const Seq& s, int b) {
  if (p.whole) return 1;
  int tiles;
  if (kList) {
    tiles = (p.sink_end + list_len(p, b / p.Hkv, b % p.Hkv) + (p.n - p.local_start) + kTile - 1) / kTile;
  } else {
    // the sink's tiles, the window's, and one more where it begins inside a tile
    const int window = (p.a.local + min(s.ql, kRows >> p.gsh) - 1 + 2 * (kTile - 1)) / kTile;
    tiles = min((s.len + kTile - 1) / kTile, window + (p.a.sink + kTile - 1) / kTile);
  }
  return ((tiles + (1 << p.ush) - 1) >> p.ush) + kItemCost;
}

// A line of U places over G blocks: block c has the places [c U / G, (c + 1) U / G),
// in 32 bits (64-bit divisions at a block's start cost it 2 us).
struct Line {
  unsigned U, G, q, r, inv;   // inv = ceil(2^32 / G): n inv / 2^32 is n / G for n < 2^16
  __device__ __forceinline__ Line(int places, int grid) {
    U = places;
    G = grid;
    inv = 0xffffffffu / G + 1;
    q = G == 1 ? U : __umulhi(U, inv);   // n / G or one above for any n < 2^31
    if (q * G > U) --q;
    r = U - q * G;
  }
  __device__ __forceinline__ int start(unsigned c) const { return static_cast<int>(c * q + (G == 1 ? 0 : __umulhi(c * r, inv))); }
  // The block that holds place x.
  __device__ __forceinline__ int block(int x) const {
    int c = clampi(static_cast<int>(__fdividef(static_cast<float>(x) * static_cast<float>(G), static_cast<float>(U))), 0, G - 1);
    while (c > 0 && start(c) > x) --c;
    while (c + 1 < static_cast<int>(G) && start(c + 1) <= x) ++c;
    return c;
  }
};

template <int kNT>
struct Smem {
  static constexpr int kRows = 8 * kNT, kWarps = warps_of(kNT), kStages = stages_of(kNT);
  static_assert(2 * kWarps <= 32, "a lane for each part");
  static_assert(kStages * kStage >= sizeof(Part<kRows>), "a warp's last part stands in its ring");
  alignas(16) uint8_t ring[kWarps][kStages * kStage];
  Part<kRows> first[kWarps];
  Piece queue[kWarps][kQueue];
  Walk walk[kWarps];
  Piece part[2 * kWarps];        // of every warp: the item that it shares with earlier ones, with later ones
  int there[2 * kWarps];         // 0: none, 1: the item goes on, 2: it ends here
  int place[kSums + 1];          // places before a group of sequences
};

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// Rows of their own, zeros behind `bytes`.  (64 bytes are fetched into L2, not the default
// 128: of scattered rows the rest would be read for nothing, 215 MB where 95 are listed:
// four 128K contexts at 20 %, 48 against 40 us.)
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8_zfill(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global.L2::64B [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// c (+)= A (16 x 16, rows) B (16 x 8, columns), fp16 operands.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) { return bits(__floats2half2_rn(lo, hi)); }

// Row of the queries and outputs of row `col` of an item.
__device__ __forceinline__ int64_t row_of(const Args& p, int tok0, int g, int col) {
  return static_cast<int64_t>(tok0 + (col >> p.gsh)) * p.Hq + (g << p.gsh) + (col & ((1 << p.gsh) - 1));
}
__device__ __forceinline__ float lse_of(float m, float l) {
  return l != 0.0f ? (m == -INFINITY ? l : (m - kBase + log2f(l)) * 0.6931471805599453f) : -INFINITY;
}
__device__ __forceinline__ float inverse_of(const Args& p, float l) {
  return l != 0.0f ? p.a.kv.v_scale / l : 0.0f;
}

// Row `pos` of a window call attends to token t.
__device__ __forceinline__ bool attends(const Args& p, int pos, int t) {
  return t <= pos && (t < p.a.sink || t > pos - p.a.local);
}

constexpr int kNoToken = INT_MIN;

// Token of slot s of an item; kNoToken: none that any of its rows attends to.  Of a window
// call the slots of the sink end with a tile and the window's begin with a multiple of
// 32 tokens, so that a tile never leaves its page and its rows stand in a line.
template <bool kList>
__device__ __forceinline__ int token_of_slot(const Args& p, const Piece& pc, int s) {
  if (s >= pc.cnt) return kNoToken;
  if (!kList) {
    if (s < pc.head) return s < p.a.sink ? s : kNoToken;
    const int t = pc.lo + s - pc.head;
    return t <= pc.p1 && (t < p.a.sink || t > pc.p0 - p.a.local) ? t : kNoToken;
  }
  if (s < pc.head) return s;
  const int i = s - pc.head;
  if (i >= pc.lo) return p.local_start + i - pc.lo;
  const int64_t list = p.a.sel_per_kv ? static_cast<int64_t>(pc.b) * p.Hkv + pc.g : pc.b;
  return __ldg(p.a.sel + list * p.a.K + i);   // (checked a tile later, where it is used: next_rows)
}

// The item that holds place x, of sequence b or a later one; `at` places stand before b.
// (Offsets of new tokens that do not ascend can make a line of more than 2^32 places: sums
// wrap then, and a place may belong to no item, w.b == p.seqs, but to none outside
// its sequence.)
template <int kKind, int kRows>
__device__ __forceinline__ Walk walk_from(const Args& p, int b, unsigned at, unsigned x) {
  constexpr bool kList = kKind == kListed;
  Walk w;
  w.rem = w.x0 = 0;
  for (w.b = b; w.b < p.seqs; ++w.b) {
    w.s = seq_of<kList>(p, w.b);
    w.items = items_of<kKind, kRows>(p, w.s, w.b);
    if (w.items == 0) continue;
    w.span = span_of<kList, kRows>(p, w.s, w.b);
    const unsigned all = static_cast<unsigned>(w.items) * static_cast<unsigned>(w.span);
    if (x - at < all) {
      w.rem = (x - at) / static_cast<unsigned>(w.span);
      w.x0 = at + w.rem * w.span;
      break;
    }
    at += all;
  }
  return w;
}

// The next item (w.b == p.seqs behind the last).
template <int kKind, int kRows>
__device__ __forceinline__ void walk_on(const Args& p, Walk& w) {
  constexpr bool kList = kKind == kListed;
  w.x0 += w.span;
  if (++w.rem < w.items) return;
  w.rem = 0;
  while (++w.b < p.seqs) {
    w.s = seq_of<kList>(p, w.b);
    w.items = items_of<kKind, kRows>(p, w.s, w.b);
    if (w.items == 0) continue;
    w.span = span_of<kList, kRows>(p, w.s, w.b);
    return;
  }
}

// The warp's part of item w.
template <bool kList, int kRows>
__device__ __forceinline__ Piece piece_of(const Args& p, const Walk& w) {
  Piece pc;
  const unsigned blocks = kList || w.items == p.Hkv ? 1 : static_cast<unsigned>(w.items) / static_cast<unsigned>(p.Hkv);
  pc.b = kList ? w.s.q0 : w.b;
  pc.g = kList ? w.b - w.s.q0 * p.Hkv : (blocks == 1 ? w.rem : static_cast<int>(static_cast<unsigned>(w.rem) / blocks));
  pc.x0 = w.x0;
  const int r0 = kList ? 0 : (w.rem - pc.g * static_cast<int>(blocks)) * kRows;
  pc.rows = static_cast<int>(min(static_cast<int64_t>(kRows), (static_cast<int64_t>(w.s.ql) << p.gsh) - r0));
  pc.tok0 = w.s.q0 + (r0 >> p.gsh);
  pc.p0 = w.s.len - w.s.ql + (r0 >> p.gsh);
  pc.p1 = w.s.len - w.s.ql + ((r0 + pc.rows - 1) >> p.gsh);
  pc.p0 = max(pc.p0, -kTokensMost);   // in front of the cache all the same
  if (kList) {
    pc.head = p.sink_end;
    pc.lo = list_len(p, pc.b, pc.g);
    pc.cnt = p.sink_end + pc.lo + (p.n - p.local_start);
  } else {
    pc.lo = max(pc.p0 - p.a.local + 1, 0) & ~(kTile - 1);
    pc.head = p.a.sink < pc.lo ? (p.a.sink + kTile - 1) & ~(kTile - 1) : pc.lo;
    if (pc.head >= pc.lo) pc.head = pc.lo = 0;   // the sink's tiles reach the window's
    pc.cnt = pc.p1 >= 0 ? pc.head + pc.p1 - pc.lo + 1 : 0;
  }
  pc.tiles = (pc.cnt + kTile - 1) / kTile;
  pc.m0 = 0;
  pc.m1 = pc.cnt / kTile;
  if (!kList) {
    const int open = max(pc.p1, 0) - p.a.local + 1 - pc.lo;   // tokens that the last row no longer sees
    pc.m0 = pc.head / kTile + (max(open, 0) + kTile - 1) / kTile;
    pc.m1 = pc.head / kTile + max(pc.p0 - pc.lo + 1, 0) / kTile;
  }
  pc.base = p.a.pm.table ? pc.b * p.a.pm.pages_per_seq : (static_cast<int64_t>(pc.b) * p.Hkv + pc.g) * p.n_cap;
  if (p.whole) {
    pc.t0 = pc.tiles * w.start / w.end;   // few tiles, few parts
    pc.n = pc.tiles * (w.start + 1) / w.end - pc.t0;
  } else {
    const int first = w.x0 + kItemCost;
    pc.t0 = max(0, w.start - first) << p.ush;
    pc.n = max(0, min(pc.tiles, min(max(w.end - first, 0), (kTilesMost >> p.ush) + 1) << p.ush) - pc.t0);
  }
  return pc;
}

// Puts the next item of a warp's range into `to`: 0 where there is none, 1 for the
// last, else 2.  Items without a token are written on the way.
template <int kNT, int kKind>
__device__ __forceinline__ int next_piece(const Args& p, Smem<kNT>& S, int warp, Piece& to) {
  constexpr bool kList = kKind == kListed;
  constexpr int kRows = 8 * kNT;
  const int lane = threadIdx.x & 31;
  Walk walk = S.walk[warp];
  bool found = false;
  // whether an item may stand behind this one
  auto more = [&]() { return p.whole ? walk.left > 1 : walk.x0 + walk.span < walk.end; };
  __syncwarp();
  while (!found) {
    if (walk.used) {
      if (!more()) break;
      --walk.left;
      walk_on<kKind, kRows>(p, walk);
    }
    if (walk.b >= p.seqs) break;
    walk.used = 1;
    const Piece pc = piece_of<kList, kRows>(p, walk);
    if (pc.tiles == 0 && (p.whole ? walk.start == 0 : walk.x0 >= walk.start)) {
      for (int i = 0; i < pc.rows; ++i) {
        const int64_t at = row_of(p, pc.tok0, pc.g, i);
        *reinterpret_cast<uint2*>(p.a.out + at * kD + 4 * lane) = make_uint2(0, 0);
        if (p.a.lse && lane == 0) p.a.lse[at] = -INFINITY;
      }
    }
    found = pc.n > 0;
    if (found && lane == 0) to = pc;
    if (kList && found) {
      // the list's next entries and the sequence's pages, all of which come one behind the other otherwise
      const int64_t list = (p.a.sel_per_kv ? static_cast<int64_t>(pc.b) * p.Hkv + pc.g : pc.b) * p.a.K;
      const int e = max(kTile * pc.t0 - pc.head, 0) + kTile * lane;
      if (lane < 8 && e < pc.lo) prefetch_l2(p.a.sel + list + e);
      if (p.a.pm.table && kTile * lane < p.a.pm.pages_per_seq)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.a.pm.table + pc.base + kTile * lane) : "memory");
    }
  }
  if (lane == 0) S.walk[warp] = walk;
  __syncwarp();
  return found ? 1 + more() : 0;
}

template <int kNT, int kKind>
__global__ void __launch_bounds__(32 * warps_of(kNT), 1) kv4_attn_kernel(const __grid_constant__ Args p) {
  using Sm = Smem<kNT>;
  constexpr bool kList = kKind == kListed;
  constexpr int kRows = Sm::kRows, kWarps = Sm::kWarps, kThreads = 32 * kWarps, kStages = Sm::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Sm& S = *reinterpret_cast<Sm*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, j = lane & 3;
  pdl_wait();
  // The copy begins beside it (Kv4Copy::beside).  From here on a call of this kind writes out and lse
  // and nothing else: whole items leave no parts in the workspace.
  if (kKind == kRest && p.whole) pdl_trigger();

  // ---- this warp's part of the work.  Whole items of single tokens need no sums.
  const int groups = (p.seqs + (1 << p.ssh) - 1) >> p.ssh;
  const bool plain = p.whole && (kList || p.a.bt.cu_q == nullptr);
  if (!kList && blockIdx.x == gridDim.x - 1)
    for (int b = tid; b < p.B; b += kThreads) {
      const int len = __ldg(p.a.bt.lens + b);
      if (len < 0 || len > p.n_cap) record_error(p.err, kErrBadPage);
    }
  // A lane has kLaneSeq sequences of a short line (every warp for itself, without a
  // barrier), a thread a group of a long one.
  constexpr int kLaneSeq = 4;
  const bool short_line = p.seqs <= 32 * kLaneSeq;
  const int each_lane = (p.seqs + 31) / 32;
  unsigned lane_places = 0, lane_before = 0;   // of the lane's sequences, and before them
  int places = p.B * p.Hkv;
  if (!plain && short_line) {
#pragma unroll
    for (int i = 0; i < kLaneSeq; ++i) {
      const int b = lane * each_lane + i;
      if (i < each_lane && b < p.seqs) {
        const Seq s = seq_of<kList>(p, b);
        const int items = items_of<kKind, kRows>(p, s, b);
        if (items > 0) lane_places += static_cast<unsigned>(items) * span_of<kList, kRows>(p, s, b);
      }
    }
    unsigned inc = lane_places;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    lane_before = inc - lane_places;
    places = static_cast<int>(__shfl_sync(0xffffffffu, inc, 31));
  } else if (!plain) {
    for (int i = tid; i < groups; i += kThreads) {
      unsigned sum = 0;
      for (int b = i << p.ssh; b < min(p.seqs, (i + 1) << p.ssh); ++b) {
        const Seq s = seq_of<kList>(p, b);
        const int items = items_of<kKind, kRows>(p, s, b);
        if (items > 0) sum += static_cast<unsigned>(items) * span_of<kList, kRows>(p, s, b);
      }
      S.place[i] = static_cast<int>(sum);
    }
    __syncthreads();
    if (warp == 0) {
      unsigned sum = 0;
      for (int b0 = 0; b0 < groups; b0 += 32) {
        const int b = b0 + lane;
        const unsigned v = b < groups ? S.place[b] : 0;
        unsigned vi = v;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned x = __shfl_up_sync(0xffffffffu, vi, o);
          if (lane >= o) vi += x;
        }
        if (b < groups) S.place[b] = static_cast<int>(sum + vi - v);
        sum += __shfl_sync(0xffffffffu, vi, 31);
      }
      if (lane == 0) S.place[groups] = static_cast<int>(sum);
    }
    __syncthreads();
    places = S.place[groups];
  }
  auto walk_at = [&](int x) {   // the item that holds place x
    if (short_line) {
      const unsigned here = __ballot_sync(0xffffffffu, static_cast<unsigned>(x) - lane_before < lane_places);
      const int from = max(__ffs(here) - 1, 0);
      return walk_from<kKind, kRows>(p, from * each_lane, __shfl_sync(0xffffffffu, lane_before, from), x);
    }
    int lo = 0, hi = groups;   // the last group with place <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (S.place[mid] <= x) lo = mid;
      else hi = mid;
    }
    return walk_from<kKind, kRows>(p, lo << p.ssh, S.place[lo], x);
  };
  const Line line(places, max(1, min(static_cast<int>(gridDim.x), p.whole ? places : (places + kLeast - 1) / kLeast)));
  Walk walk;
  walk.b = p.seqs;
  walk.x0 = walk.end = walk.start = walk.left = walk.used = 0;
  if (blockIdx.x < line.G && places > 0) {
    const unsigned first = line.start(blockIdx.x), all = line.start(blockIdx.x + 1) - first;
    if (p.whole) {   // items of its own for every warp, or warps for every item
      int item, left = 0, part = 0, parts = 1;
      if (all >= kWarps) {
        item = all * warp / kWarps;
        left = all * (warp + 1) / kWarps - item;
      } else {
        parts = kWarps / all;
        item = warp / parts;
        part = warp - item * parts;
        left = item < static_cast<int>(all);
      }
      if (left > 0) {
        if (plain) {
          walk.b = kList ? first + item : (first + item) / p.Hkv;
          walk.rem = kList ? 0 : first + item - walk.b * p.Hkv;
          walk.s = seq_of<kList>(p, walk.b);
          walk.items = kList ? 1 : p.Hkv;
          walk.span = 1;
        } else {
          walk = walk_at(first + item);
        }
      }
      walk.left = left;
      walk.used = 0;
      walk.start = part;
      walk.end = parts;
    } else {
      const unsigned each = all / kWarps, more = all - each * kWarps;
      const int start = first + each * warp + more * warp / kWarps;
      const int end = first + each * (warp + 1) + more * (warp + 1) / kWarps;
      if (start < end) walk = walk_at(start);
      walk.used = 0;
      walk.start = start;
      walk.end = end;
    }
  }
  if (lane == 0) S.walk[warp] = walk;
  if (lane < 2) S.there[2 * warp + lane] = 0;   // each warp its own: no barrier stands before its stores to them
  __syncwarp();

  uint8_t* const ring = S.ring[warp];
  const uint32_t ring_s = smem_u32(ring);

  // ---- loads: the next tile's tokens and their rows are known a tile ahead of
  // their copies each (the block table and the list are read on the way)
  enum { kNone, kLine, kRowwise };          // no tile; 32 rows in a line; rows of their own
  int pushed = 0;                           // items found
  bool more = true;                         // there may be others
  int lt = 0, left = 0;                     // next tile of the newest item, tiles left of it
  int at0 = 0, m0 = 0, m1 = 0, tg = 0;      // of that item: token of tile 0's first slot in a line, whole tiles, KV head
  int64_t base = 0;
  int tok = kNoToken, tok_g = 0, tok_kind = kNone;   // lane's token of the tile after the next (of a line: its first)
  int64_t tok_base = 0;
  bool tok_there = false;                            // listed: the lane has a slot (an entry may be any number)
  int at = kNoToken, at_g = 0, at_kind = kNone;      // lane's token of the next tile,
  int at_page = 0;                                   // and its page or first row
  auto next_tokens = [&]() {
    if (__builtin_expect(left == 0, 0)) {
      Piece& pc = S.queue[warp][pushed % kQueue];
      const int found = more ? next_piece<kNT, kKind>(p, S, warp, pc) : 0;
      more = found == 2;
      if (found == 0) {
        tok_kind = kNone;
        return;
      }
      ++pushed;
      lt = pc.t0;
      left = pc.n;
      at0 = pc.lo - pc.head;
      m0 = pc.m0;
      m1 = pc.m1;
      tg = pc.g;
      base = pc.base;
    }
    if (!kList && __builtin_expect(lt >= m0 && lt < m1, 1)) {
      tok_kind = kLine;
      tok = at0 + lt * kTile;
    } else {
      tok_kind = kRowwise;
      const Piece& pc = S.queue[warp][(pushed - 1) % kQueue];
      tok = token_of_slot<kList>(p, pc, lt * kTile + lane);
      tok_there = lt * kTile + lane < pc.cnt;
    }
    tok_g = tg;
    tok_base = base;
    ++lt;
    --left;
  };
  // What is read here is used a tile later, so that no tile waits for it.
  auto next_rows = [&]() {
    at_kind = tok_kind;
    at = tok;
    at_g = tok_g;
    if (kList && tok_kind != kNone && tok_there && (tok < 0 || tok >= p.n)) {   // an entry outside the cache
      record_error(p.err, kErrBadPage);
      at = kNoToken;
    }
    at_page = static_cast<int>(tok_base);
    if (p.a.pm.table != nullptr && at_kind != kNone && at != kNoToken)
      at_page = __ldg(p.a.pm.table + tok_base + (at >> p.a.pm.page_shift));
    next_tokens();
  };
  uint32_t put = 0;   // stage that the next copies go to
  // K rows stand as they are; V rows with the low bits of their number swapped
  // and their chunks turned by a half where bit 2 is set: a lane's four tokens, 2j
  // and 2j + 1 of eight, are then in banks of their own.
  const uint32_t k_at = 16 * lane, kf_at = kTileCodes + lane * kKv4Groups;
  const uint32_t v_at = kTileCodes + kTileScales + ((r & 4) | (r & 1) << 1 | (r >> 1 & 1)) * kKv4Codes + 16 * (j ^ (r >> 1 & 2));
  auto issue = [&]() {
    const uint32_t to = ring_s + put * kStage;
    int row = -1;   // lane's row (of a line: its first); -1: none
    if (at_kind != kNone && at != kNoToken) {
      if (p.a.pm.table == nullptr) {
        row = at_page + at;
      } else if (at_page >= 0 && at_page < p.a.pm.num_pages) {
        row = ((at_page * p.Hkv + at_g) << p.a.pm.page_shift) + (at & ((1 << p.a.pm.page_shift) - 1));
      } else {   // (of a line: in every lane)
        record_error(p.err, kErrBadPage);
        at_kind = kRowwise;
      }
    }
    if (__builtin_expect(!kList && at_kind == kLine, !kList)) {
      const int64_t codes = static_cast<int64_t>(row) * kKv4Codes + 16 * lane;
      const int64_t scales = static_cast<int64_t>(row) * kKv4Groups + kKv4Groups * lane;
      const uint8_t* k = p.a.kv.K + codes;
      const uint8_t* v = p.a.kv.V + codes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cp_async16(to + k_at + 8 * i * kKv4Codes, k + 8 * i * kKv4Codes);
        cp_async16(to + v_at + 8 * i * kKv4Codes, v + 8 * i * kKv4Codes);
      }
      cp_async8(to + kf_at, p.a.kv.K_sf + scales);
      cp_async8(to + kf_at + kTileCodes + kTileScales, p.a.kv.V_sf + scales);
    } else if (at_kind == kRowwise) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int from = __shfl_sync(0xffffffffu, row, r + 8 * i);   // rows that are none: zeros
        const int64_t src = static_cast<int64_t>(max(from, 0)) * kKv4Codes + 16 * j;
        cp_async16_zfill(to + k_at + 8 * i * kKv4Codes, p.a.kv.K + src, from >= 0 ? 16 : 0);
        cp_async16_zfill(to + v_at + 8 * i * kKv4Codes, p.a.kv.V + src, from >= 0 ? 16 : 0);
      }
      const int64_t own = static_cast<int64_t>(max(row, 0)) * kKv4Groups;
      cp_async8_zfill(to + kf_at, p.a.kv.K_sf + own, row >= 0 ? 8 : 0);
      cp_async8_zfill(to + kf_at + kTileCodes + kTileScales, p.a.kv.V_sf + own, row >= 0 ? 8 : 0);
    }
    cp_async_commit();
    put = put + 1 == kStages ? 0 : put + 1;
    next_rows();
  };
  next_tokens();

  // Queries of an item, column 8 nt + r of its rows: a lane holds 32 values.  Those of
  // the next item are on their way while an item's rows are written.
  uint4 qx[kNT][4];
  auto load_queries = [&](const Piece& pc) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const int col = 8 * nt + r;
      const uint4* q = reinterpret_cast<const uint4*>(p.a.q + row_of(p, pc.tok0, pc.g, col) * kD + 32 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) qx[nt][i] = col < pc.rows ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
    }
  };
  if (pushed > 0) load_queries(S.queue[warp][0]);
  next_rows();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) issue();
  uint32_t take = 0;   // stage of the next tile

  for (int done = 0; done < pushed; ++done) {
    __syncwarp();
    const Piece& pc = S.queue[warp][done % kQueue];   // written again only when its products are long done

    // ---- queries in fp16
    uint32_t qf[kNT][16];
    float cs[kNT][2];   // of columns 2j, 2j + 1: logits in log2 units per unit of the product
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = qx[nt][i];
        const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        top = max(top, max(m & 0xffffu, m >> 16));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = min(max(static_cast<int>(top >> 7), 32), 254);   // 2^(ex - 127) <= largest value
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);     // to 2^14 ..
      const float down = __uint_as_float(static_cast<uint32_t>(127 + ex - 141) << 23) * kScale * p.a.kv.k_scale;
      cs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * j);
      cs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * j + 4);
      const uint32_t* w = &qx[nt][0].x;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = bf2_to_f2(w[i]);
        qf[nt][i] = pack_half(f.x * up, f.y * up);
      }
    }

    float o[8][kNT][4];
    float mx[kNT][2], l[kNT][2];
    float base2[kNT][2];   // added to a logit: kBase - mx, 0 before there is a maximum
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      mx[nt][0] = mx[nt][1] = -INFINITY;
      base2[nt][0] = base2[nt][1] = 0.0f;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
    }

    const int t_end = pc.t0 + pc.n, w0 = pc.m0, w1 = pc.m1;
    for (int t = pc.t0; t < t_end; ++t) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      issue();   // into the stage that the tile before this one has left
      const uint8_t* st = ring + take * kStage;
      take = take + 1 == kStages ? 0 : take + 1;

      // ---- S^T = K Q^T
      float s[2][kNT][4];
      uint4 kw[2][2];
      __half2 kf[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          kw[mt][h] = *reinterpret_cast<const uint4*>(st + k_at + (16 * mt + 8 * h) * kKv4Codes);
          kf[mt][h] = kv4_scales(*reinterpret_cast<const uint16_t*>(st + kTileCodes + (16 * mt + 8 * h + r) * kKv4Groups + 2 * j));
        }
      }
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const __half2 g0 = w < 2 ? __low2half2(kf[mt][0]) : __high2half2(kf[mt][0]);
          const __half2 g1 = w < 2 ? __low2half2(kf[mt][1]) : __high2half2(kf[mt][1]);
          __half2 c0[4], c1[4];
          kv4_codes((&kw[mt][0].x)[w], c0);
          kv4_codes((&kw[mt][1].x)[w], c1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = bits(__hmul2(c0[2 * h], g0)), a1 = bits(__hmul2(c1[2 * h], g1));
            const uint32_t a2 = bits(__hmul2(c0[2 * h + 1], g0)), a3 = bits(__hmul2(c1[2 * h + 1], g1));
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) mma16816(s[mt][nt], a0, a1, a2, a3, qf[nt][4 * w + 2 * h], qf[nt][4 * w + 2 * h + 1]);
          }
        }

      // ---- masked where the tile is not attended to as a whole
      if (__builtin_expect(t < w0 || t >= w1, 0)) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int slot = kTile * t + 16 * mt + 8 * h + r;
            const int token = kList ? 0 : token_of_slot<false>(p, pc, slot);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int pos = pc.p0 + ((8 * nt + 2 * j + c) >> p.gsh);
                if (kList ? slot >= pc.cnt : token == kNoToken || !attends(p, pos, token)) s[mt][nt][2 * h + c] = -INFINITY;
              }
          }
      }

      // ---- the rows' maxima: the base moves where one grew by more than kGrow
      bool grown = false;
      float top[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[nt][c] = fmaxf(fmaxf(s[0][nt][c], s[0][nt][2 + c]), fmaxf(s[1][nt][c], s[1][nt][2 + c])) * cs[nt][c];
          grown |= top[nt][c] > mx[nt][c] + kGrow;
        }
      if (__builtin_expect(__any_sync(0xffffffffu, grown), 0)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = top[nt][c];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            if (m > mx[nt][c]) {
              const float f = ex2_approx(mx[nt][c] - m);   // 0 for the first
              mx[nt][c] = m;
              base2[nt][c] = kBase - m;
              l[nt][c] *= f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                o[i][nt][c] *= f;
                o[i][nt][2 + c] *= f;
              }
            }
          }
      }

      // ---- P, and turned to the second product's operand
      uint32_t pf[2][kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2_approx(fmaf(s[mt][nt][2 * h], cs[nt][0], base2[nt][0]));
            const float p1 = ex2_approx(fmaf(s[mt][nt][2 * h + 1], cs[nt][1], base2[nt][1]));
            l[nt][0] += p0;
            l[nt][1] += p1;
            pf[mt][nt][h] = transpose8x8(pack_half(p0, p1));
          }
      }

      // ---- O^T += V^T P^T: channels 16 r + 2 i and + 1 are rows r and r + 8 of tile i
      const uint8_t* vt = st + kTileCodes + kTileScales;
      const uint8_t* vf = vt + kTileCodes + r;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint2 w[2][2];
        __half2 f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = 16 * mt + 8 * h + ((j & 1) | e << 1 | (j & 2) << 1);
            w[h][e] = *reinterpret_cast<const uint2*>(vt + at * kKv4Codes + 16 * ((r >> 1) ^ (j & 2)) + 8 * (r & 1));
          }
          const uint8_t* sf = vf + (16 * mt + 8 * h + 2 * j) * kKv4Groups;
          f[h] = kv4_scales(sf[0] | static_cast<uint32_t>(sf[kKv4Groups]) << 8);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          __half2 ev[2][4], od[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = half ? w[h][0].y : w[h][0].x, y = half ? w[h][1].y : w[h][1].x;
            kv4_codes((x & 0x0f0f0f0fu) | (y << 4 & 0xf0f0f0f0u), ev[h]);
            kv4_codes((x >> 4 & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), od[h]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = bits(__hmul2(ev[0][i], f[0])), a1 = bits(__hmul2(od[0][i], f[0]));
            const uint32_t a2 = bits(__hmul2(ev[1][i], f[1])), a3 = bits(__hmul2(od[1][i], f[1]));
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) mma16816(o[4 * half + i][nt], a0, a1, a2, a3, pf[mt][nt][0], pf[mt][nt][1]);
          }
        }
      }
    }

    // ---- the piece's rows
    __syncwarp();
    if (done + 1 < pushed) load_queries(S.queue[warp][(done + 1) % kQueue]);
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
    const bool begins = pc.t0 == 0, ends = pc.t0 + pc.n == pc.tiles;
    if (begins && ends) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 8 * nt + 2 * j + c;
          if (col >= pc.rows) continue;
          const int64_t at = row_of(p, pc.tok0, pc.g, col);
          const float inv = inverse_of(p, l[nt][c]);
          uint4* dst = reinterpret_cast<uint4*>(p.a.out + at * kD + 16 * r);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            dst[i] = make_uint4(pack_bf16(o[4 * i][nt][c] * inv, o[4 * i][nt][2 + c] * inv),
                                pack_bf16(o[4 * i + 1][nt][c] * inv, o[4 * i + 1][nt][2 + c] * inv),
                                pack_bf16(o[4 * i + 2][nt][c] * inv, o[4 * i + 2][nt][2 + c] * inv),
                                pack_bf16(o[4 * i + 3][nt][c] * inv, o[4 * i + 3][nt][2 + c] * inv));
          if (p.a.lse && r == 0) p.a.lse[at] = lse_of(mx[nt][c], l[nt][c]);
        }
    } else {
      // The item that goes on behind this warp's range is its last: its ring is free by then.
      if (begins) cp_async_wait<0>();
      __syncwarp();
      Part<kRows>& to = begins ? *reinterpret_cast<Part<kRows>*>(ring) : S.first[warp];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 8 * nt + 2 * j + c;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            to.o[col][(4 * r + i) ^ j] = make_float4(o[2 * i][nt][c], o[2 * i][nt][2 + c], o[2 * i + 1][nt][c], o[2 * i + 1][nt][2 + c]);
          if (r == 0) to.ml[col] = make_float2(mx[nt][c], l[nt][c]);
        }
      if (lane == 0) {
        S.part[2 * warp + begins] = pc;
        S.there[2 * warp + begins] = ends ? 2 : 1;
      }
    }
  }

  // ---- the warps' parts joined: a chain begins with an item's first part, or with
  // the block's first one where the item began before; the firsts of the warps behind it
  // (even places) continue it until one ends.  A thread joins four channels of a row.
  // (With a warp to a row, or a warp finding a row's factors first, this took 6000
  // cycles behind the last product, 5 % of 64 sequences with a 4K window.)
  __syncthreads();
  const int state = lane < 2 * kWarps ? S.there[lane] : 0;
  const unsigned present = __ballot_sync(0xffffffffu, state != 0), ended = __ballot_sync(0xffffffffu, state == 2);
  constexpr unsigned kFirsts = 0x55555555u;   // even places
  bool left_over = false;   // an item goes on behind the block
  int x = tid;              // of the chains' rows, 32 fours of channels each, the next that is this thread's
  for (unsigned heads = present & (~kFirsts | (present & -present)); heads != 0; heads &= heads - 1) {
    const int i = __ffs(heads) - 1;
    const bool begins = (i & 1) != 0;
    // the even places behind i up to the first that ends (the one at i itself may)
    unsigned chain = ((ended >> i) & 1) ? 0 : present & kFirsts & ~((2u << i) - 1);
    const unsigned stop = chain & ended;
    const bool ends = ((ended >> i) & 1) || stop != 0;
    if (stop) chain &= (stop & -stop) * 2u - 1;
    left_over |= begins && !ends;
    const int w0 = (i >> 1) + 1, w1 = chain ? (31 - __clz(chain)) >> 1 : 0;   // warps of the others
    const Part<kRows>& head = begins ? *reinterpret_cast<const Part<kRows>*>(S.ring[i >> 1]) : S.first[i >> 1];
    const Piece& pc = S.part[i];
    const int rows = pc.rows;
#pragma unroll 1
    for (; x < 32 * rows; x += kThreads) {
      const int col = x >> 5, four = x & 31, at = four ^ (col >> 1 & 3);
      float m = head.ml[col].x;
#pragma unroll 4
      for (int w = w0; w <= w1; ++w)
        if ((chain >> 2 * w) & 1) m = fmaxf(m, S.first[w].ml[col].x);
      float l = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      auto add = [&](const Part<kRows>& part) {
        const float2 ml = part.ml[col];
        const float4 y = part.o[col][at];
        const float f = m == -INFINITY ? 1.0f : ex2_approx(ml.x - m);
        l += ml.y * f;
        o = make_float4(o.x + y.x * f, o.y + y.y * f, o.z + y.z * f, o.w + y.w * f);
      };
      add(head);
#pragma unroll 4
      for (int w = w0; w <= w1; ++w)
        if ((chain >> 2 * w) & 1) add(S.first[w]);
      if (begins && ends) {
        const int64_t row = row_of(p, pc.tok0, pc.g, col);
        const float inv = inverse_of(p, l);
        *reinterpret_cast<uint2*>(p.a.out + row * kD + 4 * four) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (p.a.lse && four == 0) p.a.lse[row] = lse_of(m, l);
      } else {
        const int64_t to = (static_cast<int64_t>(blockIdx.x) * 2 + begins) * kRows + col;
        *(reinterpret_cast<float4*>(p.part_o + to * kD) + four) = o;
        if (four == 0) p.part_ml[to] = make_float2(m, l);
      }
    }
    x -= 32 * rows;
    if (tid == kThreads - 1 && begins && !ends) {
      Share sh;
      sh.first = static_cast<int64_t>(pc.tok0) << p.gsh;
      sh.rows = rows;
      sh.g = pc.g;
      sh.last = line.block(pc.x0 + kItemCost + ((pc.tiles - 1) >> p.ush));
      sh.pad = 0;
      p.share[blockIdx.x] = sh;
    }
  }
  if (tid == 0 && !left_over && !p.whole) p.share[blockIdx.x].rows = 0;
  pdl_trigger();
}

// Joins the parts of an item that several blocks share: exact log-sum-exp,
// fp32.  Block (c, row) has a row of the item whose first tiles attention block c
// had: its warps take every eighth part, a lane four channels.
constexpr int kMergeWarps = 8;

template <int kNT>
__global__ void __launch_bounds__(32 * kMergeWarps) kv4_merge_kernel(const Args p) {
  constexpr int kRows = 8 * kNT;
  __shared__ float4 so[kMergeWarps][32];
  __shared__ float2 sml[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.y;
  pdl_wait();
  const Share sh = p.share[blockIdx.x];
  if (col < sh.rows) {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto join = [&](const float2 v, const float4 y) {
      const float mn = fmaxf(m, v.x);
      const float a = mn == -INFINITY ? 1.0f : ex2_approx(m - mn), b = mn == -INFINITY ? 1.0f : ex2_approx(v.x - mn);
      m = mn;
      l = l * a + v.y * b;
      o = make_float4(o.x * a + y.x * b, o.y * a + y.y * b, o.z * a + y.z * b, o.w * a + y.w * b);
    };
    constexpr int kAhead = 4;   // parts whose loads a warp has in flight
    for (int c0 = blockIdx.x + warp; c0 <= sh.last; c0 += kAhead * kMergeWarps) {
      float2 v[kAhead];
      float4 y[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = c0 + i * kMergeWarps;
        v[i] = make_float2(-INFINITY, 0.0f);
        y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c <= sh.last) {
          const int64_t part = (static_cast<int64_t>(c) * 2 + (c == static_cast<int>(blockIdx.x))) * kRows + col;
          v[i] = __ldcg(p.part_ml + part);
          y[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + part * kD) + lane);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) join(v[i], y[i]);
    }
    so[warp][lane] = o;
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kMergeWarps; ++w) join(sml[w], so[w][lane]);
      const int64_t row = sh.first + col;
      const int64_t at = (row >> p.gsh) * p.Hq + (sh.g << p.gsh) + (row & ((1 << p.gsh) - 1));
      const float inv = inverse_of(p, l);
      *reinterpret_cast<uint2*>(p.a.out + at * kD + 4 * lane) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
      if (p.a.lse && lane == 0) p.a.lse[at] = lse_of(m, l);
    }
  }
  pdl_trigger();
}

struct Layout {
  size_t off_ml = 0, off_o = 0, total = 0;
};
Layout layout_of(int rows, int grid) {
  Layout L;
  L.off_ml = align_up(static_cast<size_t>(grid) * sizeof(Share), 256);
  L.off_o = align_up(L.off_ml + static_cast<size_t>(grid) * 2 * rows * sizeof(float2), 256);
  L.total = align_up(L.off_o + static_cast<size_t>(grid) * 2 * rows * kD * sizeof(float), 256);
  return L;
}

using Kernel = void (*)(Args);
Kernel kernel_of(int nt, Kind kind) {
  if (nt == 1) return kind == kListed ? kv4_attn_kernel<1, kListed> : (kind == kRest ? kv4_attn_kernel<1, kRest> : kv4_attn_kernel<1, kWindow>);
  return kv4_attn_kernel<2, kWindow>;
}
Kernel merge_of(int nt) { return nt == 1 ? kv4_merge_kernel<1> : kv4_merge_kernel<2>; }
size_t smem_of(int nt) { return nt == 1 ? sizeof(Smem<1>) : sizeof(Smem<2>); }
static_assert(sizeof(Smem<1>) <= 232448 && sizeof(Smem<2>) <= 232448, "shared memory of a block");

// Columns of an item: single tokens have at most eight.
int tiles_of(const qasc_shape& s, int64_t max_q) { return max_q * (s.Hq / s.Hkv) <= 8 ? 1 : 2; }

constexpr int64_t kCopyBytes = int64_t(1) << 32;   // of a copy, at most

// Sequences of a call that are copied, of `seqs` that may be: they are taken to have two thirds
// of max_q new tokens.
double copies_of(int64_t T, int64_t max_q, int64_t seqs) { return std::min<double>(seqs, std::max(1.0, 1.5 * T / max_q)); }

// Whether the copy pays for a call that may have such sequences (microseconds on 152 SMs, within a
// quarter of what was measured for 132 to 8192 rows a sequence, 256 to 131072 tokens of window): it is two kernels more
// (23), its bytes (5.5 TB/s), and the products over it (1.4 PFLOP/s); here every block of 16 rows takes
// 1.05 ns a tile that its rows see.  2048 new of 32768 tokens, 32 / 8 heads: 4671 us here, 726 over a copy (the
// lines: 4423 and 840); 16 sequences of 64 new tokens, local 512, 8 / 2 heads: 22.5 and 23 (19 and 27).
bool copy_pays(const qasc_shape& s, int64_t T, int64_t max_q, int64_t tokens, int64_t seqs, int64_t window) {
  const double gq = s.Hq / s.Hkv, rows = T * gq, copies = copies_of(T, max_q, seqs);
  const double seen = std::min<int64_t>(tokens, window + 15), seen256 = std::min<double>(tokens, window + 255 / gq);
  const double here = 10.0 + (rows / 16.0 + 1.0) * seen * s.Hkv / kTile * 1.05e-3;
  const double copy = 23.0 + copies * tokens * s.Hkv * 656.0 / 5.5e6 + rows * seen256 * s.Hkv * 512.0 / 1.4e9;
  return copy < here;
}

// Whether it may pay for any call of up to T tokens, whatever its max_q: what attention takes here
// (which does not fall with max_q) against the least that a copy takes, both lines in the tokens.
bool copy_may_pay(const qasc_shape& s, int64_t T, int64_t window) {
  const double gq = s.Hq / s.Hkv, least = kCopyRows / (s.Hq / s.Hkv) + 1;   // new tokens of a sequence that is copied
  const double seen = std::min<int64_t>(s.n_cap, window + 15), tokens = std::min<double>(s.n_cap, window + least - 1);
  for (const double t : {static_cast<double>(T), least}) {
    const double here = 10.0 + (t * gq / 16.0 + 1.0) * seen * s.Hkv / kTile * 1.05e-3;
    const double copy = 23.0 + tokens * s.Hkv * 656.0 / 5.5e6 + t * gq * tokens * s.Hkv * 512.0 / 1.4e9;
    if (copy < here + 1e-6) return true;
  }
  return false;
}

struct CopyLayout {
  int64_t capacity = 0, pages_per_seq = 0;   // capacity 0: no copy
  int64_t seqs = 0;                          // sequences that can be long enough
  bool all = false;                          // (of a call) there is room for every sequence that is long enough
  size_t off_lists = 0, off_attn = 0, attn_bytes = 0, off_k = 0, off_v = 0, total = 0;
};
// Of calls whose sequences have at most max_q new tokens: everything that a copy takes.  No part of it
// falls with more tokens, sequences or a larger max_q.
CopyLayout copy_space(const qasc_shape& s, int64_t T, int64_t max_q, int64_t window) {
  CopyLayout L;
  const int64_t gq = s.Hq / s.Hkv, tokens = std::min<int64_t>(s.n_cap, window + max_q - 1);
  L.pages_per_seq = (tokens + kCopyPage - 1) / kCopyPage;
  L.seqs = std::min<int64_t>(s.B, T * gq / (kCopyRows + 1));   // that can be as long
  const int64_t page_bytes = static_cast<int64_t>(s.Hkv) * kCopyPage * kD * 2;
  const int64_t most = std::min(kCopyBytes / (2 * page_bytes), ((int64_t(1) << 31) - 1) / (s.Hkv * kCopyPage));
  L.capacity = std::min(L.seqs * L.pages_per_seq, most);
  L.off_lists = align_up(kv4_attn_least_bytes(), 256);
  L.off_attn = align_up(L.off_lists + static_cast<size_t>(s.B) * (2 + L.pages_per_seq) * sizeof(int32_t), 256);
  L.attn_bytes = kv_attn_workspace_bytes(T, s.B, s.Hq, s.Hkv, false, kMaxSmsForSizing);
  L.off_k = align_up(L.off_attn + L.attn_bytes, 256);
  L.off_v = L.off_k + static_cast<size_t>(L.capacity * page_bytes);
  L.total = L.off_v + static_cast<size_t>(L.capacity * page_bytes);
  return L;
}

// Of one call with a workspace of ws_bytes: the copy takes what room there is, if it is enough for
// the longest sequence.
CopyLayout copy_layout(const qasc_shape& s, int64_t T, int64_t max_q, int32_t sink, int32_t local, size_t ws_bytes) {
  const int64_t window = static_cast<int64_t>(sink) + local;
  if (max_q * (s.Hq / s.Hkv) <= kCopyRows) return CopyLayout();
  CopyLayout L = copy_space(s, T, max_q, window);
  const int64_t cap = L.pages_per_seq * kCopyPage;
  if (cap >= kTokensMost || static_cast<int64_t>(s.B) * s.Hkv * cap >= (int64_t(1) << 31)) return CopyLayout();
  if (!copy_pays(s, T, max_q, std::min(s.n_cap, window + max_q - 1), L.seqs, window)) return CopyLayout();
  const size_t page_bytes = static_cast<size_t>(s.Hkv) * kCopyPage * kD * 2;
  const size_t room = ws_bytes > L.off_k ? (ws_bytes - L.off_k) / (2 * page_bytes) : 0;
  if (room < static_cast<size_t>(L.capacity)) {
    if (room < static_cast<size_t>(L.pages_per_seq)) return CopyLayout();
    L.capacity = static_cast<int64_t>(room);
    L.off_v = L.off_k + room * page_bytes;
  }
  L.all = L.capacity == L.seqs * L.pages_per_seq;
  return L;
}

// The sequences that are copied: their copy, and kv_window_attn's kernel over it.
int attend_over_copy(const qasc_shape& s, const Kv4AttnArgs& a, const Args& p, const CopyLayout& C, uint8_t* ws,
                     const DeviceInfo& dev, cudaStream_t stream) {
  Kv4Copy c;
  c.most_rows = kCopyRows;
  c.capacity = C.capacity;
  c.pages_per_seq = C.pages_per_seq;
  const int copies = static_cast<int>(copies_of(a.bt.T, a.max_q, C.seqs) + 0.5);
  c.likely = std::min(copies * C.pages_per_seq, C.capacity);
  c.copied = reinterpret_cast<int32_t*>(ws + C.off_lists);
  c.lens = c.copied + s.B;
  c.table = c.lens + s.B;
  c.K = reinterpret_cast<uint16_t*>(ws + C.off_k);
  c.V = reinterpret_cast<uint16_t*>(ws + C.off_v);
  c.beside = C.all && p.whole;
  const cudaError_t e = launch_kv4_copy(s, a.pm, a.bt, a.kv, p.a.sink, p.a.local, c, dev, stream);
  if (e != cudaSuccess) return static_cast<int>(e);
  qasc_shape s2 = s;
  s2.n = s2.n_cap = C.pages_per_seq * kCopyPage;
  KvAttnArgs k;
  k.q = a.q;
  k.K = c.K;
  k.V = c.V;
  k.out = a.out;
  k.lse = a.lse;
  k.bt = a.bt;
  k.bt.lens = c.lens;
  k.skip_empty = true;   // those that are not copied have no tokens there
  k.seqs = copies;
  k.pm.table = c.table;
  k.pm.pages_per_seq = C.pages_per_seq;
  k.pm.num_pages = C.capacity;
  while ((1 << k.pm.page_shift) < kCopyPage) ++k.pm.page_shift;
  k.cache_rows = C.capacity * s.Hkv * kCopyPage;
  k.sink = a.sink;
  k.local = a.local;
  size_t bytes = C.attn_bytes;
  return launch_kv_attn(s2, k, ws + C.off_attn, &bytes, dev, stream);
}

}  // namespace

size_t kv4_attn_least_bytes() { return layout_of(16, kMaxSmsForSizing).total; }

size_t kv4_window_workspace_bytes(const qasc_shape& s, int64_t T, int64_t max_q, int32_t sink, int32_t local) {
  const int64_t window = static_cast<int64_t>(sink) + local;
  if (max_q * (s.Hq / s.Hkv) <= kCopyRows || !copy_may_pay(s, T, window)) return kv4_attn_least_bytes();
  return copy_space(s, T, max_q, window).total;
}

int launch_kv4_attn(const qasc_shape& s, const Kv4AttnArgs& a, uint8_t* ws, size_t ws_bytes, const DeviceInfo& dev,
                    cudaStream_t stream) {
  Args p{};
  p.a = a;
  p.a.sink = std::min(a.sink, kTokensMost);   // more mean the same
  p.a.local = std::min(a.local, kTokensMost);
  p.B = s.B;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  while ((1 << p.gsh) < s.Hq / s.Hkv) ++p.gsh;
  p.n_cap = s.n_cap;
  if (a.listed) {
    const Regions R = regions_of(s.n, a.sink, a.local);
    p.n = static_cast<int>(s.n);
    p.sink_end = static_cast<int>(R.sink_end);
    p.local_start = static_cast<int>(R.local_start);
  }
  p.seqs = a.listed ? s.B * s.Hkv : s.B;
  while ((p.seqs - 1) >> p.ssh >= kSums) ++p.ssh;
  p.err = dev.err_word;

  const CopyLayout C = a.listed ? CopyLayout() : copy_layout(s, a.bt.T, a.max_q, a.sink, a.local, ws_bytes);
  const int64_t gq = s.Hq / s.Hkv;
  // What a call with long sequences leaves is likely to be single tokens.
  const int nt = a.listed || C.capacity > 0 ? 1 : tiles_of(s, a.max_q);
  const int64_t blocks = (a.bt.T * gq + 8 * nt - 1) / (8 * nt) + s.B;   // row blocks of a KV head, at most
  while (blocks * s.Hkv * (((s.n_cap / kTile + 2) >> p.ush) + 1 + kItemCost) >= (int64_t(1) << 31)) ++p.ush;
  // Items of few tiles are not shared between blocks, which saves the merge, where no warp has
  // to take a second one.
  const int64_t most = a.listed ? p.sink_end + static_cast<int64_t>(a.K) + (p.n - p.local_start)
                                : std::min<int64_t>(s.n_cap, static_cast<int64_t>(p.a.local) + p.a.sink + 8 * nt / gq - 1);
  const int grid = dev.num_sms;
  const bool packed = !a.listed && a.bt.cu_q && C.capacity == 0;
  const int64_t items = (packed ? a.bt.T * gq / (8 * nt) + (s.B + 1) / 2 : s.B) * s.Hkv;   // about
  p.whole = most <= (items <= static_cast<int64_t>(grid) * warps_of(nt) ? kWholeTokens : kWholeMany);
  const Layout L = layout_of(8 * nt, grid);
  p.share = reinterpret_cast<Share*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + L.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + L.off_o);
  const Kind kind = a.listed ? kListed : (C.all ? kRest : kWindow);
  auto attend = [&]() {
    return launch_dependent(kernel_of(nt, kind), dim3(grid), dim3(32 * warps_of(nt)), smem_of(nt), stream, 1, p);
  };
  // Of a call with a copy the rest goes first, where no plan has to tell which sequences found
  // room (31 single tokens beside 512 new ones, 8192 cached, 64 / 8 heads: 178 us, 266 when
  // the copied ones went first and took the others for sequences without a token).  Where items
  // are short, most SMs have none and the copy is made on them at the same time (16 ragged
  // sequences: 31 us, 34.4 one behind the other); where they are long it is kept from an even
  // spread by those that run (300 new and 40 single tokens, 2048 cached: 71 and 64).
  p.copy_tokens = C.pages_per_seq * kCopyPage;
  cudaError_t e = cudaSuccess;
  if (C.capacity == 0 || C.all) e = attend();
  if (e == cudaSuccess && C.capacity > 0) {
    const int rc = attend_over_copy(s, a, p, C, ws, dev, stream);
    if (rc != 0) return rc;
    if (!C.all) {
      p.copied = reinterpret_cast<const int32_t*>(ws + C.off_lists);
      e = attend();
    }
  }
  if (e != cudaSuccess || p.whole) return static_cast<int>(e);
  e = launch_dependent(merge_of(nt), dim3(grid, 8 * nt), dim3(32 * kMergeWarps), 0, stream, 1, p);
  return static_cast<int>(e);
}

cudaError_t configure_kv4_kernels(const DeviceInfo& dev) {
  (void)dev;
  for (int nt = 1; nt <= 2; ++nt)
    for (Kind kind : {kWindow, kRest, kListed}) {
      const cudaError_t e = cudaFuncSetAttribute(kernel_of(nt, kind), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem_of(nt)));
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace qasc
