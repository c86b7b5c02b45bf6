// kv4_window_attn and kv4_sparse_attn: attention over a 4-bit cache (kv4.cuh).
//
//   out[t,h,:] = sum_{j in A(t)} softmax_j(q[t,h].K_j / sqrt(d)) V_j
// with A(t) the sink and the newest `local` tokens up to t's own position, or
// (listed) the sink, the listed and the local tokens of a decode step.
//
// What bounds it.  144 bytes of a token and KV head are read for 512 operations
// per query head: bytes, as long as the codes become operands fast enough.  At
// HBM's rate an SM gets some 22 bytes a cycle, 45 values, twice as bf16 what its
// shared memory could write and tensor cores read again (128 bytes a cycle): so
// codes go from shared memory to registers, become fp16 there, and are the
// register operand of the product (mma.sync, 16 x 8 x 16), which a tcgen05
// product does not have for 8 to 16 query rows.  The products themselves take
// a fourth of that path's rate.
//
// Work.  The queries of a KV head's group share its keys: an item is up to
// 8 kNT rows (token, head of the group) of a sequence and KV head.  Its tokens
// (sink, window or list) are numbered without gaps, in tiles of 32.  The tiles of
// all items are laid end to end, every block takes an equal range of that line,
// and its warps take every kWarps-th tile of an item, each with a running maximum
// and sum of its own, so that nothing but an item's end makes them wait for each
// other.  Keys stand as rows of the first product and channels as rows of the
// second, queries as columns of both:
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
// rounded to fp16 (2^-12 of each weight, a sixteenth of the bf16 output's own
// rounding); its base is 2^-10 of the row's maximum when it was taken, and moves
// when the maximum grows by more than 2^5: P stays below 2^15, and weights down
// to 2^-24 of the largest keep all their bits.  The sum that divides takes P
// unrounded.
//
// An item that several blocks share leaves (max, sum, O) of each in the
// workspace, two places a block (the item that it begins with, the one that it ends
// with), and kv4_merge_kernel joins them.
#include <algorithm>
#include <climits>

#include "internal.h"
#include "kv4.cuh"

namespace qasc {
namespace {

constexpr int kTile = 32;                      // tokens of a warp's tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;                     // tiles of a warp's ring
constexpr int kTileCodes = kTile * kKv4Codes;  // bytes
constexpr int kTileScales = kTile * kKv4Groups;
constexpr int kStage = 2 * (kTileCodes + kTileScales);
constexpr int kMaxSeq = 2048;
constexpr int kPieces = 64;                    // items of a block's range planned at once
constexpr int kItemCost = 8;                   // places of an item beside its tiles: queries, join, output
constexpr int kLeast = 16;                     // places that a block takes at least
constexpr float kBase = 10.0f;                 // log2 of P at the maximum that the base was taken from
constexpr float kGrow = 5.0f;                  // growth of the maximum that moves the base
constexpr int kOutPad = 4;
// log2(e) / sqrt(128): logits in base-2 units.
constexpr float kScale = 1.4426950408889634f * 0.08838834764831845f;

struct Args {
  Kv4AttnArgs a;
  int B, Hq, Hkv, gsh;      // gsh = log2(Hq / Hkv)
  int64_t n_cap;
  int n, sink_end, local_start;   // listed: tokens of every sequence, its regions
  int64_t most_rows;        // sequences with more rows are left out (0: none)
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

// A block's part of an item: tiles t0 .. t0 + n - 1.
struct Piece {
  int tok0, rows;      // first query token, rows
  int b, g;
  int p0, p1;          // positions of the first and last row
  int lo;              // window: token behind the sink's; listed: list's entries
  int head, cnt;       // tokens of the sink, of all
  int t0, n;
  int whole;           // every tile: the output is written, not a part
  int slot, last;      // part's place; last block that has one
};

struct Seq {
  int q0, ql, len;
};

__device__ __forceinline__ int clampi(int64_t v, int64_t lo, int64_t hi) {
  return static_cast<int>(v < lo ? lo : (v > hi ? hi : v));
}

template <bool kList>
__device__ __forceinline__ Seq seq_of(const Args& p, int b) {
  Seq r;
  if (kList) {
    r.q0 = b;
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
// most tiles that any of them has.
template <bool kList, int kRows>
__device__ __forceinline__ int items_of(const Args& p, const Seq& s) {
  const int64_t rows = static_cast<int64_t>(s.ql) << p.gsh;
  if (p.most_rows && rows > p.most_rows) return 0;
  return static_cast<int>((rows + kRows - 1) / kRows) * p.Hkv;
}
template <bool kList, int kRows>
__device__ __forceinline__ int span_of(const Args& p, const Seq& s, int b) {
  int64_t cnt;
  if (kList) {
    int most = 0;
    for (int g = 0; g < (p.a.sel_per_kv ? p.Hkv : 1); ++g) most = max(most, list_len(p, b, g));
    cnt = p.sink_end + most + (p.n - p.local_start);
  } else {
    cnt = min(static_cast<int64_t>(s.len),
              static_cast<int64_t>(p.a.local) + min(s.ql, kRows >> p.gsh) - 1 + p.a.sink);
  }
  return static_cast<int>((cnt + kTile - 1) / kTile) + kItemCost;
}

// The last i in [0, n) with arr[i] <= x (arr ascending, arr[0] <= x).
template <class T>
__device__ __forceinline__ int find_last(const T* arr, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (arr[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A line of U places over G blocks: block c has the places [c U / G, (c + 1) U / G).
struct Line {
  int64_t U;
  int G;
  __device__ __forceinline__ int64_t start(int c) const { return c * U / G; }
  __device__ __forceinline__ int block(int64_t x) const { return static_cast<int>(((x + 1) * G - 1) / U); }
};

template <int kNT>
struct Smem {
  static constexpr int kRows = 8 * kNT;
  uint8_t ring[kWarps][kStages][kStage];
  float o[kWarps / 2][kRows][kD + kOutPad];
  float m[kWarps][kRows], l[kWarps][kRows];
  Piece piece[kPieces];
  int64_t place[kMaxSeq + 1];    // places before sequence s
  int32_t item[kMaxSeq + 1];     // items before sequence s
  int shared_out;                // a share behind this block's range was noted
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// c (+)= A (16 x 16, rows) B (16 x 8, columns), fp16 operands.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Token of slot s of an item; -1 behind the last.
template <bool kList>
__device__ __forceinline__ int token_of_slot(const Args& p, const Piece& pc, int s) {
  if (s >= pc.cnt) return -1;
  if (s < pc.head) return s;
  if (!kList) return pc.lo + s - pc.head;
  const int i = s - pc.head;
  if (i >= pc.lo) return p.local_start + i - pc.lo;
  const int64_t list = p.a.sel_per_kv ? static_cast<int64_t>(pc.b) * p.Hkv + pc.g : pc.b;
  const int t = __ldg(p.a.sel + list * p.a.K + i);
  if (t >= 0 && t < p.n) return t;
  record_error(p.err, kErrBadPage);
  return -1;
}

template <bool kList, int kNT>
__device__ __forceinline__ Piece make_piece(const Args& p, const Smem<kNT>& S, const Line& line, int e, int64_t start,
                                            int64_t end) {
  constexpr int kRows = 8 * kNT;
  Piece pc;
  const int b = find_last(S.item, p.B, e);
  const int items = S.item[b + 1] - S.item[b], rem = e - S.item[b];
  const int span = static_cast<int>((S.place[b + 1] - S.place[b]) / items);
  const int64_t x0 = S.place[b] + static_cast<int64_t>(rem) * span;
  const int blocks = items / p.Hkv;
  const Seq s = seq_of<kList>(p, b);
  pc.b = b;
  pc.g = rem / blocks;
  const int r0 = (rem - pc.g * blocks) * kRows;
  pc.rows = static_cast<int>(min(static_cast<int64_t>(kRows), (static_cast<int64_t>(s.ql) << p.gsh) - r0));
  pc.tok0 = s.q0 + (r0 >> p.gsh);
  pc.p0 = s.len - s.ql + (r0 >> p.gsh);
  pc.p1 = s.len - s.ql + ((r0 + pc.rows - 1) >> p.gsh);
  if (kList) {
    pc.head = p.sink_end;
    pc.lo = list_len(p, b, pc.g);
    pc.cnt = p.sink_end + pc.lo + (p.n - p.local_start);
  } else {
    const int64_t lo = static_cast<int64_t>(pc.p0) - p.a.local + 1;
    pc.lo = static_cast<int>(lo > 0 ? lo : 0);
    pc.head = min(p.a.sink, pc.lo);
    pc.cnt = pc.p1 >= 0 ? pc.head + pc.p1 - pc.lo + 1 : 0;
  }
  const int tiles = (pc.cnt + kTile - 1) / kTile;
  const int64_t off = max(start, x0) - x0 - kItemCost, till = min(end, x0 + span) - x0 - kItemCost;
  pc.t0 = static_cast<int>(max(static_cast<int64_t>(0), off));
  pc.n = max(0, static_cast<int>(min(static_cast<int64_t>(tiles), till)) - pc.t0);
  pc.whole = 0;
  pc.slot = 0;
  pc.last = blockIdx.x;
  if (tiles == 0) {
    pc.whole = x0 >= start;   // rows without a token: written by the block that has the item's first place
  } else if (pc.n > 0) {
    const int first = line.block(x0 + kItemCost);
    pc.last = line.block(x0 + kItemCost + tiles - 1);
    pc.whole = first == pc.last;
    pc.slot = first == static_cast<int>(blockIdx.x);
  }
  return pc;
}

template <int kNT, bool kList>
__global__ void __launch_bounds__(kThreads, 1) kv4_attn_kernel(const Args p) {
  using Sm = Smem<kNT>;
  constexpr int kRows = Sm::kRows;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Sm& S = *reinterpret_cast<Sm*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, j = lane & 3;
  pdl_wait();

  // ---- the line
  for (int b = tid; b < p.B; b += kThreads) {
    const Seq s = seq_of<kList>(p, b);
    const int items = items_of<kList, kRows>(p, s);
    S.item[b] = items;
    S.place[b] = items > 0 ? static_cast<int64_t>(items) * span_of<kList, kRows>(p, s, b) : 0;
    if (!kList && blockIdx.x == 0) {
      const int len = __ldg(p.a.bt.lens + b);
      if (len < 0 || len > p.n_cap) record_error(p.err, kErrBadPage);
    }
  }
  if (tid == 0) S.shared_out = 0;
  __syncthreads();
  if (warp == 0) {
    int64_t places = 0;
    int items = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      const int64_t v = b < p.B ? S.place[b] : 0;
      const int w = b < p.B ? S.item[b] : 0;
      int64_t vi = v;
      int wi = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, vi, o);
        const int y = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) {
          vi += x;
          wi += y;
        }
      }
      if (b < p.B) {
        S.place[b] = places + vi - v;
        S.item[b] = items + wi - w;
      }
      places += __shfl_sync(0xffffffffu, vi, 31);
      items += __shfl_sync(0xffffffffu, wi, 31);
    }
    if (lane == 0) {
      S.place[p.B] = places;
      S.item[p.B] = items;
    }
  }
  __syncthreads();
  Line line;
  line.U = S.place[p.B];
  line.G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (line.U + kLeast - 1) / kLeast));
  int64_t start = 0, end = 0;
  int e0 = 0, count = 0;   // first item of the range, items
  if (static_cast<int>(blockIdx.x) < line.G) {
    start = line.start(blockIdx.x);
    end = line.start(blockIdx.x + 1);
    auto item_at = [&](int64_t x) {
      const int b = find_last(S.place, p.B, x);
      const int items = S.item[b + 1] - S.item[b];
      const int64_t span = (S.place[b + 1] - S.place[b]) / items;
      return S.item[b] + static_cast<int>((x - S.place[b]) / span);
    };
    e0 = item_at(start);
    count = item_at(end - 1) - e0 + 1;
  }

  uint8_t* const ring = S.ring[warp][0];
  const uint32_t ring_s = smem_u32(ring);
  for (int i0 = 0; i0 < count; i0 += kPieces) {
    const int np = min(kPieces, count - i0);
    if (tid < np) S.piece[tid] = make_piece<kList, kNT>(p, S, line, e0 + i0 + tid, start, end);
    __syncthreads();

    // ---- loads: the next tile's tokens and their rows are known a tile ahead of
    // their copies each (the block table and the list are read on the way)
    int lp = 0, lt = S.piece[0].t0 + warp;
    int tok = -1, tok_b = 0, tok_g = 0;       // lane's token of the tile after the next
    int row = -1;                             // lane's row of the next tile; -1: none
    bool row_any = false, tok_any = false;
    auto next_tokens = [&]() {
      while (lp < np && lt >= S.piece[lp].t0 + S.piece[lp].n) {
        ++lp;
        if (lp < np) lt = S.piece[lp].t0 + warp;
      }
      tok_any = lp < np;
      tok = -1;
      if (tok_any) {
        const Piece& pc = S.piece[lp];
        tok = token_of_slot<kList>(p, pc, lt * kTile + lane);
        tok_b = pc.b;
        tok_g = pc.g;
        lt += kWarps;
      }
    };
    auto next_rows = [&]() {
      row_any = tok_any;
      row = -1;
      if (tok >= 0) {
        row = static_cast<int>(cache_row(p.a.pm, tok_b, tok_g, p.Hkv, p.n_cap, tok));
        if (row < 0) record_error(p.err, kErrBadPage);
      }
      next_tokens();
    };
    uint32_t put = 0;   // stage that the next copies go to
    auto issue = [&]() {
      if (row_any) {
        const uint32_t at = ring_s + put * kStage;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rk = __shfl_sync(0xffffffffu, row, r + 8 * i);
          // V rows stand with the low bits of their number swapped and their chunks
          // turned by a half where bit 2 is set: a lane's four tokens, 2j and 2j + 1 of
          // eight, are then in banks of their own.
          const int rv = __shfl_sync(0xffffffffu, row, ((r & 4) | (r & 1) << 1 | (r >> 1 & 1)) + 8 * i);
          cp_async16(at + (r + 8 * i) * kKv4Codes + 16 * j, p.a.kv.K + static_cast<int64_t>(max(rk, 0)) * kKv4Codes + 16 * j,
                     rk >= 0 ? 16 : 0);
          cp_async16(at + kTileCodes + kTileScales + (r + 8 * i) * kKv4Codes + 16 * (j ^ (r >> 1 & 2)),
                     p.a.kv.V + static_cast<int64_t>(max(rv, 0)) * kKv4Codes + 16 * j, rv >= 0 ? 16 : 0);
        }
        const int64_t own = static_cast<int64_t>(max(row, 0)) * kKv4Groups;
        cp_async8(at + kTileCodes + lane * kKv4Groups, p.a.kv.K_sf + own, row >= 0 ? 8 : 0);
        cp_async8(at + 2 * kTileCodes + kTileScales + lane * kKv4Groups, p.a.kv.V_sf + own, row >= 0 ? 8 : 0);
      }
      cp_async_commit();
      put = put + 1 == kStages ? 0 : put + 1;
      next_rows();
    };
    next_tokens();
    next_rows();
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue();
    uint32_t take = 0;   // stage of the next tile

    for (int ip = 0; ip < np; ++ip) {
      const Piece pc = S.piece[ip];
      if (pc.n == 0 && !pc.whole) continue;

      // ---- queries: column 8 nt + r of the group's rows; a lane holds 32 values
      uint32_t qf[kNT][16];
      float cs[kNT][2];   // of columns 2j, 2j + 1: logits in log2 units per unit of the product
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const int col = 8 * nt + r;
        uint4 x[4];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = make_uint4(0, 0, 0, 0);
          if (col < pc.rows) {
            const int64_t at = static_cast<int64_t>(pc.tok0 + (col >> p.gsh)) * p.Hq + (pc.g << p.gsh) + (col & ((1 << p.gsh) - 1));
            x[i] = __ldg(reinterpret_cast<const uint4*>(p.a.q + at * kD + 32 * j) + i);
          }
          const uint32_t m = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                      __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
          top = max(top, max(m & 0xffffu, m >> 16));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = min(max(static_cast<int>(top >> 7), 32), 254);   // 2^(ex - 127) <= largest value
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);     // to 2^14 ..
        const float down = __uint_as_float(static_cast<uint32_t>(127 + ex - 141) << 23) * (kScale / kKv4HalfScale) * p.a.kv.k_scale;
        cs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * j);
        cs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * j + 4);
        const uint32_t* w = &x[0].x;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f = bf2_to_f2(w[i]);
          qf[nt][i] = pack_half(f.x * up, f.y * up);
        }
      }

      float o[8][kNT][4];
      float mx[kNT][2], l[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        mx[nt][0] = mx[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
      }

      for (int t = pc.t0 + warp; t < pc.t0 + pc.n; t += kWarps) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        issue();   // into the stage that the tile before this one has left
        const uint8_t* st = ring + take * kStage;
        take = take + 1 == kStages ? 0 : take + 1;

        // ---- S^T = K Q^T
        float s[2][kNT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.0f;
          const int row0 = 16 * mt + r;
          const uint4 k0 = *reinterpret_cast<const uint4*>(st + row0 * kKv4Codes + 16 * j);
          const uint4 k1 = *reinterpret_cast<const uint4*>(st + (row0 + 8) * kKv4Codes + 16 * j);
          const __half2 f0 = kv4_scales(*reinterpret_cast<const uint16_t*>(st + kTileCodes + row0 * kKv4Groups + 2 * j));
          const __half2 f1 = kv4_scales(*reinterpret_cast<const uint16_t*>(st + kTileCodes + (row0 + 8) * kKv4Groups + 2 * j));
          const uint32_t* w0 = &k0.x;
          const uint32_t* w1 = &k1.x;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const __half2 g0 = w < 2 ? __low2half2(f0) : __high2half2(f0), g1 = w < 2 ? __low2half2(f1) : __high2half2(f1);
            __half2 c0[4], c1[4];
            kv4_codes(w0[w], c0);
            kv4_codes(w1[w], c1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = bits(__hmul2(c0[2 * h], g0)), a1 = bits(__hmul2(c1[2 * h], g1));
              const uint32_t a2 = bits(__hmul2(c0[2 * h + 1], g0)), a3 = bits(__hmul2(c1[2 * h + 1], g1));
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt) mma16816(s[mt][nt], a0, a1, a2, a3, qf[nt][4 * w + 2 * h], qf[nt][4 * w + 2 * h + 1]);
            }
          }
        }

        // ---- logits, masked where the tile is not attended to as a whole
        bool full = kTile * (t + 1) <= pc.cnt;
        if (!kList && full && pc.p0 != pc.p1) {
          const int a0 = kTile * t, a1 = a0 + kTile - 1;
          const int first = pc.lo + max(a0, pc.head) - pc.head, last = a1 < pc.head ? a1 : pc.lo + a1 - pc.head;
          full = last <= pc.p0 && (a1 < pc.head || first > pc.p1 - p.a.local);
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][nt][e] *= cs[nt][e & 1];
        if (!full) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int slot = kTile * t + 16 * mt + 8 * h + r;
              const int token = kList ? 0 : (slot < pc.head ? slot : pc.lo + slot - pc.head);
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const int pos = pc.p0 + ((8 * nt + 2 * j + c) >> p.gsh);
                  const bool seen = slot < pc.cnt && (kList || (token <= pos && (token > pos - p.a.local || token < p.a.sink)));
                  if (!seen) s[mt][nt][2 * h + c] = -INFINITY;
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
            top[nt][c] = fmaxf(fmaxf(s[0][nt][c], s[0][nt][2 + c]), fmaxf(s[1][nt][c], s[1][nt][2 + c]));
            grown |= top[nt][c] > mx[nt][c] + kGrow;
          }
        if (__any_sync(0xffffffffu, grown)) {
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
          const float b0 = mx[nt][0] == -INFINITY ? 0.0f : mx[nt][0] - kBase;
          const float b1 = mx[nt][1] == -INFINITY ? 0.0f : mx[nt][1] - kBase;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float p0 = ex2_approx(s[mt][nt][2 * h] - b0), p1 = ex2_approx(s[mt][nt][2 * h + 1] - b1);
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

      // ---- the warps' rows joined
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
          if (r == 0) S.m[warp][8 * nt + 2 * j + c] = mx[nt][c];
        }
      __syncthreads();
      float all[kNT][2], f[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) m = fmaxf(m, S.m[w][8 * nt + 2 * j + c]);
          all[nt][c] = m;
          f[nt][c] = m == -INFINITY ? 1.0f : ex2_approx(mx[nt][c] - m);
          if (r == 0) S.l[warp][8 * nt + 2 * j + c] = l[nt][c] * f[nt][c];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i][nt][c] *= f[nt][c];
            o[i][nt][2 + c] *= f[nt][c];
          }
        }
#pragma unroll
      for (int n = kWarps; n > 1; n = (n + 1) / 2) {
        const int keep = (n + 1) / 2;
        if (warp >= keep && warp < n) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(&S.o[warp - keep][8 * nt + 2 * j + c][16 * r + 4 * i]) =
                    make_float4(o[2 * i][nt][c], o[2 * i][nt][2 + c], o[2 * i + 1][nt][c], o[2 * i + 1][nt][2 + c]);
        }
        __syncthreads();
        if (warp < n - keep) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(&S.o[warp][8 * nt + 2 * j + c][16 * r + 4 * i]);
                o[2 * i][nt][c] += y.x;
                o[2 * i][nt][2 + c] += y.y;
                o[2 * i + 1][nt][c] += y.z;
                o[2 * i + 1][nt][2 + c] += y.w;
              }
        }
        if (n > 2) __syncthreads();
      }
      if (warp == 0) {
        const int64_t part = (static_cast<int64_t>(blockIdx.x) * 2 + pc.slot) * kRows;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = 8 * nt + 2 * j + c;
            if (col >= pc.rows) continue;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += S.l[w][col];
            if (pc.whole) {
              const int64_t at = static_cast<int64_t>(pc.tok0 + (col >> p.gsh)) * p.Hq + (pc.g << p.gsh) + (col & ((1 << p.gsh) - 1));
              const float inv = sum != 0.0f ? p.a.kv.v_scale / kKv4HalfScale / sum : 0.0f;
              uint4* dst = reinterpret_cast<uint4*>(p.a.out + at * kD + 16 * r);
#pragma unroll
              for (int i = 0; i < 2; ++i)
                dst[i] = make_uint4(pack_bf16(o[4 * i][nt][c] * inv, o[4 * i][nt][2 + c] * inv),
                                    pack_bf16(o[4 * i + 1][nt][c] * inv, o[4 * i + 1][nt][2 + c] * inv),
                                    pack_bf16(o[4 * i + 2][nt][c] * inv, o[4 * i + 2][nt][2 + c] * inv),
                                    pack_bf16(o[4 * i + 3][nt][c] * inv, o[4 * i + 3][nt][2 + c] * inv));
              if (p.a.lse && r == 0)
                p.a.lse[at] = sum != 0.0f ? (all[nt][c] == -INFINITY ? sum : (all[nt][c] - kBase + log2f(sum)) * 0.6931471805599453f)
                                          : -INFINITY;
            } else {
              float4* dst = reinterpret_cast<float4*>(p.part_o + (part + col) * kD + 16 * r);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_float4(o[2 * i][nt][c], o[2 * i][nt][2 + c], o[2 * i + 1][nt][c], o[2 * i + 1][nt][2 + c]);
              if (r == 0) p.part_ml[part + col] = make_float2(all[nt][c], sum);
            }
          }
        if (lane == 0 && !pc.whole && pc.slot == 1) {
          Share sh;
          sh.first = (static_cast<int64_t>(pc.tok0) << p.gsh);
          sh.rows = pc.rows;
          sh.g = pc.g;
          sh.last = pc.last;
          sh.pad = 0;
          p.share[blockIdx.x] = sh;
          S.shared_out = 1;
        }
      }
      __syncthreads();   // S.m, S.l and S.o are the next piece's
    }
    __syncthreads();     // the pieces are the next batch's
  }
  if (tid == 0 && S.shared_out == 0 && p.share) p.share[blockIdx.x].rows = 0;
  pdl_trigger();
}

// Joins the parts of an item that several blocks share: exact log-sum-exp,
// fp32.  Block c has the item whose first tiles attention block c had; its
// threads a row's 4 channels each, 8 rows at a time.
constexpr int kMergeThreads = 256;

template <int kNT>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(const Args p) {
  constexpr int kRows = 8 * kNT;
  pdl_wait();
  const Share sh = p.share[blockIdx.x];
  const int chunk = threadIdx.x & 31;
  for (int col = threadIdx.x >> 5; col < sh.rows; col += kMergeThreads / 32) {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = blockIdx.x; c <= sh.last; ++c) {
      const int64_t part = (static_cast<int64_t>(c) * 2 + (c == static_cast<int>(blockIdx.x))) * kRows + col;
      const float2 v = __ldcg(p.part_ml + part);
      const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part_o + part * kD) + chunk);
      const float mn = fmaxf(m, v.x);
      const float a = mn == -INFINITY ? 1.0f : ex2_approx(m - mn), b = mn == -INFINITY ? 1.0f : ex2_approx(v.x - mn);
      m = mn;
      l = l * a + v.y * b;
      o = make_float4(o.x * a + y.x * b, o.y * a + y.y * b, o.z * a + y.z * b, o.w * a + y.w * b);
    }
    const int64_t row = sh.first + col;
    const int64_t at = (row >> p.gsh) * p.Hq + (sh.g << p.gsh) + (row & ((1 << p.gsh) - 1));
    const float inv = l != 0.0f ? p.a.kv.v_scale / kKv4HalfScale / l : 0.0f;
    *reinterpret_cast<uint2*>(p.a.out + at * kD + 4 * chunk) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (p.a.lse && chunk == 0)
      p.a.lse[at] = l != 0.0f ? (m == -INFINITY ? l : (m - kBase + log2f(l)) * 0.6931471805599453f) : -INFINITY;
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
Kernel kernel_of(int nt, bool list) {
  if (nt == 1) return list ? kv4_attn_kernel<1, true> : kv4_attn_kernel<1, false>;
  return kv4_attn_kernel<2, false>;
}
Kernel merge_of(int nt) { return nt == 1 ? kv4_merge_kernel<1> : kv4_merge_kernel<2>; }
size_t smem_of(int nt) { return nt == 1 ? sizeof(Smem<1>) : sizeof(Smem<2>); }
static_assert(sizeof(Smem<2>) <= 232448, "shared memory of a block");

// Columns of an item: single tokens have at most eight.
int tiles_of(const qasc_shape& s, int64_t max_q) { return max_q * (s.Hq / s.Hkv) <= 8 ? 1 : 2; }

}  // namespace

size_t kv4_attn_least_bytes() { return layout_of(16, kMaxSmsForSizing).total; }

size_t kv4_window_workspace_bytes(const qasc_shape& s, int64_t T, int64_t max_q, int32_t sink, int32_t local) {
  (void)s;
  (void)T;
  (void)max_q;
  (void)sink;
  (void)local;
  return kv4_attn_least_bytes();
}

int launch_kv4_attn(const qasc_shape& s, const Kv4AttnArgs& a, uint8_t* ws, size_t ws_bytes, const DeviceInfo& dev,
                    cudaStream_t stream) {
  Args p{};
  p.a = a;
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
  p.err = dev.err_word;
  const int nt = a.listed ? 1 : tiles_of(s, a.max_q);
  const int grid = dev.num_sms;
  const Layout L = layout_of(8 * nt, grid);
  if (ws_bytes < L.total) return static_cast<int>(cudaErrorInvalidValue);
  p.share = reinterpret_cast<Share*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + L.off_ml);
  p.part_o = reinterpret_cast<float*>(ws + L.off_o);
  cudaError_t e = launch_dependent(kernel_of(nt, a.listed), dim3(grid), dim3(kThreads), smem_of(nt), stream, 1, p);
  if (e != cudaSuccess) return static_cast<int>(e);
  e = launch_dependent(merge_of(nt), dim3(grid), dim3(kMergeThreads), 0, stream, 1, p);
  return static_cast<int>(e);
}

cudaError_t configure_kv4_kernels(const DeviceInfo& dev) {
  (void)dev;
  for (int nt = 1; nt <= 2; ++nt)
    for (int list = 0; list < 2; ++list) {
      const cudaError_t e = cudaFuncSetAttribute(kernel_of(nt, list != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem_of(nt)));
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace qasc
