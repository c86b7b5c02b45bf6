// kv4_rope_append and kv4_read: new tokens' keys and values into the 4-bit
// cache (kv4.cuh), keys and queries rotated on the way, and cached rows back in
// bf16.
//
// Append.  The rotation is kv_rope_append's (rounded once to bf16; values
// behind rot_dim are copied), and what is quantised is its bf16 result:
//   a = max |x| of 16 values,  scale = e4m3(a / 6),  code = e2m1(x / scale)
// both rounded to nearest, ties to even.  Near the border between two codes
// the smallest error of a rotated key moves its code by a step, so that its
// rotation is computed to 2^-38 and then rounded once.  The angle is a fixed-point number of
// turns, position times the frequency's 96 bits of a turn: good to 2^-63 at every
// position.  cos and sin of an angle come as
// pairs (high, low part), good to 2^-39, from a table of 1024 points of the turn and the
// series of the remainder r < 2^-8:
//   cos(t + r) = C - (S sin r + C (1 - cos r)),  sin(t + r) = S + (C sin r - S (1 - cos r))
// (Knuth's exact sum).  cos and sin are handed on as 16 bits and the rest: products
// of the 16 bits with a bf16 value are exact in fp32.  The queries take the whole cos and
// sin, with fp32's error.
//
// Append's bound: bytes, (2 Hq + 2 Hkv) 256 + 144 Hkv a token.  32768 tokens of 64 + 8 + 8
// heads (1.21 GB): 193 us, 6.3 TB/s, 92 % of a copy's rate; issue slots 66 % (a
// key's rotation and quantising take 9 times a query's instructions).  What that took: a thread's
// units (two 16-byte chunks of a head) are copied into a ring of its own ahead of
// their use, so that the loads go on under a key's arithmetic (245 us with loads a
// loop ahead in registers), queries, keys and values in loops of their own (565 us in
// one, with the angles read from shared memory), no division, one barrier a tile, and 80
// registers (64 spill: 253 us; two blocks of 128 an SM: 199).
//
// Read.  A thread takes two chunks of 8 values of a row, 4 bytes of codes, a scale and
// 16 bytes out each, of two rows at a time; scale * code is exact.  Bound: bytes, 656
// a token and KV head.  131072 tokens, 8 KV heads (688 MB): 108 us, 6.4 TB/s, 94 % of a
// copy's rate; 16 contexts of up to 5003 tokens, 2 KV heads: 11.6 us.  With a
// chunk a thread, four rows at a time: 119 and 12.2.
#include <algorithm>

#include "kv4.cuh"
#include "internal.h"

namespace qasc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;       // tokens of an append block's tile
constexpr int kFreqs = kD / 2;
constexpr int kUnits = 8;        // threads of a head: 16 values each
constexpr int kRing = 4;         // units that a thread's copies are ahead
constexpr size_t kRingBytes = static_cast<size_t>(kThreads) * kRing * 32;
constexpr int kPoints = 256;     // of a quarter turn

struct Points {
  float4 at[kPoints];   // cos and sin of i / 1024 turn: high and low parts
};
constexpr double series_sin(double x) {
  double t = x, s = x;
  for (int k = 1; k < 14; ++k) {
    t *= -x * x / ((2 * k) * (2 * k + 1));
    s += t;
  }
  return s;
}
constexpr double series_cos(double x) {
  double t = 1.0, s = 1.0;
  for (int k = 1; k < 14; ++k) {
    t *= -x * x / ((2 * k - 1) * (2 * k));
    s += t;
  }
  return s;
}
constexpr Points make_points() {
  Points p{};
  for (int i = 0; i < kPoints; ++i) {
    const double x = 6.283185307179586476925 * i / (4 * kPoints);
    const double c = series_cos(x), s = series_sin(x);
    p.at[i].x = static_cast<float>(c);
    p.at[i].y = static_cast<float>(c - static_cast<double>(p.at[i].x));
    p.at[i].z = static_cast<float>(s);
    p.at[i].w = static_cast<float>(s - static_cast<double>(p.at[i].z));
  }
  return p;
}
__device__ constexpr Points g_points = make_points();

struct Pair {
  float h, l;
};

// h + l of a + b exactly (Knuth; l = -0 where there is no rest: its three sums are exact, and
// rounded down a sum of nothing is -0), and with a low part added, renormalised.
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float t = __fadd_rn(a, b), bb = __fadd_rn(t, -a);
  return {t, __fadd_rd(__fadd_rd(a, -__fadd_rn(t, -bb)), __fadd_rd(b, -bb))};
}
__device__ __forceinline__ Pair add_low(Pair t, float low) {
  const float l = __fadd_rn(t.l, low), h = __fadd_rn(t.h, l);
  return {h, __fadd_rn(l, -__fadd_rn(h, -t.h))};
}

// A frequency in turns per position: the 96 bits behind the point, hi and lo.
struct Turns {
  uint64_t hi;
  uint32_t lo;
};
// f / 2 pi: the float's 24 bits times 128 of 1 / 2 pi, shifted by its exponent; good to 2^-96,
// and from a frequency of 2^32 on to 2^-128 of itself.  (One fp64 product is good to 2^-53: at
// position 2^24 that is an angle 2^-29 off, more than a border forgives.)
__device__ __forceinline__ Turns turns_of_frequency(float f) {
  constexpr uint64_t inv_hi = 0x28be60db9391054aull, inv_lo = 0x7f09d5f47d4d3770ull;   // of 2^128 / 2 pi
  const uint32_t u = __float_as_uint(f);
  const int exponent = static_cast<int>(u >> 23 & 255);
  if (exponent == 0 || exponent == 255) return {0, 0};   // less than 2^-128 turns; no number
  const uint64_t m = (u & 0x7fffff) | 0x800000;
  // m / 2 pi: w[0] whole turns, then 64 bits each
  const uint64_t low = __umul64hi(m, inv_lo);
  uint64_t w[3] = {__umul64hi(m, inv_hi), m * inv_hi + low, m * inv_lo};
  w[0] += w[1] < low;
  int right = 150 - exponent;
  if (right < 0) {   // (no frequency of use)
    right += 64;
    if (right <= 0) return {0, 0};
    w[0] = w[1];
    w[1] = w[2];
    w[2] = 0;
  }
  for (; right >= 64; right -= 64) {
    w[2] = w[1];
    w[1] = w[0];
    w[0] = 0;
  }
  if (right > 0) {
    w[2] = w[2] >> right | w[1] << (64 - right);
    w[1] = w[1] >> right | w[0] << (64 - right);
  }
  Turns t{w[1], static_cast<uint32_t>(w[2] >> 32)};
  if (u >> 31) {   // the other way round
    t.hi = ~t.hi + (t.lo == 0);
    t.lo = ~t.lo + 1;
  }
  return t;
}
// The angle at `pos`, in turns times 2^64.
__device__ __forceinline__ uint64_t angle_at(Turns t, int32_t pos) {
  const int64_t n = pos;
  return t.hi * static_cast<uint64_t>(n) + static_cast<uint64_t>((n * static_cast<int64_t>(t.lo)) >> 32);
}

// cos and sin of `ang` / 2^64 turns, to 2^-39.
__device__ __forceinline__ void turn_cos_sin(uint64_t ang, Pair& c, Pair& s) {
  const uint64_t j = (ang + (1ull << 53)) >> 54;
  const int64_t rem = static_cast<int64_t>(ang - (j << 54));       // [-2^53, 2^53)
  const float4 p = __ldg(&g_points.at[j & (kPoints - 1)]);
  Pair C{p.x, p.y}, S{p.z, p.w};
  if (j & kPoints) {   // a quarter turn on: (cos, sin) = (-sin, cos)
    const Pair t = C;
    C = {-S.h, -S.l};
    S = t;
  }
  if (j & (2 * kPoints)) {
    C = {-C.h, -C.l};
    S = {-S.h, -S.l};
  }
  // r = rem 2 pi / 2^64 as rh + rl, from 24 and 24 bits of rem
  const float a = static_cast<float>(static_cast<int32_t>(rem >> 30));
  const float b = static_cast<float>(static_cast<int32_t>((rem & 0x3fffffff) >> 6));
  constexpr double unit = 6.283185307179586476925 / 17179869184.0;
  constexpr float k1 = static_cast<float>(unit), k1l = static_cast<float>(unit - static_cast<double>(k1));
  constexpr float k2 = static_cast<float>(unit / 16777216.0);
  const float rh = __fmul_rn(a, k1);
  const float rl = fmaf(a, k1, -rh) + (a * k1l + b * k2);
  const float r2 = rh * rh;
  const float sl = rl - rh * r2 * 0.16666667f;                     // sin r = rh + sl
  const float v = 0.5f * r2 - r2 * r2 * 0.041666668f + rh * rl;    // 1 - cos r
  const float pc = __fmul_rn(S.h, rh), ec = fmaf(S.h, rh, -pc);
  c = add_low(two_sum(C.h, -pc), C.l - (ec + (S.h * sl + (S.l * rh + C.h * v))));
  const float ps = __fmul_rn(C.h, rh), es = fmaf(C.h, rh, -ps);
  s = add_low(two_sum(S.h, ps), S.l + (es + (C.h * sl + (C.l * rh - S.h * v))));
}

// p1 + p2 + low to 2^-38 of p1 and p2, as what rounds to its bf16 value: where the sum
// in fp32 stands on the middle between two bf16 values the rest decides.  (The low parts are
// summed rounded down: no rest is -0, which leaves a zero the sign of p1 + p2.)
__device__ __forceinline__ float sum_for_bf16(float p1, float p2, float low) {
  const Pair t = two_sum(p1, p2);
  const float l = __fadd_rd(t.l, low), h = __fadd_rn(t.h, l), rest = __fadd_rn(l, -__fadd_rn(h, -t.h));
  int u = __float_as_int(h);
  const int away = ((u ^ __float_as_int(rest)) >> 31) | 1;   // 1: the rest has the sum's sign
  if ((u & 0xffff) == 0x8000 && rest != 0.0f) u += away;
  return t.l == t.l ? __int_as_float(u) : t.h;   // (an infinity leaves no exact rest)
}

// The pair (a, b) rotated.  c and s are the high parts, of 16 bits, so that their
// products with a bf16 value are exact in fp32, cl and sl the rest.
__device__ __forceinline__ void rotate_exactly(float& a, float& b, float c, float s, float cl, float sl) {
  const float x = sum_for_bf16(__fmul_rn(a, c), -__fmul_rn(b, s), fmaf(a, cl, -__fmul_rn(b, sl)));
  b = sum_for_bf16(__fmul_rn(b, c), __fmul_rn(a, s), fmaf(b, cl, __fmul_rn(a, sl)));
  a = x;
}

struct AppendArgs {
  const uint16_t* q;       // NULL: no queries
  const uint16_t* k;
  const uint16_t* v;
  int64_t qs, ks, vs;      // values between tokens
  uint16_t* q_out;
  Kv4Cache kv;
  float k_inv, v_inv;      // 1 / the cache's factors
  const float* inv_freq;
  const int32_t* positions;
  int rot, interleaved;
  PageMap pm;
  Batch bt;
  int Hq, Hkv;
  int64_t n_cap;
  int tok;                 // tokens per tile
  unsigned* err;
};

// Largest magnitude of eight bf16 values, as bits (those of a NaN are above all others).
__device__ __forceinline__ uint32_t abs_max(const uint4& x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// Codes of eight values, `f` what turns them into quotients.
__device__ __forceinline__ uint32_t codes_of(const uint4& x, float f) {
  const uint32_t* w = &x.x;
  float q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = bf2_to_f2(w[i]);
    q[2 * i] = kv4_quotient(v.x * f);
    q[2 * i + 1] = kv4_quotient(v.y * f);
  }
  return kv4_pack(q);
}

// A unit's two chunks of a head, cx and cy, quantised into row r.  Each of them is
// half of a group of 16; px and py are their other halves: whose lane they are on
// and whether they are its second chunk.
struct Halves {
  int lane;
  bool second;
};
__device__ __forceinline__ void store_quantised(const uint4& x, const uint4& y, int cx, int cy, bool together, Halves px, Halves py,
                                                float inv, uint8_t* codes, uint8_t* sf, unsigned unit_mask, bool first) {
  uint32_t mx = abs_max(x), my = abs_max(y);
  if (together) {
    mx = my = max(mx, my);
  } else {
    const uint32_t xx = __shfl_sync(unit_mask, mx, px.lane), xy = __shfl_sync(unit_mask, my, px.lane);
    const uint32_t yx = __shfl_sync(unit_mask, mx, py.lane), yy = __shfl_sync(unit_mask, my, py.lane);
    mx = max(mx, px.second ? xy : xx);
    my = max(my, py.second ? yy : yx);
  }
  const uint32_t sx = kv4_scale_of(__uint_as_float(mx << 16) * inv), sy = kv4_scale_of(__uint_as_float(my << 16) * inv);
  *reinterpret_cast<uint32_t*>(codes + 4 * cx) = codes_of(x, kv4_divisor(sx) * inv);
  *reinterpret_cast<uint32_t*>(codes + 4 * cy) = codes_of(y, kv4_divisor(sy) * inv);
  // the row's eight scales, gathered from its eight threads
  const int gx = 8 * (cx >> 1), gy = 8 * (cy >> 1);
  const uint32_t lo = __reduce_or_sync(unit_mask, (gx < 32 ? sx << gx : 0u) | (gy < 32 ? sy << gy : 0u));
  const uint32_t hi = __reduce_or_sync(unit_mask, (gx < 32 ? 0u : sx << (gx - 32)) | (gy < 32 ? 0u : sy << (gy - 32)));
  if (first) *reinterpret_cast<uint2*>(sf) = make_uint2(lo, hi);
}

// A unit of a head is 16 values in two 16-byte chunks: both members of eight
// pairs, or values that are only copied; unit u of a head uses the frequencies
// 8u .. 8u + 7 in either pairing.
__global__ void __launch_bounds__(kThreads, 3) kv4_append_kernel(const AppendArgs a) {
  // of this tile and the next one, which is prepared ahead: one barrier a tile
  __shared__ __align__(16) float turns_of[2][4][kMaxTok][kFreqs];   // cos, sin (16 bits) and their rests
  __shared__ int64_t rows_of[2][kMaxTok];    // cache row of KV head 0; -1: not written, -2: a token of no sequence
  __shared__ Turns turns_at[kThreads];       // each thread's own (as registers they would spill)
  const int tid = threadIdx.x;
  const int freq = tid & (kFreqs - 1), half = a.rot >> 1;
  pdl_wait();
  // Lengths outside the cache are recorded, of sequences without new tokens as
  // well (the first warp, whose loads the block waits for, has no part in it).
  if (tid >= 32)
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * (kThreads - 32) + tid - 32; b < a.bt.B;
         b += static_cast<int64_t>(gridDim.x) * (kThreads - 32)) {
      const int len = __ldg(a.bt.lens + b);
      if (len < 0 || len > a.n_cap) record_error(a.err, kErrBadPage);
    }
  if (freq < half) turns_at[tid] = turns_of_frequency(__ldg(a.inv_freq + freq));
  const int64_t head_rows = a.pm.table ? (int64_t(1) << a.pm.page_shift) : a.n_cap;   // rows from head to head
  const int nq = a.q ? a.Hq : 0;
  const unsigned unit_mask = 0xffu << (tid & 24);
  // A thread has the angle of one frequency of a token.
  auto prepare = [&](int64_t t0, int buf) {
    const int tk = tid / kFreqs;   // kThreads / kFreqs = kMaxTok
    if (tk >= a.tok || t0 + tk >= a.bt.T) return;
    const int64_t t = t0 + tk;
    const TokenAt at = token_of(a.bt, t);
    if (freq == 0) {
      int64_t row = -2;
      if (at.b >= 0) {
        row = -1;
        if (at.pos >= 0 && at.pos < a.n_cap) row = cache_row(a.pm, at.b, 0, a.Hkv, a.n_cap, at.pos);
        if (row < 0) record_error(a.err, kErrBadPage);
      }
      rows_of[buf][tk] = row;
    }
    if (freq < half) {
      const int32_t pos = a.positions ? __ldg(a.positions + t) : static_cast<int32_t>(at.pos);
      Pair c, s;
      turn_cos_sin(angle_at(turns_at[tid], pos), c, s);
      const float ch = __uint_as_float(__float_as_uint(c.h) & 0xffffff00u), sh = __uint_as_float(__float_as_uint(s.h) & 0xffffff00u);
      turns_of[buf][0][tk][freq] = ch;
      turns_of[buf][1][tk][freq] = sh;
      turns_of[buf][2][tk][freq] = __fadd_rn(__fadd_rn(c.h, -ch), c.l);
      turns_of[buf][3][tk][freq] = __fadd_rn(__fadd_rn(s.h, -sh), s.l);
    }
  };
  // A thread's units: of every tile its slice's heads of queries, then of keys and
  // values in turn, two 16-byte chunks of each.  They are copied into a ring of its own
  // ahead of their use, from tile to tile, whatever the unit at hand costs.
  const int u = tid & (kUnits - 1), tk = (tid / kUnits) & (a.tok - 1), slice = tid / (kUnits * a.tok);
  const int step = kThreads / (kUnits * a.tok);
  const int q_units = (nq + step - 1) / step, units = q_units + 2 * ((a.Hkv + step - 1) / step);
  const int r16 = a.rot / 16;
  const bool turns = u < r16;
  // chunks of the unit in a rotated head and in a copied one
  const int c0 = turns && !a.interleaved ? u : 2 * u, c1 = turns && !a.interleaved ? u + r16 : 2 * u + 1;
  // the lane, and which of its chunks, that holds chunk c of a rotated head
  auto holder = [&](int c) {
    const bool pairs = a.interleaved || c >= 2 * r16;
    return Halves{(tid & 24) + (pairs ? c >> 1 : (c < r16 ? c : c - r16)), pairs ? (c & 1) != 0 : c >= r16};
  };
  const Halves px = holder(c0 ^ 1), py = holder(c1 ^ 1);
  const int64_t t_step = static_cast<int64_t>(gridDim.x) * a.tok;
  extern __shared__ __align__(16) uint4 ring_of[];
  uint4* const ring = ring_of + (tid / 32) * (kRing * 64) + (tid & 31);
  // the next unit to copy: its token's rows, the unit
  int64_t load_t = static_cast<int64_t>(blockIdx.x) * a.tok + tk;
  const int head0 = slice * kD;
  const uint16_t *load_q = a.q + load_t * a.qs + head0 + 8 * c0, *load_k = a.k + load_t * a.ks + head0 + 8 * c0,
                 *load_v = a.v + load_t * a.vs + head0 + 16 * u;
  const int apart = 8 * (c1 - c0);   // values from chunk to chunk
  const uint32_t ring_s = smem_u32(ring);
  int unit = 0, load_place = 0, place = 0;
  auto load = [&]() {
    const uint32_t to = ring_s + load_place * 1024;
    if (load_t < a.bt.T) {
      if (unit < q_units) {
        if (slice + unit * step < nq) {
          const uint16_t* src = load_q + unit * step * kD;
          cp_async16(to, src);
          cp_async16(to + 512, src + apart);
        }
      } else {
        const int i = unit - q_units, h = (i >> 1) * step;
        if (slice + h < a.Hkv) {
          const uint16_t* src = ((i & 1) ? load_v : load_k) + h * kD;
          cp_async16(to, src);
          cp_async16(to + 512, src + ((i & 1) ? 8 : apart));
        }
      }
      if (++unit == units) {
        unit = 0;
        load_t += t_step;
        load_q += t_step * a.qs;
        load_k += t_step * a.ks;
        load_v += t_step * a.vs;
      }
    }
    cp_async_commit();
    load_place = load_place + 1 == kRing ? 0 : load_place + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) load();
  int buf = 0;
  prepare(static_cast<int64_t>(blockIdx.x) * a.tok, 0);
  __syncthreads();
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tok; t0 < a.bt.T; t0 += t_step, buf ^= 1) {
    const int n = static_cast<int>(min(static_cast<int64_t>(a.tok), a.bt.T - t0));
    if (t0 + t_step < a.bt.T) prepare(t0 + t_step, buf ^ 1);
    const float (&turn)[4][kMaxTok][kFreqs] = turns_of[buf];
    const int64_t* row0 = rows_of[buf];
    const int64_t t = t0 + tk, row = tk < n ? row0[tk] : -2;
    // the unit just arrived, and its place for the one after the next kRing - 1
    auto take = [&](uint4& x, uint4& y) {
      cp_async_wait<kRing - 1>();
      const uint4* from = ring + place * 64;   // what this lane has copied itself
      x = from[0];
      y = from[32];
      load();
      place = place + 1 == kRing ? 0 : place + 1;
    };
    auto angles = [&](int i, float (&v)[8]) {
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(&turn[i][tk][8 * u]);
      *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(&turn[i][tk][8 * u + 4]);
    };
    if (nq > 0) {
      float cs[8], sn[8], cl[8], sl[8];
      angles(0, cs);
      angles(1, sn);
      angles(2, cl);
      angles(3, sl);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] += cl[i];
        sn[i] += sl[i];
      }
      uint16_t* dst = a.q_out + (t * a.Hq + slice) * kD + 8 * c0;
#pragma unroll 1
      for (int h = slice; h < q_units * step + slice; h += step, dst += step * kD) {
        uint4 x, y;
        take(x, y);
        if (h >= nq || row == -2) continue;
        uint32_t* xa = &x.x;
        uint32_t* ya = &y.x;
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = bf2_to_f2(xa[e]), g = bf2_to_f2(ya[e]);
            if (a.interleaved) {
              xa[e] = pack_bf16(f.x * cs[e] - f.y * sn[e], f.y * cs[e] + f.x * sn[e]);
              ya[e] = pack_bf16(g.x * cs[4 + e] - g.y * sn[4 + e], g.y * cs[4 + e] + g.x * sn[4 + e]);
            } else {
              xa[e] = pack_bf16(f.x * cs[2 * e] - g.x * sn[2 * e], f.y * cs[2 * e + 1] - g.y * sn[2 * e + 1]);
              ya[e] = pack_bf16(g.x * cs[2 * e] + f.x * sn[2 * e], g.y * cs[2 * e + 1] + f.y * sn[2 * e + 1]);
            }
          }
        }
        *reinterpret_cast<uint4*>(dst) = x;
        *reinterpret_cast<uint4*>(dst + apart) = y;
      }
    }
#pragma unroll 1
    for (int k = q_units; k < units; k += 2) {
      const int h = slice + ((k - q_units) >> 1) * step;
      const bool mine = h < a.Hkv && row >= 0;
      const int64_t r = row + h * head_rows;
      uint4 x, y;
      take(x, y);
      if (mine) {
        if (turns) {
          float c[8], sx[8], cl[8], sl[8];
          angles(0, c);
          angles(1, sx);
          angles(2, cl);
          angles(3, sl);
          uint32_t* xa = &x.x;
          uint32_t* ya = &y.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 f = bf2_to_f2(xa[e]), g = bf2_to_f2(ya[e]);
            if (a.interleaved) {
              rotate_exactly(f.x, f.y, c[e], sx[e], cl[e], sl[e]);
              rotate_exactly(g.x, g.y, c[4 + e], sx[4 + e], cl[4 + e], sl[4 + e]);
            } else {
              rotate_exactly(f.x, g.x, c[2 * e], sx[2 * e], cl[2 * e], sl[2 * e]);
              rotate_exactly(f.y, g.y, c[2 * e + 1], sx[2 * e + 1], cl[2 * e + 1], sl[2 * e + 1]);
            }
            xa[e] = pack_bf16(f.x, f.y);
            ya[e] = pack_bf16(g.x, g.y);
          }
        }
        store_quantised(x, y, c0, c1, a.interleaved != 0, px, py, a.k_inv, a.kv.K + r * kKv4Codes, a.kv.K_sf + r * kKv4Groups,
                        unit_mask, u == 0);
      }
      take(x, y);
      if (mine)
        store_quantised(x, y, 2 * u, 2 * u + 1, true, px, py, a.v_inv, a.kv.V + r * kKv4Codes, a.kv.V_sf + r * kKv4Groups,
                        unit_mask, u == 0);
    }
    __syncthreads();   // the next tile is ready, and this one's place free
  }
  pdl_trigger();
}

constexpr int kReadTok = 32;     // tokens of a read block's tile
constexpr int kRowLanes = 8;     // threads of a row: chunks c and c + 8 of 8 values each
static_assert(kThreads / kRowLanes == kReadTok, "a pass has a row of every token of the tile");
constexpr int kReadBlocks = 6;   // blocks of an SM
constexpr int kReadBatch = 2;     // rows whose loads a thread has in flight

struct ReadArgs {
  Kv4Cache kv;
  uint16_t* K_out;
  uint16_t* V_out;
  int64_t k_token, k_head, v_token, v_head;   // values between tokens and heads of the outputs
  PageMap pm;
  Batch bt;
  int Hkv;
  int64_t n_cap;
  unsigned* err;
};

// The tile's rows in bf16: token i's row of KV head 0 is row0[i] (-1: rows of zeros
// where `zeros` is -1, none written otherwise; -2: none written), strides of the
// outputs in values.
__device__ __forceinline__ void read_rows(const Kv4Cache& kv, int Hkv, const int64_t* row0, int64_t head_rows, uint16_t* K_out,
                                          int64_t k_token, int64_t k_head, uint16_t* V_out, int64_t v_token, int64_t v_head,
                                          int zeros) {
  const int c = threadIdx.x & (kRowLanes - 1), tk = threadIdx.x / kRowLanes;
  const int64_t row = row0[tk];
  if (row < zeros) return;
  const bool there = row >= 0;
  // keys and values of a head in turn
  const int64_t from = max(row, int64_t(0));
  for (int i0 = 0; i0 < 2 * Hkv; i0 += kReadBatch) {
    uint32_t w[kReadBatch][2], sf[kReadBatch][2];
#pragma unroll
    for (int k = 0; k < kReadBatch; ++k) {
      const int side = k & 1, g = (i0 + k) >> 1;
      w[k][0] = w[k][1] = sf[k][0] = sf[k][1] = 0;
      if (there && i0 + k < 2 * Hkv) {
        const int64_t r = from + g * head_rows;
        const uint32_t* codes = reinterpret_cast<const uint32_t*>((side ? kv.V : kv.K) + r * kKv4Codes) + c;
        const uint8_t* scales = (side ? kv.V_sf : kv.K_sf) + r * kKv4Groups + (c >> 1);
        w[k][0] = __ldg(codes);
        w[k][1] = __ldg(codes + 8);
        sf[k][0] = __ldg(scales);
        sf[k][1] = __ldg(scales + 4);
      }
    }
#pragma unroll
    for (int k = 0; k < kReadBatch; ++k) {
      const int side = k & 1, g = (i0 + k) >> 1;
      if (i0 + k >= 2 * Hkv) continue;
      const float f = side ? kv.v_scale : kv.k_scale;
      uint16_t* dst = (side ? V_out + tk * v_token + g * v_head : K_out + tk * k_token + g * k_head) + 8 * c;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const __half2 s = kv4_scales(sf[k][half] * 0x101u);
        __half2 h[4];
        kv4_codes(w[k][half], h);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = __half22float2(__hmul2(h[e], s));
          o[e] = pack_bf16(v.x * f, v.y * f);
        }
        *reinterpret_cast<uint4*>(dst + 64 * half) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, kReadBlocks) kv4_read_kernel(const ReadArgs a) {
  __shared__ int64_t row0[kReadTok];
  const int tid = threadIdx.x;
  pdl_wait();
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kThreads + tid; b < a.bt.B; b += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int len = __ldg(a.bt.lens + b);
    if (len < 0 || len > a.n_cap) record_error(a.err, kErrBadPage);
  }
  const int64_t head_rows = a.pm.table ? (int64_t(1) << a.pm.page_shift) : a.n_cap;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kReadTok;
  if (tid < kReadTok) {
    int64_t row = -1;
    if (t0 + tid < a.bt.T) {
      const TokenAt at = token_of(a.bt, t0 + tid);
      if (at.b >= 0) {
        if (at.pos >= 0 && at.pos < a.n_cap) row = cache_row(a.pm, at.b, 0, a.Hkv, a.n_cap, at.pos);
        if (row < 0) record_error(a.err, kErrBadPage);
      }
    }
    row0[tid] = row;
  }
  __syncthreads();
  read_rows(a.kv, a.Hkv, row0, head_rows, a.K_out + t0 * a.k_token, a.k_token, a.k_head, a.V_out + t0 * a.v_token, a.v_token,
            a.v_head, 0);
  pdl_trigger();
}

// ---- the bf16 copy that long sequences of a window call attend to
struct CopyArgs {
  Kv4Cache kv;
  Kv4Copy c;
  PageMap pm;
  Batch bt;
  int B, Hkv, gsh;
  int32_t sink, local;
  int64_t n_cap;
  unsigned* err;
};

constexpr int kCopySeq = 2048;
constexpr size_t kCopyShared = 216 << 10;   // of an SM, for the blocks that it may have
constexpr size_t kCopyStatic = 10 << 10;    // of a block beside what it asks for, at least

// Every block makes the plan for itself: which sequences are copied and their
// first pages (sequences take pages in their order as long as all of theirs
// are left); block 0 writes it down.  Then tiles of kReadTok tokens.
__global__ void __launch_bounds__(kThreads, kReadBlocks) kv4_copy_kernel(const CopyArgs a) {
  __shared__ int64_t row0[kReadTok];
  __shared__ int32_t first[kCopySeq + 1];
  __shared__ int32_t sums[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!a.c.beside) pdl_wait();   // (beside: see Kv4Copy)
  auto shape_of = [&](int b, int* drop) {   // tokens of the copy and those left out behind the sink; 0: not copied
    const int64_t q0 = min(max(a.bt.cu_q ? __ldg(a.bt.cu_q + b) : static_cast<int64_t>(b), int64_t(0)), a.bt.T);
    const int64_t q1 = min(max(a.bt.cu_q ? __ldg(a.bt.cu_q + b + 1) : static_cast<int64_t>(b) + 1, q0), a.bt.T);
    const int64_t len = min(max(static_cast<int64_t>(__ldg(a.bt.lens + b)), int64_t(0)), a.n_cap);
    if (((q1 - q0) << a.gsh) <= a.c.most_rows) return 0;
    const int tokens = kv4_tokens_seen(len, q1 - q0, a.sink, a.local, drop);
    return tokens <= a.c.pages_per_seq * kCopyPage ? tokens : 0;   // (0: more new tokens than the call said)
  };
  int taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int drop = 0;
    const int tokens = b < a.B ? shape_of(b, &drop) : 0, pages = (tokens + kCopyPage - 1) / kCopyPage;
    int inc = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += w;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int before = taken + inc - pages, total = taken;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    if (b < a.B) {
      first[b] = before;
      if (blockIdx.x == 0) {
        // Offsets that do not ascend make more long sequences than there is room for, and rows that the
        // attention over the copy holds for two of them.
        if (a.bt.cu_q && min(max(__ldg(a.bt.cu_q + b), 0), static_cast<int>(a.bt.T)) > max(__ldg(a.bt.cu_q + b + 1), 0))
          record_error(a.err, kErrBadPage);
        const bool fits = pages > 0 && before + pages <= a.c.capacity;
        a.c.copied[b] = fits;
        a.c.lens[b] = fits ? tokens : 0;
      }
    }
    taken = total;
    __syncthreads();
  }
  const int64_t head_rows = a.pm.table ? (int64_t(1) << a.pm.page_shift) : a.n_cap;
  constexpr int kParts = kCopyPage / kReadTok;
  const int tiles = static_cast<int>(min(static_cast<int64_t>(taken), a.c.capacity)) * kParts;
  for (int i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int page = i / kParts, part = i - page * kParts;
    int lo = 0, hi = a.B;   // the last sequence whose pages begin at or before this one: those of none stand before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= page) lo = mid;
      else hi = mid;
    }
    int drop = 0;
    const int tokens = shape_of(lo, &drop), pages = (tokens + kCopyPage - 1) / kCopyPage;
    if (first[lo] + pages > a.c.capacity) continue;   // the whole block: it has not got all of its pages
    const int at = (page - first[lo]) * kCopyPage + part * kReadTok;
    __syncthreads();
    if (tid < kReadTok) {
      int64_t row = -2;   // behind the last token: not written
      if (at + tid < tokens) {
        const int t = at + tid < a.sink ? at + tid : at + tid + drop;
        row = cache_row(a.pm, lo, 0, a.Hkv, a.n_cap, t);
        if (row < 0) record_error(a.err, kErrBadPage);   // rows of zeros
      }
      row0[tid] = row;
    }
    if (part == 0 && tid == 0) a.c.table[lo * a.c.pages_per_seq + page - first[lo]] = page;
    __syncthreads();
    const int64_t to = (static_cast<int64_t>(page) * a.Hkv * kCopyPage + part * kReadTok) * kD;
    read_rows(a.kv, a.Hkv, row0, head_rows, a.c.K + to, kD, static_cast<int64_t>(kCopyPage) * kD, a.c.V + to, kD,
              static_cast<int64_t>(kCopyPage) * kD, -1);
  }
  pdl_trigger();
  if (a.c.beside) pdl_wait();   // so that what waits for this kernel waits for the one before as well
}

}  // namespace

cudaError_t launch_kv4_append(const qasc_shape& s, const PageMap& pm, const Batch& bt, const RopeArgs& r,
                              const uint16_t* q, int64_t qs, const uint16_t* k, int64_t ks, const uint16_t* v,
                              int64_t vs, uint16_t* q_out, const Kv4Cache& kv, const DeviceInfo& dev,
                              cudaStream_t stream) {
  AppendArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = qs;
  a.ks = ks;
  a.vs = vs;
  a.q_out = q_out;
  a.kv = kv;
  a.k_inv = 1.0f / kv.k_scale;
  a.v_inv = 1.0f / kv.v_scale;
  a.inv_freq = r.inv_freq;
  a.positions = r.positions;
  a.rot = r.rot_dim;
  a.interleaved = r.interleaved;
  a.pm = pm;
  a.bt = bt;
  a.Hq = s.Hq;
  a.Hkv = s.Hkv;
  a.n_cap = s.n_cap;
  a.err = dev.err_word;
  // Tiles of four tokens fill the block's 256 threads with angles; few tokens
  // go one to a block, over more SMs.
  a.tok = bt.T >= 4 * dev.num_sms ? kMaxTok : 1;
  const int64_t tiles = (bt.T + a.tok - 1) / a.tok;
  const int64_t most = static_cast<int64_t>(dev.num_sms) * 12;
  return launch_dependent(kv4_append_kernel, dim3(static_cast<unsigned>(tiles < most ? tiles : most)), dim3(kThreads),
                          kRingBytes, stream, 1, a);
}

cudaError_t configure_kv4_cache_kernels(const DeviceInfo& dev) {
  (void)dev;
  const cudaError_t e = cudaFuncSetAttribute(kv4_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kCopyShared - kCopyStatic));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kv4_append_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes));
}

cudaError_t launch_kv4_read(const qasc_shape& s, const PageMap& pm, const Batch& bt, const Kv4Cache& kv, uint16_t* K_out,
                            int64_t k_token, int64_t k_head, uint16_t* V_out, int64_t v_token, int64_t v_head,
                            const DeviceInfo& dev, cudaStream_t stream) {
  ReadArgs a;
  a.kv = kv;
  a.K_out = K_out;
  a.V_out = V_out;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_token = v_token;
  a.v_head = v_head;
  a.pm = pm;
  a.bt = bt;
  a.Hkv = s.Hkv;
  a.n_cap = s.n_cap;
  a.err = dev.err_word;
  // a block a tile, so that the device shares them out (six tiles' blocks an SM, each
  // with every 912th tile: 115 us for 131072 tokens, 108 so)
  const int64_t tiles = (bt.T + kReadTok - 1) / kReadTok;
  return launch_dependent(kv4_read_kernel, dim3(static_cast<unsigned>(tiles)), dim3(kThreads), 0, stream, 1, a);
}

cudaError_t launch_kv4_copy(const qasc_shape& s, const PageMap& pm, const Batch& bt, const Kv4Cache& kv, int32_t sink,
                            int32_t local, const Kv4Copy& c, const DeviceInfo& dev, cudaStream_t stream) {
  CopyArgs a{};
  a.kv = kv;
  a.c = c;
  a.pm = pm;
  a.bt = bt;
  a.B = s.B;
  a.Hkv = s.Hkv;
  while ((1 << a.gsh) < s.Hq / s.Hkv) ++a.gsh;
  a.sink = sink;
  a.local = local;
  a.n_cap = s.n_cap;
  a.err = dev.err_word;
  // Beside another kernel blocks go where there is room first, and those with work, the first
  // ones, were all on few SMs (512 tokens of 8 heads, 16 blocks: 34 us with the attention, 25
  // spread out): so a block asks for as much shared memory as leaves none on an SM for more
  // than its share of them, and of a third more, which ragged batches may have (16 of
  // 1 to 257 new tokens: 31 us, 34 without that).
  constexpr int kParts = kCopyPage / kReadTok;
  const int64_t sms = dev.num_sms, tiles = c.capacity * kParts;
  const int64_t share = c.beside ? std::min<int64_t>(kReadBlocks, (c.likely * kParts * 4 / 3 + sms - 1) / sms) : kReadBlocks;
  const int64_t grid = std::min(tiles, sms * share);
  return launch_dependent(kv4_copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                          c.beside ? kCopyShared / static_cast<size_t>(share) - kCopyStatic : 0, stream, 1, a);
}

}  // namespace qasc
