// kv_rope_append: new tokens' keys and values into the cache, keys and
// queries rotated by their positions on the way.
//
// Rotation of a head x by position p, for the pairs (a, b) of its first
// rot_dim values (a = i, b = i + rot_dim / 2, or a = 2i, b = 2i + 1 when
// interleaved):
//   x_a' = x_a cos(p f_i) - x_b sin(p f_i),   x_b' = x_b cos(p f_i) + x_a sin(p f_i)
// in fp32, rounded once to bf16; the values behind rot_dim are copied.
//
// Angles.  p f_i in fp32 would be off by up to half a radian at p = 2^23, so
// the angle is held in turns as a 64-bit fixed-point fraction: F_i =
// frac(f_i / 2 pi) 2^64, and p F_i mod 2^64 is the fraction of a turn exactly,
// whatever the number of whole turns (integer arithmetic wraps where the
// angle does).  F_i comes from one fp64 product, relative error 2^-53: below
// 2^-29 turns at p = 2^24 and f_i <= 1.  The fraction is rounded to fp32 (24 bits
// of at most half a turn) and goes to sincospi.  (The fp64 units of this GPU
// are slow; F_i is computed once per thread and the products are integer.)
//
// Bound: bytes.  Every value is read and written once, (Hq + 2 Hkv) 256 bytes
// each way per token.  32768 tokens of 64 + 8 + 8 heads (1.34 GB): 201 us, 6.68
// TB/s, a plain copy's rate.  What that took: a thread keeps the angles
// of its 16 values in registers over all heads of its slice (no division, no
// shared-memory reads per head), has two heads in flight, and four blocks of
// 256 threads share an SM (five or six spill: 234, 296 us; one head in flight:
// 253; four and two blocks an SM: 223; streaming hints on loads or stores: 203
// to 206).
#include "common.cuh"
#include "internal.h"

namespace qasc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;       // tokens of a block's tile
constexpr int kFreqs = kD / 2;
constexpr int kUnits = 8;        // threads of a head: 16 values each
constexpr int kBatch = 2;        // heads whose loads a thread has in flight

struct AppendArgs {
  const uint16_t* q;       // NULL: no queries
  const uint16_t* k;
  const uint16_t* v;
  int64_t qs, ks, vs;      // values between tokens
  uint16_t* q_out;
  uint16_t* K;
  uint16_t* V;
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&r);
}

// A unit of 16 values of a head, two 16-byte chunks: both members of eight
// pairs (or values that are only copied).  Unit u of a head uses the
// frequencies 8u .. 8u + 7 in either pairing.
__device__ __forceinline__ void rotate_split(uint4& x, uint4& y, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t* xa = &x.x;
  uint32_t* ya = &y.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = bf2_to_f2(xa[i]), b = bf2_to_f2(ya[i]);
    const float c0 = cs[2 * i], c1 = cs[2 * i + 1], s0 = sn[2 * i], s1 = sn[2 * i + 1];
    xa[i] = pack_bf16(a.x * c0 - b.x * s0, a.y * c1 - b.y * s1);
    ya[i] = pack_bf16(b.x * c0 + a.x * s0, b.y * c1 + a.y * s1);
  }
}

template <int F0>
__device__ __forceinline__ void rotate_pairs(uint4& x, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t* xa = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = bf2_to_f2(xa[i]);
    xa[i] = pack_bf16(a.x * cs[F0 + i] - a.y * sn[F0 + i], a.y * cs[F0 + i] + a.x * sn[F0 + i]);
  }
}

__global__ void __launch_bounds__(kThreads, 4) rope_append_kernel(const AppendArgs a) {
  __shared__ float cosv[kMaxTok][kFreqs], sinv[kMaxTok][kFreqs];
  __shared__ int64_t row0[kMaxTok];     // cache row of KV head 0, -1: not written
  __shared__ int32_t rpos[kMaxTok];     // position that rotates
  __shared__ int8_t live[kMaxTok];      // the token belongs to a sequence
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
  uint64_t F = 0;
  if (freq < half) {
    const double turns = static_cast<double>(__ldg(a.inv_freq + freq)) * 0.15915494309189533577;
    const double frac = turns - floor(turns);
    F = frac < 1.0 ? __double2ull_rn(frac * 18446744073709551616.0) : 0;
  }
  const int64_t head_rows = a.pm.table ? (int64_t(1) << a.pm.page_shift) : a.n_cap;   // rows from head to head
  const int nq = a.q ? a.Hq : 0, heads = nq + 2 * a.Hkv;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tok; t0 < a.bt.T; t0 += static_cast<int64_t>(gridDim.x) * a.tok) {
    const int n = static_cast<int>(min(static_cast<int64_t>(a.tok), a.bt.T - t0));
    if (tid < n) {
      const int64_t t = t0 + tid;
      TokenAt at = token_of(a.bt, t);
      live[tid] = at.b >= 0;
      int64_t row = -1;
      if (at.b >= 0) {
        if (at.pos >= 0 && at.pos < a.n_cap) row = cache_row(a.pm, at.b, 0, a.Hkv, a.n_cap, at.pos);
        if (row < 0) record_error(a.err, kErrBadPage);
      }
      row0[tid] = row;
      rpos[tid] = a.positions ? __ldg(a.positions + t) : static_cast<int32_t>(at.pos);
    }
    __syncthreads();
    for (int i = tid; i < n * kFreqs; i += kThreads) {   // i mod 64 = freq: the block is a multiple of 64
      const int tk = i / kFreqs;
      const uint64_t ang = F * static_cast<uint64_t>(static_cast<int64_t>(rpos[tk]));
      float s, c;
      sincospif(static_cast<float>(static_cast<int64_t>(ang)) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
      cosv[tk][freq] = c;
      sinv[tk][freq] = s;
    }
    __syncthreads();
    // thread = (head slice, token, unit): its angles stay in registers over
    // the heads of its slice
    const int u = tid & (kUnits - 1), tk = (tid / kUnits) & (a.tok - 1), slice = tid / (kUnits * a.tok);
    const int step = kThreads / (kUnits * a.tok);
    if (tk < n && live[tk]) {
      const int64_t t = t0 + tk, row = row0[tk];
      const bool turns = u < a.rot / 16;
      float cs[8], sn[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = turns ? cosv[tk][8 * u + i] : 1.0f;
        sn[i] = turns ? sinv[tk][8 * u + i] : 0.0f;
      }
      // chunks of the unit in a rotated head and in a copied one
      const int c0 = turns && !a.interleaved ? u : 2 * u, c1 = turns && !a.interleaved ? u + a.rot / 16 : 2 * u + 1;
      for (int h0 = slice; h0 < heads; h0 += kBatch * step) {
        uint4 x[kBatch], y[kBatch];
        uint16_t* dst[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int h = h0 + i * step;
          dst[i] = nullptr;
          if (h < heads && (h < nq || row >= 0)) {
            const uint16_t* src;
            const bool value = h >= nq + a.Hkv;
            if (h < nq) {
              src = a.q + t * a.qs + h * kD;
              dst[i] = a.q_out + (t * a.Hq + h) * kD;
            } else if (!value) {
              src = a.k + t * a.ks + (h - nq) * kD;
              dst[i] = a.K + (row + (h - nq) * head_rows) * kD;
            } else {
              src = a.v + t * a.vs + (h - nq - a.Hkv) * kD;
              dst[i] = a.V + (row + (h - nq - a.Hkv) * head_rows) * kD;
            }
            x[i] = *reinterpret_cast<const uint4*>(src + 8 * (value ? 2 * u : c0));
            y[i] = *reinterpret_cast<const uint4*>(src + 8 * (value ? 2 * u + 1 : c1));
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (dst[i] == nullptr) continue;
          const bool value = h0 + i * step >= nq + a.Hkv;
          if (turns && !value) {
            if (a.interleaved) {
              rotate_pairs<0>(x[i], cs, sn);
              rotate_pairs<4>(y[i], cs, sn);
            } else {
              rotate_split(x[i], y[i], cs, sn);
            }
          }
          *reinterpret_cast<uint4*>(dst[i] + 8 * (value ? 2 * u : c0)) = x[i];
          *reinterpret_cast<uint4*>(dst[i] + 8 * (value ? 2 * u + 1 : c1)) = y[i];
        }
      }
    }
    __syncthreads();   // the next tile rewrites the angles
  }
  pdl_trigger();
}

}  // namespace

cudaError_t launch_rope_append(const qasc_shape& s, const PageMap& pm, const Batch& bt, const RopeArgs& r,
                               const uint16_t* q, int64_t qs, const uint16_t* k, int64_t ks, const uint16_t* v,
                               int64_t vs, uint16_t* q_out, uint16_t* K, uint16_t* V, const DeviceInfo& dev,
                               cudaStream_t stream) {
  AppendArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qs = qs;
  a.ks = ks;
  a.vs = vs;
  a.q_out = q_out;
  a.K = K;
  a.V = V;
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
  const int64_t most = static_cast<int64_t>(dev.num_sms) * 8;
  return launch_dependent(rope_append_kernel, dim3(static_cast<unsigned>(tiles < most ? tiles : most)), dim3(kThreads), 0,
                          stream, 1, a);
}

}  // namespace qasc
