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
// each way per token.
#include "common.cuh"
#include "internal.h"

namespace qasc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;       // tokens of a block's tile
constexpr int kFreqs = kD / 2;

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
__device__ __forceinline__ void unit_chunks(int u, int rot, int interleaved, int* c0, int* c1) {
  if (interleaved || u >= rot / 16) {
    *c0 = 2 * u;
    *c1 = 2 * u + 1;
  } else {
    *c0 = u;
    *c1 = u + rot / 16;
  }
}

__device__ __forceinline__ void rotate_split(uint4& x, uint4& y, const float* cs, const float* sn) {
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

__device__ __forceinline__ void rotate_pairs(uint4& x, const float* cs, const float* sn) {
  uint32_t* xa = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = bf2_to_f2(xa[i]);
    xa[i] = pack_bf16(a.x * cs[i] - a.y * sn[i], a.y * cs[i] + a.x * sn[i]);
  }
}

__global__ void __launch_bounds__(kThreads) rope_append_kernel(const AppendArgs a) {
  __shared__ float cosv[kMaxTok][kFreqs], sinv[kMaxTok][kFreqs];
  __shared__ int64_t row0[kMaxTok];     // cache row of KV head 0, -1: not written
  __shared__ int32_t rpos[kMaxTok];     // position that rotates
  __shared__ int8_t live[kMaxTok];      // the token belongs to a sequence
  const int tid = threadIdx.x;
  const int freq = tid & (kFreqs - 1), half = a.rot >> 1;
  pdl_wait();
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
    const int units = n * heads * 8;
    for (int i = tid; i < units; i += kThreads) {
      const int u = i & 7, rest = i >> 3;
      const int tk = rest / heads, h = rest - tk * heads;
      if (!live[tk]) continue;
      const int64_t t = t0 + tk;
      const uint16_t* src;
      uint16_t* dst;
      bool rotated = u < a.rot / 16;
      if (h < nq) {
        src = a.q + t * a.qs + h * kD;
        dst = a.q_out + (t * a.Hq + h) * kD;
      } else {
        if (row0[tk] < 0) continue;
        const int g = h - nq;
        if (g < a.Hkv) {
          src = a.k + t * a.ks + g * kD;
          dst = a.K + (row0[tk] + g * head_rows) * kD;
        } else {
          src = a.v + t * a.vs + (g - a.Hkv) * kD;
          dst = a.V + (row0[tk] + (g - a.Hkv) * head_rows) * kD;
          rotated = false;
        }
      }
      int c0, c1;
      unit_chunks(u, rotated ? a.rot : 0, a.interleaved, &c0, &c1);
      uint4 x = *reinterpret_cast<const uint4*>(src + 8 * c0);
      uint4 y = *reinterpret_cast<const uint4*>(src + 8 * c1);
      if (rotated) {
        const float* cs = &cosv[tk][8 * u];
        const float* sn = &sinv[tk][8 * u];
        if (a.interleaved) {
          rotate_pairs(x, cs, sn);
          rotate_pairs(y, cs + 4, sn + 4);
        } else {
          rotate_split(x, y, cs, sn);
        }
      }
      *reinterpret_cast<uint4*>(dst + 8 * c0) = x;
      *reinterpret_cast<uint4*>(dst + 8 * c1) = y;
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
