// kv_window_attn and kv_prefix_attn: causal attention of packed new tokens.
//
//   out[t,h,:] = sum_{j in A(t)} softmax_j(q[t,h].K_j / sqrt(d)) V_j
// with A(t) the sink and the newest `local` tokens up to t's own position, or
// a shared prefix and everything up to t's own position behind it.
//
// One warp per (token, head): lane l holds dimensions 4l .. 4l + 3, the dot
// product of a key is a shuffle sum, and the running maximum, sum and output
// stay in fp32 registers.
#include "common.cuh"
#include "internal.h"

namespace qasc {
namespace {

constexpr int kWarps = 4;

struct Args {
  KvAttnArgs a;
  int Hq, Hkv;
  int64_t n_cap;
  unsigned* err;
};

__global__ void __launch_bounds__(32 * kWarps) kv_attn_rows_kernel(const Args p) {
  const KvAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  pdl_wait();
  if (row >= a.bt.T * p.Hq) return;
  const int64_t t = row / p.Hq;
  const int h = static_cast<int>(row - t * p.Hq), g = h / (p.Hq / p.Hkv);
  const TokenAt at = token_of(a.bt, t);
  if (at.b < 0) return;
  int64_t pos = at.pos;
  if (pos >= p.n_cap) {
    record_error(p.err, kErrBadPage);
    pos = p.n_cap - 1;
  }
  const uint2 qv = *reinterpret_cast<const uint2*>(a.q + row * kD + 4 * lane);
  const float2 q0 = bf2_to_f2(qv.x), q1 = bf2_to_f2(qv.y);
  float M = -INFINITY, L = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
  auto visit = [&](const PageMap& pm, int b, int64_t j) {
    int64_t r = cache_row(pm, b, g, p.Hkv, p.n_cap, j);
    if (r < 0) {
      record_error(p.err, kErrBadPage);
      r = 0;
    }
    const uint2 kv = __ldg(reinterpret_cast<const uint2*>(a.K + r * kD + 4 * lane));
    const uint2 vv = __ldg(reinterpret_cast<const uint2*>(a.V + r * kD + 4 * lane));
    const float2 k0 = bf2_to_f2(kv.x), k1 = bf2_to_f2(kv.y), v0 = bf2_to_f2(vv.x), v1 = bf2_to_f2(vv.y);
    float z = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z *= 0.08838834764831845f;
    const float m = fmaxf(M, z);
    const float al = M == -INFINITY ? 0.0f : expf(M - m);
    const float w = m == -INFINITY ? 0.0f : expf(z - m);
    M = m;
    L = L * al + w;
    o0 = o0 * al + w * v0.x;
    o1 = o1 * al + w * v0.y;
    o2 = o2 * al + w * v1.x;
    o3 = o3 * al + w * v1.y;
  };
  for (int64_t j = 0; j < a.n_prefix; ++j) visit(a.pm_prefix, 0, j);
  const int64_t lo = a.n_prefix > 0 ? 0 : max(static_cast<int64_t>(0), pos - a.local + 1);
  const int64_t head = a.n_prefix > 0 ? 0 : min(static_cast<int64_t>(a.sink), lo);
  for (int64_t j = 0; j < head; ++j) visit(a.pm, at.b, j);
  for (int64_t j = lo; j <= pos; ++j) visit(a.pm, at.b, j);
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  const __nv_bfloat162 y0 = __floats2bfloat162_rn(o0 * inv, o1 * inv), y1 = __floats2bfloat162_rn(o2 * inv, o3 * inv);
  *reinterpret_cast<uint2*>(a.out + row * kD + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
  if (a.lse && lane == 0) a.lse[row] = L > 0.0f ? M + logf(L) : -INFINITY;
}

}  // namespace

size_t kv_attn_workspace_bytes(int64_t, int, int, int, bool, int) { return 256; }

cudaError_t configure_kv_attn_kernels(const DeviceInfo&) { return cudaSuccess; }

int launch_kv_attn(const qasc_shape& s, const KvAttnArgs& a, uint8_t*, const DeviceInfo& dev, cudaStream_t stream) {
  Args p;
  p.a = a;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.n_cap = s.n_cap;
  p.err = dev.err_word;
  const int64_t rows = a.bt.T * s.Hq;
  return launch_dependent(kv_attn_rows_kernel, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)),
                          dim3(32 * kWarps), 0, stream, 1, p);
}

}  // namespace qasc
