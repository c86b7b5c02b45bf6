// Host-side interfaces between the C-ABI layer (api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "qasc.h"

namespace qasc {

// Launches `kernel` as a programmatic dependent of the preceding kernel in
// the stream (see pdl_wait / pdl_trigger), optionally as clusters of
// `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             unsigned cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  unsigned n = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    n = 2;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

constexpr int kHeadDim = 128;
constexpr int kIndexDim = 32;
// Workspace queries made without a device size split-K scratch for this many
// SMs, an upper bound for any device the library runs on.
constexpr int kMaxSmsForSizing = 256;

// Token regions of a cache of n tokens (TokenSelect page, table of
// always-included tokens): sink [0, sink_end), candidates C [c0, c1),
// local [local_start, n).
struct Regions {
  int64_t sink_end, c0, c1, local_start;
  int64_t nc() const { return c1 - c0; }
};

// Where the rows of token t of (b, g) live.  Contiguous (table == nullptr):
// row (b Hkv + g) n_cap + t of a [B][Hkv][n_cap] cache.  Paged: row
// (page Hkv + g) P + t mod P of a [num_pages][Hkv][P] pool, page =
// table[b][t / P] (P = 2^page_shift).
struct PageMap {
  const int32_t* table = nullptr;   // [B][pages_per_seq]
  int64_t pages_per_seq = 0, num_pages = 0;
  int page_shift = 0;
};

// Circular local buffer: K and V rows of token t of (b, g) at slot t mod R
// of [B][Hkv][R][d] (K == nullptr: none).
struct RingMap {
  const uint16_t* K = nullptr;
  const uint16_t* V = nullptr;
  int64_t R = 0;
};

// The new tokens of a batch, packed: sequence b has tokens
// [cu_q[b], cu_q[b + 1]) of T (one token each when cu_q is NULL) and lens[b]
// cached tokens, its new ones the last of them.
struct Batch {
  const int32_t* cu_q = nullptr;
  const int32_t* lens = nullptr;
  int64_t T = 0;
  int B = 0;
};

// Rotation of keys and queries: frequencies of the rot_dim / 2 pairs, and the
// positions that rotate (NULL: the cache positions).
struct RopeArgs {
  const float* inv_freq = nullptr;
  const int32_t* positions = nullptr;
  int rot_dim = 0, interleaved = 0;
};

#ifdef __CUDACC__
// Sequence and cache position of packed token t; b < 0: the token belongs to
// no sequence (it lies outside [cu_q[0], cu_q[B])).
struct TokenAt {
  int b;
  int64_t pos;
};
__device__ __forceinline__ TokenAt token_of(const Batch& bt, int64_t t) {
  TokenAt r;
  if (bt.cu_q == nullptr) {
    r.b = static_cast<int>(t);
    r.pos = static_cast<int64_t>(__ldg(bt.lens + t)) - 1;
    return r;
  }
  int lo = 0, hi = bt.B;   // the last b with cu_q[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(bt.cu_q + mid) <= t) lo = mid;
    else hi = mid;
  }
  int64_t q0 = __ldg(bt.cu_q + lo), q1 = __ldg(bt.cu_q + lo + 1);
  if (q1 > bt.T) q1 = bt.T;   // clamped, as the attention calls do
  r.b = t >= q0 && t < q1 ? lo : -1;
  r.pos = static_cast<int64_t>(__ldg(bt.lens + lo)) - (q1 - t);
  return r;
}

// Row of token t of (b, g) under m, or -1 when its block-table entry lies
// outside the pool.
__device__ __forceinline__ int64_t cache_row(const PageMap& m, int b, int g, int Hkv, int64_t n_cap, int64_t t) {
  if (m.table == nullptr) return (static_cast<int64_t>(b) * Hkv + g) * n_cap + t;
  const int32_t page = __ldg(m.table + b * m.pages_per_seq + (t >> m.page_shift));
  if (page < 0 || page >= m.num_pages) return -1;
  return ((static_cast<int64_t>(page) * Hkv + g) << m.page_shift) + (t & ((int64_t(1) << m.page_shift) - 1));
}
#endif

inline Regions regions_of(int64_t n, int32_t sink, int32_t local) {
  Regions r;
  r.sink_end = n < sink ? n : sink;
  r.c0 = sink;
  r.c1 = n - local > r.c0 ? n - local : r.c0;
  r.local_start = n - local > r.sink_end ? n - local : r.sink_end;
  return r;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Workspace of ts_score_vote_select.
struct SelectLayout {
  int64_t nc = 0, nc_pad = 0;
  size_t off_scores = 0, off_theta = 0, off_keys = 0, off_hist = 0, off_vhist = 0, total = 0;
  int hist_splits = 0;   // partial-histogram slots per (b, g), sized for kMaxSmsForSizing
};
SelectLayout select_layout(const qasc_shape& s, const qasc_ts_params& p);

// Workspace of ts_sparse_attn.
struct AttnLayout {
  int64_t t_len = 0;       // |T| = sink + K + local tokens attended
  int splits = 1;          // split-K pieces per (b, g)
  int64_t per_split = 0;   // T positions per split
  size_t off_part = 0, total = 0;
};
AttnLayout attn_layout(const qasc_shape& s, const qasc_ts_params& p, int num_sms);

// Per-device facts the launchers need.
struct DeviceInfo {
  int device = 0;
  int num_sms = 0;
  int max_smem_optin = 0;
  unsigned* err_word = nullptr;   // device address of the error word
  int cut_clusters16 = 0;         // co-resident 16-CTA clusters of the top-K cutoff (0: not schedulable)
  int topc_clusters[3] = {0, 0, 0};  // co-resident top-c clusters of 8, 4 and 2 CTAs
};
const DeviceInfo* device_info();  // current device; nullptr on CUDA failure

// One-time per-device kernel attributes (dynamic shared memory limits), run
// by device_info() so that no attribute call happens while a stream is being
// captured into a graph.
cudaError_t configure_score_kernels(const DeviceInfo& dev);
cudaError_t configure_select_kernels(DeviceInfo& dev);
cudaError_t configure_attn_kernels(const DeviceInfo& dev);
cudaError_t configure_snapkv_kernels(DeviceInfo& dev);

// cuTensorMapEncodeTiled resolved through the runtime (no libcuda link).
using EncodeTiledFn = int (*)(void* tmap, int dtype, unsigned rank, void* gaddr, const uint64_t* gdim,
                              const uint64_t* gstride, const unsigned* box, const unsigned* estride, int interleave,
                              int swizzle, int l2promo, int oobfill);
EncodeTiledFn encode_tiled_fn();

// Workspace of snapkv_compress.
struct SnapLayout {
  int64_t c_out = 0;      // kept entries per KV head: min(c, n)
  int parts = 1;          // key-range pieces per (b, g)
  size_t off_stats = 0, off_score = 0, off_pool = 0, off_phist = 0, off_khist = 0, total = 0;
};
SnapLayout snap_layout(const qasc_shape& s, const qasc_snap_params& p);

int launch_snapkv(const qasc_shape& s, const qasc_snap_params& p, const SnapLayout& L, const uint16_t* q_obs,
                  const uint16_t* K, const uint16_t* V, int32_t* idx, uint16_t* K_out, uint16_t* V_out, uint8_t* ws,
                  const DeviceInfo& dev, cudaStream_t stream);

cudaError_t launch_index_append(const qasc_shape& s, const uint16_t* K, const uint16_t* W, uint16_t* index,
                                int64_t start, int64_t count, cudaStream_t stream);
// The same over a paged pool (K and index rows through pm).
cudaError_t launch_index_append_paged(const qasc_shape& s, const PageMap& pm, const uint16_t* K, const uint16_t* W,
                                      uint16_t* index, int64_t start, int64_t count, unsigned* err,
                                      cudaStream_t stream);
// Tokens [start, start + count) from the ring into their pages: K and V rows
// copied, index rows written.
cudaError_t launch_ring_flush(const qasc_shape& s, const PageMap& pm, const RingMap& ring, const uint16_t* W,
                              uint16_t* K_pool, uint16_t* V_pool, uint16_t* index, int64_t start, int64_t count,
                              unsigned* err, cudaStream_t stream);

// Geometry of the persistent scoring grid (one CTA per SM over 256-token
// tiles) and of the per-(b, g) partial histograms it writes.
struct ScoreGrid {
  int tiles_per_bg = 0, total = 0, grid = 1, max_splits = 1, hist_bits = 12;
};
// span = tokens the score tiles of one (b, g) cover: score_span().
ScoreGrid score_grid(const qasc_shape& s, int64_t span, int num_sms);
// The candidates for the contiguous cache; tokens [0, c1) for a paged pool
// (its tiles start at token 0 so that they split at page boundaries).
inline int64_t score_span(const Regions& R, bool paged) { return paged ? R.c1 : R.nc(); }

struct ScoreOut {
  float* scores;        // [B][Hq][nc_pad]
  uint32_t* hist;       // [B*Hkv][max_splits][GQ][2^hist_bits] partial histograms
  int64_t nc_pad;
  int max_splits;
  PageMap pm;           // index rows of a paged pool (pm.table != nullptr)
};

// Scores for all (b, h, i in C); returns a CUDA error or a negative value
// for an unsupported configuration.
int launch_scores(const qasc_shape& s, const qasc_ts_params& p, const uint16_t* q, const uint16_t* W,
                  const uint16_t* index, const ScoreOut& o, const DeviceInfo& dev, cudaStream_t stream);

// paged: the scores were computed over a paged pool (tiles from token 0).
int launch_select(const qasc_shape& s, const qasc_ts_params& p, const SelectLayout& L, uint8_t* ws, int32_t* sel,
                  const DeviceInfo& dev, cudaStream_t stream, bool paged = false);

// Per-KV-head selection (no voting): each (b, g) keeps the K candidates
// with the largest group-summed score, ascending in sel [B][Hkv][K].  A q'
// pass and the group scoring pass (ts_group.cu) write the group sums and the
// key range of every 512-token block; the top-c kernel selects.
constexpr int kGroupBlock = 512;
struct HeadSelLayout {
  int64_t nc = 0, nc_pad = 0;
  int parts = 0;             // range partials per (b, g) row (blocks, sized for either blocking)
  size_t off_qp = 0, off_gsum = 0, off_range = 0, total = 0;
};
HeadSelLayout head_select_layout(const qasc_shape& s, const qasc_ts_params& p);

struct GroupScoreArgs {
  float* qp = nullptr;       // [B*Hq][32] q'_h / sqrt(d'), written by the q' pass
  float* gsum = nullptr;     // [B*Hkv][nc_pad] group sums
  uint2* range = nullptr;    // [B*Hkv][blocks] {min, max} order-preserving key per block
  int64_t nc_pad = 0;
  PageMap pm;                // index rows of a paged pool (pm.table != nullptr)
};
// 512-token blocks of one (b, g): of the candidates (contiguous cache), of
// tokens [0, c1) for a paged pool (its blocks start at token 0).
int group_score_blocks(const Regions& R, bool paged);
// The q' pass, then the group scoring pass.
int launch_group_scores(const qasc_shape& s, const qasc_ts_params& p, const uint16_t* q, const uint16_t* W,
                        const uint16_t* index, const GroupScoreArgs& a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t configure_group_kernels(const DeviceInfo& dev);
int launch_head_topc(const qasc_shape& s, const qasc_ts_params& p, const HeadSelLayout& L, uint8_t* ws, int parts,
                     int32_t* sel, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t configure_head_select_kernels(DeviceInfo& dev);

// sel holds one list of K per sequence ([B][K]), or one per KV head
// ([B][Hkv][K]) when sel_per_kv; sel_len, when given, holds the entries in
// use of each list ([B] or [B][Hkv]); the others are masked.
int launch_sparse_attn(const qasc_shape& s, const qasc_ts_params& p, const AttnLayout& L, const uint16_t* q,
                       const uint16_t* K, const uint16_t* V, const int32_t* sel, float* out, float* lse,
                       uint8_t* ws, const DeviceInfo& dev, cudaStream_t stream, bool sel_per_kv = false,
                       const int32_t* sel_len = nullptr, const PageMap* pm = nullptr,
                       const RingMap* ring = nullptr);

// New tokens' K and V rows into the cache, keys and queries rotated; qs, ks,
// vs: values between tokens of q, k, v.
cudaError_t launch_rope_append(const qasc_shape& s, const PageMap& pm, const Batch& bt, const RopeArgs& r,
                               const uint16_t* q, int64_t qs, const uint16_t* k, int64_t ks, const uint16_t* v,
                               int64_t vs, uint16_t* q_out, uint16_t* K, uint16_t* V, const DeviceInfo& dev,
                               cudaStream_t stream);

// Causal attention of packed new tokens over the sink and local tokens of
// their sequences (n_prefix == 0), or over a prefix shared by all sequences
// and everything before them in their own (n_prefix > 0: pm_prefix, lens and
// pm count the tokens behind the prefix).
struct KvAttnArgs {
  const uint16_t* q = nullptr;   // [T][Hq][d]
  const uint16_t* K = nullptr;
  const uint16_t* V = nullptr;
  uint16_t* out = nullptr;       // [T][Hq][d] bf16
  float* lse = nullptr;          // [T][Hq], optional
  Batch bt;
  PageMap pm, pm_prefix;
  int64_t cache_rows = 0;        // rows of K and of V
  int32_t sink = 0, local = 0;
  int64_t n_prefix = 0;
  bool skip_empty = false;       // (with cu_q) rows of sequences without a cached token are left as they are,
  int seqs = 0;                  // and about as many sequences have some (0: all)
  int64_t stall = -1;            // self-test (>= 0): the tile at this place of each block's ring never comes,
  unsigned long long wait_ns = 0;   // and waits give up after this time
};
size_t kv_attn_workspace_bytes(int64_t T, int B, int Hq, int Hkv, bool prefix, int num_sms);
size_t kv_attn_whole_bytes();   // of a call that is not split: the least of any
// kSmallWorkspace, with *ws_bytes set to what the call's schedule needs, where it is less.
constexpr int kSmallWorkspace = -2;
int launch_kv_attn(const qasc_shape& s, const KvAttnArgs& a, uint8_t* ws, size_t* ws_bytes, const DeviceInfo& dev,
                   cudaStream_t stream);
cudaError_t configure_kv_attn_kernels(const DeviceInfo& dev);

// A 4-bit cache (kv4.cuh): codes [B][Hkv][n_cap][64] or of a pool, scales
// [..][8], and the factors of keys and values, powers of two.
struct Kv4Cache {
  uint8_t* K = nullptr;
  uint8_t* K_sf = nullptr;
  uint8_t* V = nullptr;
  uint8_t* V_sf = nullptr;
  float k_scale = 1.0f, v_scale = 1.0f;
};

// kv_rope_append's arguments, into a 4-bit cache.
cudaError_t launch_kv4_append(const qasc_shape& s, const PageMap& pm, const Batch& bt, const RopeArgs& r,
                              const uint16_t* q, int64_t qs, const uint16_t* k, int64_t ks, const uint16_t* v,
                              int64_t vs, uint16_t* q_out, const Kv4Cache& kv, const DeviceInfo& dev,
                              cudaStream_t stream);
// The newest tokens of a batch (its new ones) from the cache in bf16; strides
// of the outputs in values.
cudaError_t launch_kv4_read(const qasc_shape& s, const PageMap& pm, const Batch& bt, const Kv4Cache& kv, uint16_t* K_out,
                            int64_t k_token, int64_t k_head, uint16_t* V_out, int64_t v_token, int64_t v_head,
                            const DeviceInfo& dev, cudaStream_t stream);

// A bf16 copy of the tokens that the long sequences of a window call attend to, as a
// paged cache of its own: pages of kCopyPage tokens, those between sink and window left out.
constexpr int kCopyPage = 256;
struct Kv4Copy {
  int64_t most_rows = 0;           // sequences with more query rows of a KV head are copied
  int64_t capacity = 0;            // pages of K and of V
  int64_t likely = 0;              // of them that the call is likely to take
  int64_t pages_per_seq = 0;       // of the copy's block table
  int32_t* copied = nullptr;       // [B] 1: copied
  int32_t* lens = nullptr;         // [B] tokens in the copy (0: not copied)
  int32_t* table = nullptr;        // [B][pages_per_seq]
  uint16_t* K = nullptr;           // [capacity][Hkv][kCopyPage][d]
  uint16_t* V = nullptr;
  // The copy runs beside the kernel launched before it: it reads and writes without waiting for
  // that one, and waits before it ends.  This is sound as long as the kernel before
  //   - triggers only behind its own pdl_wait(): the copy begins when all blocks have triggered, and where that wait has
  //     returned whatever was launched earlier has completed and its writes are visible;
  //   - writes nothing that the copy reads, and neither reads nor writes the part of the workspace that
  //     the copy writes (copied, lens, table, K, V);
  // and as the copy's wait makes what comes behind it wait for both.
  bool beside = false;
};
cudaError_t launch_kv4_copy(const qasc_shape& s, const PageMap& pm, const Batch& bt, const Kv4Cache& kv, int32_t sink,
                            int32_t local, const Kv4Copy& c, const DeviceInfo& dev, cudaStream_t stream);

// Attention over a 4-bit cache: a window call's batch, or one token of every
// sequence over sink, listed and local tokens (listed: lists as in
// launch_sparse_attn, shape.n tokens in every sequence).
struct Kv4AttnArgs {
  const uint16_t* q = nullptr;   // [T][Hq][d]
  uint16_t* out = nullptr;       // [T][Hq][d] bf16
  float* lse = nullptr;          // [T][Hq], optional
  Kv4Cache kv;
  Batch bt;
  PageMap pm;
  int32_t sink = 0, local = 0;
  int64_t max_q = 1;             // most new tokens of a sequence, as the caller has them
  bool listed = false;
  const int32_t* sel = nullptr;
  const int32_t* sel_len = nullptr;
  int32_t K = 0;                 // entries of a list
  bool sel_per_kv = false;
};
size_t kv4_attn_least_bytes();   // for the most SMs; what every call has to have
// With room for the copies of any call of up to T tokens and max_q of a sequence.
size_t kv4_window_workspace_bytes(const qasc_shape& s, int64_t T, int64_t max_q, int32_t sink, int32_t local);
int launch_kv4_attn(const qasc_shape& s, const Kv4AttnArgs& a, uint8_t* ws, size_t ws_bytes, const DeviceInfo& dev,
                    cudaStream_t stream);
cudaError_t configure_kv4_kernels(const DeviceInfo& dev);
cudaError_t configure_kv4_cache_kernels(const DeviceInfo& dev);

// Neighbour expansion: rows of K ascending candidates in, the ascending union
// of their +-radius neighbourhoods within C out ([rows][cap], the first
// len[row] entries in use, the rest repeating the last).
size_t expand_workspace_bytes(const qasc_shape& s, const qasc_ts_params& p, int rows);
int launch_expand(const qasc_shape& s, const qasc_ts_params& p, int rows, const int32_t* sel, int radius,
                  int32_t* out, int cap, int32_t* len, void* ws, cudaStream_t stream);
cudaError_t configure_expand_kernels(const DeviceInfo& dev);

// ts_sparse_attn with its split-K scratch in a fixed area built into the
// library (see ts_attn.cu); the caller checks L.total against the capacity.
size_t sparse_attn_noalloc_capacity();
int launch_sparse_attn_noalloc(const qasc_shape& s, const qasc_ts_params& p, const AttnLayout& L, const uint16_t* q,
                               const uint16_t* K, const uint16_t* V, const int32_t* sel, float* out, float* lse,
                               const DeviceInfo& dev, cudaStream_t stream);

}  // namespace qasc
