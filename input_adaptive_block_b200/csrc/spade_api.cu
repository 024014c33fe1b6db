// C ABI of the SPADE executor hot path (declared in include/spade.h):
// argument validation, workspace layout, and the order of launches for the
// single steps and for the grouped (mixed-scheme) layer.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "spade_internal.cuh"
#include "spade_selftest.h"

// Latched device status (SPADE_OK / SPADE_ERR_TIMEOUT), one per device.
__device__ int g_spade_status;

// Fixed scratch for spade_block_sparse_attn_noalloc: the cost-ranked work list
// (up to SPADE_NOALLOC_MAX_ITEMS entries) followed by the work-hand-out ticket.
// Lives for as long as the library is loaded, on every device that uses it.
#define SPADE_NOALLOC_MAX_ITEMS 65536
static __device__ __align__(256) int g_noalloc_scratch[SPADE_NOALLOC_MAX_ITEMS + 64];

namespace spade {

namespace {

thread_local std::string g_err;

spade_status fail(spade_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return s;
}

spade_status cuda_fail(cudaError_t e, const char* where) {
  return fail(SPADE_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;

int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  return dev;
}

// Per-device caches below are atomics: callers on several host threads may
// fill the same slot at once (with the same value).
int* status_ptr() {
  static std::atomic<int*> ptrs[kMaxDevices];
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  int* p = ptrs[dev].load(std::memory_order_acquire);
  if (!p) {
    void* a = nullptr;
    if (cudaGetSymbolAddress(&a, g_spade_status) != cudaSuccess) return nullptr;
    p = static_cast<int*>(a);
    ptrs[dev].store(p, std::memory_order_release);
  }
  return p;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

spade_status check_geom(const spade_geom& g) {
  if (g.T <= 0 || g.H <= 0 || g.W <= 0 || g.bt <= 0 || g.bh <= 0 || g.bw <= 0)
    return fail(SPADE_ERR_INVALID, "geometry has a non-positive extent");
  if (g.bt > 256 || g.bh > 256 || g.bw > 256) return fail(SPADE_ERR_UNSUPPORTED, "block extent above 256");
  const long long bs = (long long)g.bt * g.bh * g.bw;
  if (bs > 1024) return fail(SPADE_ERR_UNSUPPORTED, "block size %lld above 1024", bs);
  const Geo gg = make_geo(g);
  if (gg.nb > 65535) return fail(SPADE_ERR_UNSUPPORTED, "more than 65535 blocks");
  return SPADE_OK;
}

spade_status check_d_dt(int d, spade_dtype dt) {
  if (d != 64 && d != 128) return fail(SPADE_ERR_UNSUPPORTED, "d=%d (supported: 64, 128)", d);
  if (dt != SPADE_F32 && dt != SPADE_BF16) return fail(SPADE_ERR_INVALID, "unknown dtype %d", (int)dt);
  return SPADE_OK;
}

cudaStream_t as_cuda(spade_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Layout of the grouped workspace (byte offsets).
struct GroupLayout {
  int n_sparse[SPADE_MAX_SCHEMES];
  std::vector<int> heads_of[SPADE_MAX_SCHEMES];   // sparse heads per scheme, ascending
  size_t qmean[SPADE_MAX_SCHEMES], kmean[SPADE_MAX_SCHEMES], prob[SPADE_MAX_SCHEMES];
  size_t cnt[SPADE_MAX_SCHEMES], idx[SPADE_MAX_SCHEMES];
  std::vector<int> pos;                             // position of head h in its scheme group
  size_t work;
  size_t ticket;
  int n_items;
  size_t total;
};

spade_status plan_group(const spade_geom* schemes, int n_schemes, const spade_head_scheme* table, int heads,
                        int d, int text_tokens, GroupLayout& L) {
  if (!schemes || !table) return fail(SPADE_ERR_INVALID, "null scheme table");
  if (n_schemes < 1 || n_schemes > SPADE_MAX_SCHEMES)
    return fail(SPADE_ERR_UNSUPPORTED, "n_schemes=%d (1..%d)", n_schemes, SPADE_MAX_SCHEMES);
  if (heads < 1 || heads > SPADE_MAX_HEADS) return fail(SPADE_ERR_UNSUPPORTED, "heads=%d (1..128)", heads);
  if (text_tokens < 0) return fail(SPADE_ERR_INVALID, "negative text_tokens");
  if (d != 64 && d != 128) return fail(SPADE_ERR_UNSUPPORTED, "d=%d (supported: 64, 128)", d);
  const long long N = (long long)schemes[0].T * schemes[0].H * schemes[0].W;
  for (int s = 0; s < n_schemes; ++s) {
    spade_status st = check_geom(schemes[s]);
    if (st != SPADE_OK) return st;
    if ((long long)schemes[s].T * schemes[s].H * schemes[s].W != N)
      return fail(SPADE_ERR_INVALID, "scheme %d covers a different number of tokens", s);
  }
  L.pos.assign(heads, -1);
  for (int s = 0; s < n_schemes; ++s) { L.n_sparse[s] = 0; L.heads_of[s].clear(); }
  for (int h = 0; h < heads; ++h) {
    const spade_head_scheme& r = table[h];
    if (r.scheme < 0 || r.scheme >= n_schemes) return fail(SPADE_ERR_INVALID, "head %d: scheme %d", h, r.scheme);
    if (r.dense != 0 && r.dense != 1) return fail(SPADE_ERR_INVALID, "head %d: dense flag %d", h, r.dense);
    if (!r.dense && !(r.tau > 0.f && r.tau <= 1e30f)) return fail(SPADE_ERR_INVALID, "head %d: tau", h);
    if (!r.dense) {
      L.pos[h] = L.n_sparse[r.scheme]++;
      L.heads_of[r.scheme].push_back(h);
    }
  }
  size_t off = 0;
  const int ntb = text_blocks(text_tokens);
  L.n_items = 0;
  for (int h = 0; h < heads; ++h) L.n_items += make_geo(schemes[table[h].scheme]).nb + ntb;
  for (int s = 0; s < n_schemes; ++s) {
    const Geo g = make_geo(schemes[s]);
    const size_t hs = L.n_sparse[s];
    if (hs > 0) {
      if (g.nb > SPADE_SELECT_MAX_NB) return fail(SPADE_ERR_UNSUPPORTED, "scheme %d: nb=%d above 1024", s, g.nb);
    }
    L.qmean[s] = off; off = align256(off + hs * g.nb * d * sizeof(float));
    L.kmean[s] = off; off = align256(off + hs * g.nb * d * sizeof(float));
    L.prob[s] = off;  off = align256(off + hs * g.nb * g.nb * sizeof(float));
    L.cnt[s] = off;   off = align256(off + hs * g.nb * sizeof(int));
    L.idx[s] = off;   off = align256(off + hs * g.nb * g.nb * sizeof(int));
  }
  L.work = off;
  off = align256(off + (size_t)L.n_items * sizeof(int));
  L.ticket = off;
  off = align256(off + sizeof(int));
  L.total = off;
  return SPADE_OK;
}

// Step 3: the tensor-core estimator (split-precision TF32); the FMA-pipe
// kernel only when the tensor-map encoder is unavailable.  want_probs = false
// asks for the scaled pooled scores (the index search then forms the
// softmax); *holds_scores says which of the two `out` received (the FMA-pipe
// kernel always writes probabilities).
cudaError_t run_estimate(const float* qm, const float* km, float* out, int heads, int nb, int d, int* status,
                         bool want_probs, bool* holds_scores, cudaStream_t s) {
  cudaError_t e = launch_estimate_tc(qm, km, out, heads, nb, d, status, want_probs, s);
  *holds_scores = !want_probs;
  if (e == cudaErrorNotSupported) {
    cudaGetLastError();
    e = launch_estimate(qm, km, out, heads, nb, d, s);
    *holds_scores = false;
  }
  return e;
}

// Host checks of an attention launch that do not depend on pointers; every
// entry point runs them before it enqueues anything.  A work item is packed
// as (head << 16) | query block, so a head's query blocks (video blocks plus
// text blocks) must number at most 65536; the CUDA-core kernel (taken when
// the tensor-core kernel does not support the shape) holds at most 128 slots
// per block.
spade_status check_attention(const AttnArgs& a) {
  const int ntb = text_blocks(a.text_tokens);
  for (int h = 0; h < a.heads; ++h)
    if ((long long)a.head[h].nb + ntb > 65536)
      return fail(SPADE_ERR_UNSUPPORTED, "head %d: %d blocks + %d text blocks exceed 65536 query blocks", h,
                  a.head[h].nb, ntb);
  if (!attn_tc_supported(a))
    for (int sc = 0; sc < a.n_schemes; ++sc)
      if (a.geo[sc].bs > 128) return fail(SPADE_ERR_UNSUPPORTED, "CUDA-core attention needs blocks <= 128 slots");
  return SPADE_OK;
}

// Enqueues the work list and the attention launch (check_attention has passed).
spade_status run_attention(AttnArgs& a, cudaStream_t s) {
  a.status = status_ptr();
  if (!a.status) return fail(SPADE_ERR_CUDA, "device status word unavailable");
  const bool tc = attn_tc_supported(a);
  cudaError_t e = launch_worklist(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "work list");
  if (tc) {
    const char* why = "";
    e = launch_attn_tc(a, s, &why);
    if (e != cudaSuccess) return fail(SPADE_ERR_CUDA, "tensor-core attention: %s (%s)", cudaGetErrorString(e), why);
  } else {
    e = launch_attn_simt(a, s);
    if (e != cudaSuccess) return cuda_fail(e, "CUDA-core attention");
  }
  return SPADE_OK;
}

// The attention launch of a grouped layer: every head of the table, kept
// lists of the sparse heads read from their places in the grouped workspace.
void grouped_attn_args(const void* q, const void* k, const void* v, void* out, const spade_geom* schemes,
                       int n_schemes, const spade_head_scheme* table, int heads, int d, int text_tokens,
                       spade_dtype dt, const GroupLayout& L, uint8_t* ws, AttnArgs& a) {
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v; a.out = out;
  a.n_schemes = n_schemes;
  for (int sc = 0; sc < n_schemes; ++sc) a.geo[sc] = make_geo(schemes[sc]);
  a.heads = heads; a.d = d; a.text_tokens = text_tokens; a.N = schemes[0].T * schemes[0].H * schemes[0].W;
  a.dt = dt;
  for (int h = 0; h < heads; ++h) {
    const int sc = table[h].scheme;
    const Geo& g = a.geo[sc];
    a.head[h].scheme = sc;
    a.head[h].nb = g.nb;
    a.head[h].dense = table[h].dense;
    if (!table[h].dense) {
      a.head[h].cnt_off = (int)((L.cnt[sc] + (size_t)L.pos[h] * g.nb * sizeof(int)) / sizeof(int));
      a.head[h].idx_off = (long long)((L.idx[sc] + (size_t)L.pos[h] * g.nb * g.nb * sizeof(int)) / sizeof(int));
    }
  }
  a.cnt = reinterpret_cast<const int*>(ws);
  a.idx = reinterpret_cast<const int*>(ws);
  a.work = reinterpret_cast<int*>(ws + L.work);
  a.ticket = reinterpret_cast<int*>(ws + L.ticket);
  a.n_items = L.n_items;
}

// Device address of g_noalloc_scratch on the current device.  The name is only
// a host-side stand-in in host code, so the address is looked up once per
// device (with that device current) and cached.
int* noalloc_scratch(spade_status* st) {
  static std::atomic<int*> ptrs[kMaxDevices];
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) {
    *st = fail(SPADE_ERR_CUDA, "no current CUDA device");
    return nullptr;
  }
  int* p = ptrs[dev].load(std::memory_order_acquire);
  if (!p) {
    void* a = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&a, g_noalloc_scratch);
    if (e != cudaSuccess) {
      *st = cuda_fail(e, "fixed scratch address");
      return nullptr;
    }
    p = static_cast<int*>(a);
    ptrs[dev].store(p, std::memory_order_release);
  }
  return p;
}

// ---- host-to-host pipelined layer (spade_grouped_attn_host) ----
constexpr int kHostSlots = 3;        // device group slots in flight
constexpr int kHostComputes = 2;     // compute streams the groups alternate over

// Layout of the caller's workspace for the host-to-host call.
struct HostLayout {
  int heads, head_chunk, n_groups, hc_max;
  size_t slot_bytes;       // one of Q, K, V, O for the largest group
  size_t ws_off;           // first grouped workspace
  size_t ws_bytes;         // each grouped workspace
  size_t total;
};

spade_status plan_host(const spade_geom* schemes, int n_schemes, const spade_head_scheme* table, int heads, int d,
                       int text_tokens, spade_dtype dt, int head_chunk, HostLayout& H) {
  GroupLayout L;
  spade_status st = plan_group(schemes, n_schemes, table, heads, d, text_tokens, L);   // the whole table
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (head_chunk < 1 || head_chunk > heads) return fail(SPADE_ERR_INVALID, "head_chunk=%d (1..%d)", head_chunk, heads);
  H.heads = heads;
  H.head_chunk = head_chunk;
  H.n_groups = (heads + head_chunk - 1) / head_chunk;
  H.hc_max = head_chunk;
  const size_t rows = (size_t)schemes[0].T * schemes[0].H * schemes[0].W + (size_t)text_tokens;
  const size_t esz = dt == SPADE_BF16 ? 2 : 4;
  H.slot_bytes = align256(rows * (size_t)H.hc_max * d * esz);
  H.ws_bytes = 0;
  for (int g = 0; g < H.n_groups; ++g) {
    const int h0 = g * head_chunk, hc = std::min(head_chunk, heads - h0);
    GroupLayout Lg;
    if ((st = plan_group(schemes, n_schemes, table + h0, hc, d, text_tokens, Lg)) != SPADE_OK) return st;
    H.ws_bytes = std::max(H.ws_bytes, Lg.total);
  }
  H.ws_bytes = align256(H.ws_bytes);
  const int ns = std::min(kHostSlots, H.n_groups);
  H.ws_off = (size_t)ns * 4 * H.slot_bytes;
  H.total = H.ws_off + (size_t)kHostComputes * H.ws_bytes;
  return SPADE_OK;
}

// Streams and events of the host-to-host call, created once per device.
struct HostPipe {
  std::mutex mu;                    // one call enqueues at a time
  bool ready = false;
  cudaStream_t up = nullptr, down = nullptr, comp[kHostComputes] = {nullptr, nullptr};
  std::vector<cudaEvent_t> ev;      // 3 per group (loaded, done, returned) + joins
};

HostPipe& host_pipe(int dev) {
  static HostPipe pipes[kMaxDevices];
  return pipes[dev];
}

// Creates the streams, and enough events for n_events (caller holds P.mu).
cudaError_t host_pipe_setup(HostPipe& P, size_t n_events) {
  cudaError_t e = cudaSuccess;
  if (!P.ready) {
    e = cudaStreamCreateWithFlags(&P.up, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&P.down, cudaStreamNonBlocking);
    for (int c = 0; e == cudaSuccess && c < kHostComputes; ++c)
      e = cudaStreamCreateWithFlags(&P.comp[c], cudaStreamNonBlocking);
    if (e != cudaSuccess) return e;
    P.ready = true;
  }
  while (P.ev.size() < n_events) {
    cudaEvent_t ev;
    if ((e = cudaEventCreateWithFlags(&ev, cudaEventDisableTiming)) != cudaSuccess) return e;
    P.ev.push_back(ev);
  }
  return cudaSuccess;
}

// ---- row passes around the attention: checks of their operands ----

constexpr long long kMaxRows = 1LL << 37;     // a block's share of them is counted in 31 bits

// A list of rows in memory, for the overlap checks (bytes).
struct Region {
  const char* name;
  uintptr_t p;
  unsigned long long rows, stride, len;
  bool out, row;      // written; token rows (not a parameter, a gradient of one, or scratch)
};

struct Regions {
  Region r[24];
  int n = 0;
  void add(const char* name, const void* p, long long rows, long long stride, long long len, bool out,
           bool row = false) {
    if (p && rows > 0 && len > 0)
      r[n++] = {name, reinterpret_cast<uintptr_t>(p), (unsigned long long)rows, (unsigned long long)stride,
                (unsigned long long)len, out, row};
  }
};

bool disjoint(const Region& a, const Region& b) {
  const uintptr_t ae = a.p + (a.rows - 1) * a.stride + a.len, be = b.p + (b.rows - 1) * b.stride + b.len;
  if (ae <= b.p || be <= a.p) return true;
  if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return false;
  // rows of one spacing: b's rows start `gap` bytes into a's spacing
  const unsigned long long gap = b.p >= a.p ? (b.p - a.p) % a.stride : (a.stride - (a.p - b.p) % a.stride) % a.stride;
  return gap >= a.len && gap + b.len <= a.stride;
}

// Outputs overlap nothing, except that token rows may be written exactly over
// token rows that come in: every element is read by the thread that then
// writes it.
spade_status check_overlap(const Regions& rs) {
  for (int i = 0; i < rs.n; ++i) {
    if (!rs.r[i].out) continue;
    for (int j = 0; j < rs.n; ++j) {
      const Region &a = rs.r[i], &b = rs.r[j];
      if (i == j || (b.out && j < i)) continue;
      const bool same = a.row && b.row && !b.out && a.p == b.p && a.rows == b.rows && a.len == b.len &&
                        (a.stride == b.stride || a.rows == 1);
      if (!same && !disjoint(a, b)) return fail(SPADE_ERR_INVALID, "%s overlaps %s", a.name, b.name);
    }
  }
  return SPADE_OK;
}

bool row_dtype(int dt) { return dt == SPADE_F32 || dt == SPADE_BF16; }
int dtype_size(int dt) { return dt == SPADE_BF16 ? 2 : 4; }

// A stride (0: packed) of rows of len elements, in elements.
spade_status check_stride(const char* name, int64_t stride, long long len, long long* out) {
  *out = stride == 0 ? len : stride;
  if (*out < len || *out > (1LL << 40))
    return fail(SPADE_ERR_INVALID, "%s: stride %lld for rows of %lld", name, (long long)stride, len);
  return SPADE_OK;
}

spade_status check_operand(const char* name, const void* p, int dt) {
  if (!p) return fail(SPADE_ERR_INVALID, "%s is null", name);
  if (reinterpret_cast<uintptr_t>(p) % dtype_size(dt)) return fail(SPADE_ERR_INVALID, "%s is not aligned to its type", name);
  return SPADE_OK;
}

spade_status check_scratch(const void* workspace, size_t ws_bytes, size_t need) {
  if (!need) return SPADE_OK;
  if (!workspace || ws_bytes < need)
    return fail(SPADE_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? ws_bytes : 0, need);
  if (!aligned16(workspace)) return fail(SPADE_ERR_INVALID, "workspace must be 16-byte aligned");
  return SPADE_OK;
}

// by = 1 .. 2^31 - 1: with 2^s the power of two at or above it, the multiplier
// 2^(31 + s) / by rounded up past the quotient is below 2^32 and off by at
// most one, which 2^31 multiples of it do not carry over 2^(31 + s) / by.
QkArgs::Divisor divisor(unsigned by) {
  unsigned s = 0;
  while ((1ULL << s) < by) ++s;
  return {by, (unsigned)((1ULL << (31 + s)) / by + 1), 31 + s};
}

// Sizes, types, strides and rotation of a Q/K pass; rope == nullptr skips the
// rotation and the grid (workspace query).
spade_status plan_qk(const spade_qk_desc* D, const spade_rope* rope, const int32_t* positions, QkArgs& a) {
  memset(&a, 0, sizeof(a));
  if (!D) return fail(SPADE_ERR_INVALID, "null descriptor");
  const spade_qk_desc& d = *D;
  if (d.rows < 0 || d.rows > kMaxRows || d.text_tokens < 0 || d.text_tokens > d.rows)
    return fail(SPADE_ERR_INVALID, "rows=%lld, text_tokens=%lld", (long long)d.rows, (long long)d.text_tokens);
  if (d.q_heads < 0 || d.k_heads < 0 || (!d.q_heads && !d.k_heads))
    return fail(SPADE_ERR_INVALID, "q_heads=%d, k_heads=%d", d.q_heads, d.k_heads);
  if (d.q_heads > SPADE_MAX_HEADS || d.k_heads > SPADE_MAX_HEADS)
    return fail(SPADE_ERR_UNSUPPORTED, "q_heads=%d, k_heads=%d (up to %d)", d.q_heads, d.k_heads, SPADE_MAX_HEADS);
  if (d.d < 2 || d.d > 2 * SPADE_ROPE_MAX_PAIRS || d.d % 2)
    return fail(SPADE_ERR_UNSUPPORTED, "d=%d (even, 2..%d)", d.d, 2 * SPADE_ROPE_MAX_PAIRS);
  if (!row_dtype(d.dt) || !row_dtype(d.weight_dt))
    return fail(SPADE_ERR_INVALID, "unknown dtype %d, %d", d.dt, d.weight_dt);
  if (d.norm < SPADE_QK_NORM_NONE || d.norm > SPADE_QK_NORM_HEAD) return fail(SPADE_ERR_INVALID, "norm %d", d.norm);
  if (d.norm != SPADE_QK_NORM_NONE && !(d.eps >= 0.f && std::isfinite(d.eps)))
    return fail(SPADE_ERR_INVALID, "eps %g", (double)d.eps);
  a.rows = d.rows;
  a.video_rows = d.rows - d.text_tokens;
  a.heads[0] = d.q_heads;
  a.heads[1] = d.k_heads;
  a.d = d.d;
  a.norm = d.norm;
  a.eps = d.eps;
  a.weight_bf16 = d.weight_dt == SPADE_BF16;
  for (a.lanes = 1; a.lanes * 16 < d.d;) a.lanes *= 2;
  for (int t = 0; t < 2; ++t)
    a.inv_count[t] = 1.f / (float)(d.norm == SPADE_QK_NORM_TOKEN ? std::max(a.heads[t], 1) * d.d : d.d);
  spade_status st;
  const int64_t strides[6] = {d.q_stride, d.k_stride, d.q_out_stride, d.k_out_stride, d.q_dout_stride, d.k_dout_stride};
  long long* to[6] = {&a.x_stride[0], &a.x_stride[1], &a.out_stride[0], &a.out_stride[1], &a.dout_stride[0],
                      &a.dout_stride[1]};
  const char* names[6] = {"q", "k", "q output", "k output", "q gradient", "k gradient"};
  for (int i = 0; i < 6; ++i)
    if (a.heads[i & 1] && (st = check_stride(names[i], strides[i], (long long)a.heads[i & 1] * d.d, to[i])) != SPADE_OK)
      return st;
  if (!rope) return SPADE_OK;
  if (rope->style != SPADE_ROPE_INTERLEAVED && rope->style != SPADE_ROPE_HALF)
    return fail(SPADE_ERR_INVALID, "rotation style %d", rope->style);
  if (rope->pairs < 0 || rope->pairs > d.d / 2)
    return fail(SPADE_ERR_INVALID, "%d rotated pairs in heads of %d channels", rope->pairs, d.d);
  if (rope->style == SPADE_ROPE_HALF && rope->pairs != d.d / 2)
    return fail(SPADE_ERR_UNSUPPORTED, "half style with %d of %d pairs", rope->pairs, d.d / 2);
  a.half = rope->style == SPADE_ROPE_HALF;
  a.pairs = rope->pairs;
  for (int i = 0; i < rope->pairs; ++i) {
    if (rope->axis[i] < 0 || rope->axis[i] > 2) return fail(SPADE_ERR_INVALID, "pair %d: axis %d", i, rope->axis[i]);
    if (!std::isfinite(rope->freq[i])) return fail(SPADE_ERR_INVALID, "pair %d: frequency not finite", i);
    a.axis[i] = (uint8_t)rope->axis[i];
    a.turn[i] = rope->freq[i] / 6.283185307179586476925286766559;
  }
  a.H = a.W = divisor(1);
  if (positions) {
    if (d.text_tokens) return fail(SPADE_ERR_INVALID, "text_tokens with positions");
    if (reinterpret_cast<uintptr_t>(positions) % 4) return fail(SPADE_ERR_INVALID, "positions are not aligned to their type");
    a.positions = positions;
  } else if (a.video_rows > 0) {
    if (d.T <= 0 || d.H <= 0 || d.W <= 0) return fail(SPADE_ERR_INVALID, "grid has a non-positive extent");
    const long long plane = (long long)d.H * d.W;
    if (plane > INT32_MAX || plane * d.T > INT32_MAX) return fail(SPADE_ERR_UNSUPPORTED, "grid of 2^31 tokens or more");
    if (d.token_offset < 0 || d.token_offset > plane * d.T || a.video_rows > plane * d.T - d.token_offset)
      return fail(SPADE_ERR_INVALID, "rows past the end of the grid: offset %lld, %lld rows, %lld tokens",
                  (long long)d.token_offset, a.video_rows, plane * d.T);
    a.tok0 = (int)d.token_offset;
    a.H = divisor((unsigned)d.H);
    a.W = divisor((unsigned)d.W);
  }
  return SPADE_OK;
}

long long qk_weight_len(const QkArgs& a, int t) {
  return a.norm == SPADE_QK_NORM_TOKEN ? (long long)a.heads[t] * a.d : (a.heads[t] ? a.d : 0);
}

// Pointers of a Q/K pass, and whether it can move 16 bytes at a time.
spade_status bind_qk(const spade_qk_desc* D, QkArgs& a, const void* const x[2], const void* const dout[2],
                     const void* const w[2], void* const out[2], float* const dw[2], const void* workspace,
                     size_t ws_need) {
  const char* xn[2] = {"q", "k"};
  const char* gn[2] = {"dq_out", "dk_out"};
  const char* on[2] = {dout ? "dq" : "q_out", dout ? "dk" : "k_out"};
  const char* wn[2] = {"q_weight", "k_weight"};
  const bool need_x = !dout || a.norm != SPADE_QK_NORM_NONE;
  const int es = dtype_size(D->dt), ws = dtype_size(D->weight_dt);
  Regions rs;
  spade_status st;
  for (int t = 0; t < 2; ++t) {
    if (!a.heads[t]) {
      if (dw && dw[t]) return fail(SPADE_ERR_INVALID, "weight gradient of an absent tensor");
      continue;
    }
    const long long len = (long long)a.heads[t] * a.d;
    if (a.rows) {
      if (need_x && (st = check_operand(xn[t], x[t], D->dt)) != SPADE_OK) return st;
      if (dout && (st = check_operand(gn[t], dout[t], D->dt)) != SPADE_OK) return st;
      if ((st = check_operand(on[t], out[t], D->dt)) != SPADE_OK) return st;
    }
    if (w[t] && a.norm == SPADE_QK_NORM_NONE) return fail(SPADE_ERR_INVALID, "%s without a norm", wn[t]);
    if (w[t] && (st = check_operand(wn[t], w[t], D->weight_dt)) != SPADE_OK) return st;
    if (dw && dw[t] && (st = check_operand("weight gradient", dw[t], SPADE_F32)) != SPADE_OK) return st;
    a.x[t] = need_x ? x[t] : nullptr;
    a.dout[t] = dout ? dout[t] : nullptr;
    a.out[t] = out[t];
    a.weight[t] = w[t];
    a.dweight[t] = dw ? dw[t] : nullptr;
    rs.add(xn[t], a.x[t], a.rows, a.x_stride[t] * es, len * es, false, true);
    rs.add(gn[t], a.dout[t], a.rows, a.dout_stride[t] * es, len * es, false, true);
    rs.add(on[t], a.out[t], a.rows, a.out_stride[t] * es, len * es, true, true);
    rs.add(wn[t], w[t], 1, 0, qk_weight_len(a, t) * ws, false);
    rs.add("weight gradient", a.dweight[t], 1, 0, qk_weight_len(a, t) * 4, true);
  }
  rs.add("positions", a.positions, 1, 0, a.rows * 12, false);
  rs.add("workspace", workspace, 1, 0, (long long)ws_need, true);
  // Q's output over K's input (or the reverse) is no in-place call: their heads are on other threads
  for (int i = 0; i < rs.n; ++i)
    for (int j = 0; j < rs.n; ++j)
      if (rs.r[i].out && rs.r[i].name == on[0] && (rs.r[j].name == xn[1] || rs.r[j].name == gn[1]) &&
          !disjoint(rs.r[i], rs.r[j]))
        return fail(SPADE_ERR_INVALID, "%s overlaps %s", rs.r[i].name, rs.r[j].name);
      else if (rs.r[i].out && rs.r[i].name == on[1] && (rs.r[j].name == xn[0] || rs.r[j].name == gn[0]) &&
               !disjoint(rs.r[i], rs.r[j]))
        return fail(SPADE_ERR_INVALID, "%s overlaps %s", rs.r[i].name, rs.r[j].name);
  return check_overlap(rs);
}

// Sizes, types, strides and parameters of a row pass; bwd: the gradients'
// strides are checked too.
spade_status plan_row(const spade_row_desc* D, const spade_row_params* P, bool bwd, RowArgs& a) {
  memset(&a, 0, sizeof(a));
  if (!D) return fail(SPADE_ERR_INVALID, "null descriptor");
  const spade_row_desc& d = *D;
  if (d.rows < 0 || d.rows > kMaxRows || d.groups < 1 || d.groups > kMaxRows || d.rows % d.groups)
    return fail(SPADE_ERR_INVALID, "rows=%lld in groups=%lld", (long long)d.rows, (long long)d.groups);
  if (d.dim < 1) return fail(SPADE_ERR_INVALID, "dim=%d", d.dim);
  if (d.dim > SPADE_ROW_MAX_DIM) return fail(SPADE_ERR_UNSUPPORTED, "dim=%d (up to %d)", d.dim, SPADE_ROW_MAX_DIM);
  if (!row_dtype(d.x_dt) || !row_dtype(d.branch_dt) || !row_dtype(d.param_dt))
    return fail(SPADE_ERR_INVALID, "unknown dtype %d, %d, %d", d.x_dt, d.branch_dt, d.param_dt);
  if (d.x_dt == SPADE_BF16 && d.branch_dt == SPADE_F32)
    return fail(SPADE_ERR_UNSUPPORTED, "a float32 branch on a bfloat16 stream");
  if (d.norm < SPADE_NORM_NONE || d.norm > SPADE_NORM_LAYER || d.post_norm < SPADE_NORM_NONE ||
      d.post_norm > SPADE_NORM_LAYER)
    return fail(SPADE_ERR_INVALID, "norm %d, post_norm %d", d.norm, d.post_norm);
  a.rows = d.rows;
  a.groups = d.groups;
  a.rows_per_group = d.rows / d.groups;
  a.chunks = 1;
  a.dim = d.dim;
  a.norm = d.norm;
  a.post_norm = d.post_norm;
  a.eps = d.eps;
  a.post_eps = d.post_eps;
  a.residual_scale = d.residual_scale;
  a.inv_dim = 1.f / (float)d.dim;
  a.x_bf16 = d.x_dt == SPADE_BF16;
  a.branch_bf16 = d.branch_dt == SPADE_BF16;
  a.param_bf16 = d.param_dt == SPADE_BF16;
  const struct { const char* name; int64_t stride; long long* to; bool used; } strides[] = {
      {"x", d.x_stride, &a.x_stride, true},
      {"y", d.y_stride, &a.y_stride, true},
      {"x_out", d.x_out_stride, &a.x_out_stride, !bwd},
      {"h", d.h_stride, &a.h_stride, !bwd},
      {"dx_out", d.dx_out_stride, &a.dx_out_stride, bwd},
      {"dh", d.dh_stride, &a.dh_stride, bwd},
      {"dx", d.dx_stride, &a.dx_stride, bwd},
      {"dy", d.dy_stride, &a.dy_stride, bwd},
      {"gate", d.gate_stride, &a.gate_stride, true},
      {"scale", d.scale_stride, &a.scale_stride, true},
      {"shift", d.shift_stride, &a.shift_stride, true}};
  spade_status st;
  for (const auto& s : strides)
    if (s.used && (st = check_stride(s.name, s.stride, d.dim, s.to)) != SPADE_OK) return st;
  if (P) {
    const struct { const char* name; const void* p; const void** to; } params[] = {
        {"gate", P->gate, &a.gate},       {"post_weight", P->post_weight, &a.post_weight},
        {"weight", P->weight, &a.weight}, {"bias", P->bias, &a.bias},
        {"scale", P->scale, &a.scale},    {"shift", P->shift, &a.shift}};
    for (const auto& p : params) {
      if (p.p && (st = check_operand(p.name, p.p, d.param_dt)) != SPADE_OK) return st;
      *p.to = p.p;
    }
  }
  return SPADE_OK;
}

spade_status check_eps(int norm, float eps) {
  if (norm != SPADE_NORM_NONE && !(eps >= 0.f && std::isfinite(eps)))
    return fail(SPADE_ERR_INVALID, "eps %g", (double)eps);
  return SPADE_OK;
}

// What the residual half and the norm half of a pass need and may not have.
spade_status check_halves(RowArgs& a, bool res, bool norm) {
  spade_status st;
  if (norm) {
    if (a.norm == SPADE_NORM_NONE) return fail(SPADE_ERR_INVALID, "norm is none");
    if ((st = check_eps(a.norm, a.eps)) != SPADE_OK) return st;
  } else {
    if (a.weight || a.bias || a.scale || a.shift) return fail(SPADE_ERR_INVALID, "norm parameters without a norm");
    a.norm = SPADE_NORM_NONE;
  }
  if (res) {
    if (a.post_weight && a.post_norm == SPADE_NORM_NONE)
      return fail(SPADE_ERR_INVALID, "post_weight without a post_norm");
    if ((st = check_eps(a.post_norm, a.post_eps)) != SPADE_OK) return st;
  } else {
    if (a.gate || a.post_weight) return fail(SPADE_ERR_INVALID, "gate parameters without a residual");
    a.post_norm = SPADE_NORM_NONE;
  }
  return SPADE_OK;
}

void add_params(Regions& rs, const RowArgs& a) {
  const int ep = a.param_bf16 ? 2 : 4;
  const long long len = (long long)a.dim * ep;
  rs.add("gate", a.gate, a.groups, a.gate_stride * ep, len, false);
  rs.add("scale", a.scale, a.groups, a.scale_stride * ep, len, false);
  rs.add("shift", a.shift, a.groups, a.shift_stride * ep, len, false);
  rs.add("post_weight", a.post_weight, 1, 0, len, false);
  rs.add("weight", a.weight, 1, 0, len, false);
  rs.add("bias", a.bias, 1, 0, len, false);
}

struct RowOperand {
  const char* name;
  const void* p;
  long long stride;
  bool branch, out, optional;
};

// Row operands: present, aligned, apart from one another.
spade_status check_rows(const RowArgs& a, const RowOperand* ops, int n, Regions& rs) {
  spade_status st;
  for (int i = 0; i < n; ++i) {
    const int dt = (ops[i].branch ? a.branch_bf16 : a.x_bf16) ? SPADE_BF16 : SPADE_F32;
    if (!ops[i].p && (ops[i].optional || !a.rows)) continue;
    if ((st = check_operand(ops[i].name, ops[i].p, dt)) != SPADE_OK) return st;
    const int es = dtype_size(dt);
    rs.add(ops[i].name, ops[i].p, a.rows, ops[i].stride * es, (long long)a.dim * es, ops[i].out, true);
  }
  return check_overlap(rs);
}

spade_status run_row_fwd(const spade_row_desc* desc, const spade_row_params* params, const void* x, const void* y,
                         void* x_out, void* h, bool res, bool norm, cudaStream_t s, const char* where) {
  RowArgs a;
  spade_status st = plan_row(desc, params, false, a);
  if (st != SPADE_OK) return st;
  if ((st = check_halves(a, res, norm)) != SPADE_OK) return st;
  a.x = x;
  a.y = y;
  a.x_out = x_out;
  a.h = h;
  const RowOperand ops[] = {{"x", x, a.x_stride, false, false, false},
                            {"y", y, a.y_stride, true, false, !res},
                            {"x_out", x_out, a.x_out_stride, false, true, !res},
                            {"h", h, a.h_stride, true, true, !norm}};
  Regions rs;
  add_params(rs, a);
  if ((st = check_rows(a, ops, 4, rs)) != SPADE_OK) return st;
  if (!a.rows) return SPADE_OK;
  const cudaError_t e = launch_row_fwd(a, s);
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, where);
}

spade_status run_row_bwd(const spade_row_desc* desc, const spade_row_params* params, const void* dx_out,
                         const void* dh, const void* x, const void* y, void* dx, void* dy,
                         const spade_row_grads* grads, void* workspace, size_t ws_bytes, bool res, bool norm,
                         cudaStream_t s, const char* where) {
  RowArgs a;
  spade_status st = plan_row(desc, params, true, a);
  if (st != SPADE_OK) return st;
  if ((st = check_halves(a, res, norm)) != SPADE_OK) return st;
  a.x = x;
  a.y = y;
  a.dx_out = dx_out;
  a.dh = dh;
  a.dx = dx;
  a.dy = dy;
  if (grads) {
    a.dgate = grads->gate;
    a.dpost_weight = grads->post_weight;
    a.dweight = grads->weight;
    a.dbias = grads->bias;
    a.dscale = grads->scale;
    a.dshift = grads->shift;
  }
  if (!norm && (a.dweight || a.dbias || a.dscale || a.dshift))
    return fail(SPADE_ERR_INVALID, "gradients of norm parameters without a norm");
  if (!res && (a.dgate || a.dpost_weight)) return fail(SPADE_ERR_INVALID, "gradients of gate parameters without a residual");
  if (a.dpost_weight && a.post_norm == SPADE_NORM_NONE)
    return fail(SPADE_ERR_INVALID, "gradient of post_weight without a post_norm");
  if (a.rows && res && norm && dx == y) return fail(SPADE_ERR_INVALID, "dx overlaps y");   // y is read again after dx
  Regions rs;
  add_params(rs, a);
  const struct { const char* name; float* p; long long len; } gs[] = {
      {"gate gradient", a.dgate, a.groups * a.dim},   {"post_weight gradient", a.dpost_weight, a.dim},
      {"weight gradient", a.dweight, a.dim},          {"bias gradient", a.dbias, a.dim},
      {"scale gradient", a.dscale, a.groups * a.dim}, {"shift gradient", a.dshift, a.groups * a.dim}};
  for (const auto& g : gs) {
    if (g.p && (st = check_operand(g.name, g.p, SPADE_F32)) != SPADE_OK) return st;
    rs.add(g.name, g.p, 1, 0, g.len * 4, true);
  }
  const RowOperand ops[] = {{"x", x, a.x_stride, false, false, !norm},
                            {"y", y, a.y_stride, true, false, !res},
                            {norm && !res ? "dres" : "dx_out", dx_out, a.dx_out_stride, false, false, norm},
                            {"dh", dh, a.dh_stride, true, false, !norm},
                            {"dx", dx, a.dx_stride, false, true, !norm},
                            {"dy", dy, a.dy_stride, true, true, !res}};
  if (!a.rows) {
    if ((st = check_rows(a, ops, 6, rs)) != SPADE_OK) return st;
    for (const auto& g : gs)
      if (g.p) {
        const cudaError_t e = cudaMemsetAsync(g.p, 0, sizeof(float) * (size_t)g.len, s);
        if (e != cudaSuccess) return cuda_fail(e, where);
      }
    return SPADE_OK;
  }
  const bool weights = a.dweight || a.dbias || a.dpost_weight;
  const RowPlan plan = plan_row_bwd(a.rows, a.groups, a.dim, weights);
  a.chunks = plan.chunks;
  const bool sums = weights || a.dgate || a.dscale || a.dshift;      // else no column sum leaves its block
  const size_t need = sums || workspace ? plan.floats * sizeof(float) : 0;      // one that is given is whole
  if ((st = check_scratch(workspace, ws_bytes, need)) != SPADE_OK) return st;
  a.part = need && sums ? static_cast<float*>(workspace) : nullptr;
  rs.add("workspace", a.part, 1, 0, (long long)need, true);
  if ((st = check_rows(a, ops, 6, rs)) != SPADE_OK) return st;
  const cudaError_t e = launch_row_bwd(a, plan.grid, s);
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, where);
}

}  // namespace

int num_sms() {
  static std::atomic<int> sms[kMaxDevices];
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return 1;
  int v = sms[dev].load(std::memory_order_relaxed);
  if (!v) {
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    if (v <= 0) v = 1;
    sms[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

long long device_wait_timeout_ns() {
  static const long long ns = [] {
    const char* e = getenv("SPADE_WAIT_TIMEOUT_MS");
    long long ms = e ? atoll(e) : 10000;
    if (ms <= 0) ms = 10000;
    return ms * 1000000LL;
  }();
  return ns;
}

}  // namespace spade

using namespace spade;

extern "C" {

int spade_version(void) { return 1; }

const char* spade_status_string(spade_status s) {
  switch (s) {
    case SPADE_OK: return "ok";
    case SPADE_ERR_INVALID: return "invalid argument";
    case SPADE_ERR_UNSUPPORTED: return "unsupported configuration";
    case SPADE_ERR_CUDA: return "CUDA error";
    case SPADE_ERR_TIMEOUT: return "device wait timed out";
    case SPADE_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

const char* spade_last_error_message(void) { return g_err.c_str(); }

spade_status spade_tile3d(const void* x, void* xt, spade_geom g, int heads, int d, spade_dtype dt,
                          spade_stream_t stream) {
  spade_status st = check_geom(g);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!x || !xt) return fail(SPADE_ERR_INVALID, "null pointer");
  if (!aligned16(x) || !aligned16(xt)) return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (heads < 1) return fail(SPADE_ERR_INVALID, "heads=%d", heads);
  cudaError_t e = launch_tile3d(x, xt, make_geo(g), heads, d, dt, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "tile3d");
}

spade_status spade_summarize(const void* x, float* xmean, spade_geom g, int heads, int d, spade_dtype dt,
                             spade_stream_t stream) {
  spade_status st = check_geom(g);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!x || !xmean) return fail(SPADE_ERR_INVALID, "null pointer");
  if (!aligned16(x) || !aligned16(xmean)) return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (heads < 1) return fail(SPADE_ERR_INVALID, "heads=%d", heads);
  cudaError_t e = launch_summarize(x, xmean, make_geo(g), heads, 0, heads, d, dt, 0, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "summarize");
}

spade_status spade_summarize_mode(const void* x, float* out, spade_geom g, int heads, int d, spade_dtype dt,
                                  spade_summary mode, spade_stream_t stream) {
  if (mode != SPADE_SUM_MEAN && mode != SPADE_SUM_MAX && mode != SPADE_SUM_MIN)
    return fail(SPADE_ERR_INVALID, "summary mode %d", (int)mode);
  if (mode == SPADE_SUM_MEAN) return spade_summarize(x, out, g, heads, d, dt, stream);
  spade_status st = check_geom(g);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!x || !out) return fail(SPADE_ERR_INVALID, "null pointer");
  if (!aligned16(x) || !aligned16(out)) return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (heads < 1) return fail(SPADE_ERR_INVALID, "heads=%d", heads);
  cudaError_t e = launch_summarize(x, out, make_geo(g), heads, 0, heads, d, dt, (int)mode, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "summarize");
}

spade_status spade_summarize_qk(const void* q, const void* k, float* qmean, float* kmean, spade_geom g, int heads,
                                int d, spade_dtype dt, spade_stream_t stream) {
  spade_status st = check_geom(g);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!q || !k || !qmean || !kmean) return fail(SPADE_ERR_INVALID, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(qmean) || !aligned16(kmean))
    return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (heads < 1) return fail(SPADE_ERR_INVALID, "heads=%d", heads);
  cudaError_t e = launch_summarize_pair(q, k, qmean, kmean, make_geo(g), heads, 0, heads, d, dt, 0, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "summarize");
}

static spade_status check_estimate_args(const float* qmean, const float* kmean, const float* out, int heads, int nb,
                                       int d) {
  if (!qmean || !kmean || !out) return fail(SPADE_ERR_INVALID, "null pointer");
  if (!aligned16(qmean) || !aligned16(kmean) || !aligned16(out))
    return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (heads < 1 || heads > 65535) return fail(SPADE_ERR_INVALID, "heads=%d", heads);
  if (nb < 1) return fail(SPADE_ERR_INVALID, "nb=%d", nb);
  if (nb > SPADE_ESTIMATE_MAX_NB) return fail(SPADE_ERR_UNSUPPORTED, "nb=%d above %d", nb, SPADE_ESTIMATE_MAX_NB);
  if (d != 64 && d != 128) return fail(SPADE_ERR_UNSUPPORTED, "d=%d (supported: 64, 128)", d);
  return SPADE_OK;
}

spade_status spade_estimate(const float* qmean, const float* kmean, float* prob, int heads, int nb, int d,
                            spade_stream_t stream) {
  spade_status st0 = check_estimate_args(qmean, kmean, prob, heads, nb, d);
  if (st0 != SPADE_OK) return st0;
  int* st = status_ptr();
  if (!st) return fail(SPADE_ERR_CUDA, "device status word unavailable");
  bool scores = false;
  cudaError_t e = run_estimate(qmean, kmean, prob, heads, nb, d, st, true, &scores, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "estimate");
}

spade_status spade_estimate_scores(const float* qmean, const float* kmean, float* scores, int heads, int nb, int d,
                                   spade_stream_t stream) {
  spade_status st0 = check_estimate_args(qmean, kmean, scores, heads, nb, d);
  if (st0 != SPADE_OK) return st0;
  int* st = status_ptr();
  if (!st) return fail(SPADE_ERR_CUDA, "device status word unavailable");
  cudaError_t e = launch_estimate_tc(qmean, kmean, scores, heads, nb, d, st, false, as_cuda(stream));
  if (e == cudaErrorNotSupported) {
    cudaGetLastError();
    return fail(SPADE_ERR_UNSUPPORTED, "tensor-map encoder unavailable: no score-only estimator");
  }
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "estimate scores");
}

static spade_status check_select_args(const float* in, const float* tau_host, const int* cnt, const int* idx,
                                     int heads, int nb) {
  if (!in || !tau_host || !cnt || !idx) return fail(SPADE_ERR_INVALID, "null pointer");
  if (heads < 1 || heads > SPADE_SELECT_MAX_HEADS) return fail(SPADE_ERR_UNSUPPORTED, "heads=%d (1..1024)", heads);
  if (nb < 1) return fail(SPADE_ERR_INVALID, "nb=%d", nb);
  if (nb > SPADE_SELECT_MAX_NB) return fail(SPADE_ERR_UNSUPPORTED, "nb=%d above %d", nb, SPADE_SELECT_MAX_NB);
  for (int h = 0; h < heads; ++h)
    if (!(tau_host[h] > 0.f && tau_host[h] <= 1e30f)) return fail(SPADE_ERR_INVALID, "tau[%d] must be > 0", h);
  return SPADE_OK;
}

spade_status spade_select(const float* prob, const float* tau_host, int* cnt, int* idx, int heads, int nb,
                          spade_stream_t stream) {
  spade_status st = check_select_args(prob, tau_host, cnt, idx, heads, nb);
  if (st != SPADE_OK) return st;
  cudaError_t e = launch_select(prob, tau_host, cnt, idx, heads, nb, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "select");
}

spade_status spade_select_scores(const float* scores, const float* tau_host, int* cnt, int* idx, int heads, int nb,
                                 spade_stream_t stream) {
  spade_status st = check_select_args(scores, tau_host, cnt, idx, heads, nb);
  if (st != SPADE_OK) return st;
  cudaError_t e = launch_select(scores, tau_host, cnt, idx, heads, nb, as_cuda(stream), nullptr, nullptr, true);
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "select scores");
}

spade_status spade_select_window(const float* prob, const float* tau_host, const int* radius_host, spade_geom g,
                                 int* cnt, int* idx, int heads, spade_stream_t stream) {
  spade_status st = check_geom(g);
  if (st != SPADE_OK) return st;
  if (!prob || !tau_host || !radius_host || !cnt || !idx) return fail(SPADE_ERR_INVALID, "null pointer");
  if (heads < 1 || heads > SPADE_SELECT_MAX_HEADS) return fail(SPADE_ERR_UNSUPPORTED, "heads=%d (1..1024)", heads);
  const Geo gg = make_geo(g);
  if (gg.nb > SPADE_SELECT_MAX_NB) return fail(SPADE_ERR_UNSUPPORTED, "nb=%d above %d", gg.nb, SPADE_SELECT_MAX_NB);
  for (int h = 0; h < heads; ++h) {
    if (!(tau_host[h] > 0.f && tau_host[h] <= 1e30f)) return fail(SPADE_ERR_INVALID, "tau[%d] must be > 0", h);
    for (int a = 0; a < 3; ++a)
      if (radius_host[3 * h + a] < 0) return fail(SPADE_ERR_INVALID, "window radius of head %d is negative", h);
  }
  cudaError_t e = launch_select(prob, tau_host, cnt, idx, heads, gg.nb, as_cuda(stream), radius_host, &gg);
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "select");
}

size_t spade_attn_workspace_bytes(spade_geom g, int heads, int d, int text_tokens) {
  (void)d;
  if (heads < 1 || text_tokens < 0 || g.bt <= 0 || g.bh <= 0 || g.bw <= 0 || g.T <= 0 || g.H <= 0 || g.W <= 0)
    return 0;
  const Geo gg = make_geo(g);
  return align256((size_t)heads * (gg.nb + text_blocks(text_tokens)) * sizeof(int)) + 256;   // + ticket
}

spade_status spade_block_sparse_attn(const void* q, const void* k, const void* v, void* out, const int* cnt,
                                     const int* idx, spade_geom g, int heads, int d, int text_tokens,
                                     spade_dtype dt, void* workspace, size_t ws_bytes, spade_stream_t stream) {
  spade_status st = check_geom(g);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!q || !k || !v || !out) return fail(SPADE_ERR_INVALID, "null tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if ((cnt == nullptr) != (idx == nullptr)) return fail(SPADE_ERR_INVALID, "cnt and idx must both be set or both NULL");
  if (heads < 1 || heads > SPADE_MAX_HEADS) return fail(SPADE_ERR_UNSUPPORTED, "heads=%d (1..128)", heads);
  if (text_tokens < 0) return fail(SPADE_ERR_INVALID, "negative text_tokens");
  const size_t need = spade_attn_workspace_bytes(g, heads, d, text_tokens);
  if (!workspace || ws_bytes < need) return fail(SPADE_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v; a.out = out;
  a.n_schemes = 1;
  a.geo[0] = make_geo(g);
  a.heads = heads; a.d = d; a.text_tokens = text_tokens; a.N = g.T * g.H * g.W; a.dt = dt;
  const int nb = a.geo[0].nb;
  for (int h = 0; h < heads; ++h) {
    a.head[h].scheme = 0;
    a.head[h].nb = nb;
    a.head[h].dense = cnt == nullptr;
    a.head[h].cnt_off = h * nb;
    a.head[h].idx_off = (long long)h * nb * nb;
  }
  a.cnt = cnt; a.idx = idx;
  a.work = static_cast<int*>(workspace);
  a.n_items = heads * (nb + text_blocks(text_tokens));
  a.ticket = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + need - 256);
  if ((st = check_attention(a)) != SPADE_OK) return st;
  return run_attention(a, as_cuda(stream));
}

spade_status spade_block_sparse_attn_noalloc(const void* q, const void* k, const void* v, void* out,
                                             const int* cnt, const int* idx, spade_geom g, int heads, int d,
                                             int text_tokens, spade_dtype dt, spade_stream_t stream) {
  spade_status st = check_geom(g);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!q || !k || !v || !out) return fail(SPADE_ERR_INVALID, "null tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if ((cnt == nullptr) != (idx == nullptr)) return fail(SPADE_ERR_INVALID, "cnt and idx must both be set or both NULL");
  if (heads < 1 || heads > SPADE_MAX_HEADS) return fail(SPADE_ERR_UNSUPPORTED, "heads=%d (1..128)", heads);
  if (text_tokens < 0) return fail(SPADE_ERR_INVALID, "negative text_tokens");
  const int nb = make_geo(g).nb;
  const long long n_items = (long long)heads * (nb + text_blocks(text_tokens));
  if (n_items > SPADE_NOALLOC_MAX_ITEMS)
    return fail(SPADE_ERR_UNSUPPORTED, "heads * (blocks + text blocks) = %lld exceeds the fixed scratch of %d work items",
                n_items, SPADE_NOALLOC_MAX_ITEMS);
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v; a.out = out;
  a.n_schemes = 1;
  a.geo[0] = make_geo(g);
  a.heads = heads; a.d = d; a.text_tokens = text_tokens; a.N = g.T * g.H * g.W; a.dt = dt;
  for (int h = 0; h < heads; ++h) {
    a.head[h].scheme = 0;
    a.head[h].nb = nb;
    a.head[h].dense = cnt == nullptr;
    a.head[h].cnt_off = h * nb;
    a.head[h].idx_off = (long long)h * nb * nb;
  }
  a.cnt = cnt; a.idx = idx;
  a.n_items = (int)n_items;
  if ((st = check_attention(a)) != SPADE_OK) return st;
  int* scratch = noalloc_scratch(&st);
  if (!scratch) return st;
  a.work = scratch;                                   // written in full by the work-list kernel
  a.ticket = scratch + SPADE_NOALLOC_MAX_ITEMS;       // reset to 0 by the work-list kernel
  return run_attention(a, as_cuda(stream));
}

size_t spade_grouped_workspace_bytes(const spade_geom* schemes, int n_schemes, const spade_head_scheme* table,
                                     int heads, int d, int text_tokens) {
  GroupLayout L;
  if (plan_group(schemes, n_schemes, table, heads, d, text_tokens, L) != SPADE_OK) return 0;
  return L.total;
}

spade_status spade_copy_head_slice(void* device, void* host, int64_t rows, int heads_total, int h0, int hc, int d,
                                   spade_dtype dt, int to_device, spade_stream_t stream) {
  if (!device || !host) return fail(SPADE_ERR_INVALID, "null pointer");
  if (rows < 1 || heads_total < 1 || d < 1 || h0 < 0 || hc < 1 || h0 + hc > heads_total)
    return fail(SPADE_ERR_INVALID, "slice [%d, %d) of %d heads, %lld rows", h0, h0 + hc, heads_total, (long long)rows);
  if (dt != SPADE_F32 && dt != SPADE_BF16) return fail(SPADE_ERR_INVALID, "unknown dtype %d", (int)dt);
  const size_t esz = dt == SPADE_BF16 ? 2 : 4;
  const size_t hpitch = (size_t)heads_total * d * esz, dpitch = (size_t)hc * d * esz;
  char* hp = static_cast<char*>(host) + (size_t)h0 * d * esz;
  cudaError_t e = to_device
                      ? cudaMemcpy2DAsync(device, dpitch, hp, hpitch, dpitch, (size_t)rows, cudaMemcpyHostToDevice,
                                          as_cuda(stream))
                      : cudaMemcpy2DAsync(hp, hpitch, device, dpitch, dpitch, (size_t)rows, cudaMemcpyDeviceToHost,
                                          as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "copy_head_slice");
}

size_t spade_sics_workspace_bytes(const spade_geom* candidates, int n_candidates, int heads) {
  if (!candidates || n_candidates < 1 || n_candidates > SPADE_MAX_SCHEMES || heads < 1) return 0;
  Geo g[SPADE_MAX_SCHEMES];
  for (int c = 0; c < n_candidates; ++c) g[c] = make_geo(candidates[c]);
  return sics_workspace_floats(g, n_candidates, heads) * sizeof(float);
}

spade_status spade_sics(const void* q, const void* k, const spade_geom* candidates, int n_candidates, int heads,
                        int d, spade_dtype dt, float* scores, int* choice, void* workspace, size_t ws_bytes,
                        spade_stream_t stream) {
  if (!q || !k || !candidates || !scores || !choice || !workspace) return fail(SPADE_ERR_INVALID, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(workspace))
    return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (n_candidates < 1 || n_candidates > SPADE_MAX_SCHEMES)
    return fail(SPADE_ERR_INVALID, "n_candidates=%d (1..%d)", n_candidates, SPADE_MAX_SCHEMES);
  if (heads < 1 || heads > 1024) return fail(SPADE_ERR_INVALID, "heads=%d", heads);
  spade_status st = check_d_dt(d, dt);
  if (st != SPADE_OK) return st;
  Geo g[SPADE_MAX_SCHEMES];
  for (int c = 0; c < n_candidates; ++c) {
    if ((st = check_geom(candidates[c])) != SPADE_OK) return st;
    if ((long long)candidates[c].T * candidates[c].H * candidates[c].W !=
        (long long)candidates[0].T * candidates[0].H * candidates[0].W)
      return fail(SPADE_ERR_INVALID, "candidate %d covers a different number of tokens", c);
    g[c] = make_geo(candidates[c]);
  }
  const size_t need = sics_workspace_floats(g, n_candidates, heads) * sizeof(float);
  if (ws_bytes < need) return fail(SPADE_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  cudaError_t e = launch_sics(q, k, g, n_candidates, heads, d, dt, static_cast<float*>(workspace), scores, choice,
                              as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "sics");
}

spade_status spade_grouped_head_lists(const spade_geom* schemes, int n_schemes, const spade_head_scheme* table,
                                      int heads, int d, int text_tokens, int head, int64_t* cnt_offset,
                                      int64_t* idx_offset) {
  GroupLayout L;
  spade_status st = plan_group(schemes, n_schemes, table, heads, d, text_tokens, L);
  if (st != SPADE_OK) return st;
  if (head < 0 || head >= heads || !cnt_offset || !idx_offset) return fail(SPADE_ERR_INVALID, "head/outputs");
  if (table[head].dense) { *cnt_offset = -1; *idx_offset = -1; return SPADE_OK; }
  const int s = table[head].scheme;
  const Geo g = make_geo(schemes[s]);
  *cnt_offset = (int64_t)(L.cnt[s] + (size_t)L.pos[head] * g.nb * sizeof(int));
  *idx_offset = (int64_t)(L.idx[s] + (size_t)L.pos[head] * g.nb * g.nb * sizeof(int));
  return SPADE_OK;
}

spade_status spade_grouped_attn(const void* q, const void* k, const void* v, void* out, const spade_geom* schemes,
                                int n_schemes, const spade_head_scheme* table, int heads, int d, int text_tokens,
                                spade_dtype dt, void* workspace, size_t ws_bytes, spade_stream_t stream) {
  return spade_grouped_attn_ex(q, k, v, out, schemes, n_schemes, table, heads, d, text_tokens, dt, SPADE_SUM_MEAN,
                               SPADE_SUM_MEAN, nullptr, workspace, ws_bytes, stream);
}

spade_status spade_grouped_attn_ex(const void* q, const void* k, const void* v, void* out, const spade_geom* schemes,
                                   int n_schemes, const spade_head_scheme* table, int heads, int d, int text_tokens,
                                   spade_dtype dt, spade_summary q_summary, spade_summary k_summary,
                                   const int* window_radius, void* workspace, size_t ws_bytes,
                                   spade_stream_t stream) {
  if (window_radius)
    for (int h = 0; h < heads; ++h)
      for (int a = 0; a < 3; ++a)
        if (window_radius[3 * h + a] < 0) return fail(SPADE_ERR_INVALID, "window radius of head %d is negative", h);
  if ((q_summary != SPADE_SUM_MEAN && q_summary != SPADE_SUM_MAX && q_summary != SPADE_SUM_MIN) ||
      (k_summary != SPADE_SUM_MEAN && k_summary != SPADE_SUM_MAX && k_summary != SPADE_SUM_MIN))
    return fail(SPADE_ERR_INVALID, "summary modes %d/%d", (int)q_summary, (int)k_summary);
  GroupLayout L;
  spade_status st = plan_group(schemes, n_schemes, table, heads, d, text_tokens, L);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!q || !k || !v || !out) return fail(SPADE_ERR_INVALID, "null tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace))
    return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (!workspace || ws_bytes < L.total) return fail(SPADE_ERR_WORKSPACE, "workspace needs %zu bytes", L.total);
  cudaStream_t s = as_cuda(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  // the attention launch of step 5, set up (and checked) before anything is enqueued
  AttnArgs a;
  grouped_attn_args(q, k, v, out, schemes, n_schemes, table, heads, d, text_tokens, dt, L, ws, a);
  if ((st = check_attention(a)) != SPADE_OK) return st;
  // steps 1-4 per scheme, for its non-dense heads
  for (int sc = 0; sc < n_schemes; ++sc) {
    const int hs = L.n_sparse[sc];
    if (hs == 0) continue;
    const Geo g = make_geo(schemes[sc]);
    float* qm = reinterpret_cast<float*>(ws + L.qmean[sc]);
    float* km = reinterpret_cast<float*>(ws + L.kmean[sc]);
    const std::vector<int>& hl = L.heads_of[sc];
    for (int i = 0; i < hs;) {                        // contiguous runs of heads
      int j = i + 1;
      while (j < hs && hl[j] == hl[j - 1] + 1) ++j;
      const size_t o = (size_t)i * g.nb * d;
      cudaError_t e;
      if (q_summary == k_summary) {               // Q and K in one launch
        e = launch_summarize_pair(q, k, qm + o, km + o, g, heads, hl[i], j - i, d, dt, (int)q_summary, s);
      } else {
        e = launch_summarize(q, qm + o, g, heads, hl[i], j - i, d, dt, (int)q_summary, s);
        if (e == cudaSuccess) e = launch_summarize(k, km + o, g, heads, hl[i], j - i, d, dt, (int)k_summary, s);
      }
      if (e != cudaSuccess) return cuda_fail(e, "summarize");
      i = j;
    }
    std::vector<float> taus(hs);
    std::vector<int> rad(3 * hs, 0);
    for (int i = 0; i < hs; ++i) {
      taus[i] = table[hl[i]].tau;
      if (window_radius)
        for (int a = 0; a < 3; ++a) rad[3 * i + a] = window_radius[3 * hl[i] + a];
    }
    int* cnt_s = reinterpret_cast<int*>(ws + L.cnt[sc]);
    int* idx_s = reinterpret_cast<int*>(ws + L.idx[sc]);
    float* prob = reinterpret_cast<float*>(ws + L.prob[sc]);
    int* st = status_ptr();
    if (!st) return fail(SPADE_ERR_CUDA, "device status word unavailable");
    bool scores = false;
    cudaError_t e = run_estimate(qm, km, prob, hs, g.nb, d, st, false, &scores, s);
    if (e != cudaSuccess) return cuda_fail(e, "estimate");
    e = launch_select(prob, taus.data(), cnt_s, idx_s, hs, g.nb, s, window_radius ? rad.data() : nullptr, &g, scores);
    if (e != cudaSuccess) return cuda_fail(e, "select");
  }
  // step 5: one grouped launch over every head
  return run_attention(a, s);
}

spade_status spade_grouped_attn_lists(const void* q, const void* k, const void* v, void* out,
                                      const spade_geom* schemes, int n_schemes, const spade_head_scheme* table,
                                      int heads, int d, int text_tokens, spade_dtype dt, void* workspace,
                                      size_t ws_bytes, spade_stream_t stream) {
  GroupLayout L;
  spade_status st = plan_group(schemes, n_schemes, table, heads, d, text_tokens, L);
  if (st != SPADE_OK) return st;
  if ((st = check_d_dt(d, dt)) != SPADE_OK) return st;
  if (!q || !k || !v || !out) return fail(SPADE_ERR_INVALID, "null tensor pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace))
    return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  if (!workspace || ws_bytes < L.total) return fail(SPADE_ERR_WORKSPACE, "workspace needs %zu bytes", L.total);
  AttnArgs a;
  grouped_attn_args(q, k, v, out, schemes, n_schemes, table, heads, d, text_tokens, dt, L,
                    static_cast<uint8_t*>(workspace), a);
  if ((st = check_attention(a)) != SPADE_OK) return st;
  return run_attention(a, as_cuda(stream));
}

size_t spade_grouped_host_workspace_bytes(const spade_geom* schemes, int n_schemes, const spade_head_scheme* table,
                                          int heads, int d, int text_tokens, spade_dtype dt, int head_chunk) {
  HostLayout H;
  if (plan_host(schemes, n_schemes, table, heads, d, text_tokens, dt, head_chunk, H) != SPADE_OK) return 0;
  return H.total;
}

spade_status spade_grouped_attn_host(const void* q_host, const void* k_host, const void* v_host, void* out_host,
                                     const spade_geom* schemes, int n_schemes, const spade_head_scheme* table,
                                     int heads, int d, int text_tokens, spade_dtype dt, int head_chunk,
                                     void* workspace, size_t ws_bytes, spade_stream_t stream) {
  HostLayout H;
  spade_status st = plan_host(schemes, n_schemes, table, heads, d, text_tokens, dt, head_chunk, H);
  if (st != SPADE_OK) return st;
  if (!q_host || !k_host || !v_host || !out_host) return fail(SPADE_ERR_INVALID, "null host pointer");
  if (!workspace || ws_bytes < H.total) return fail(SPADE_ERR_WORKSPACE, "workspace needs %zu bytes", H.total);
  if (!aligned16(workspace)) return fail(SPADE_ERR_INVALID, "pointers must be 16-byte aligned");
  // every group's grouped call is checked before anything is enqueued
  const int N = schemes[0].T * schemes[0].H * schemes[0].W;
  for (int g = 0; g < H.n_groups; ++g) {
    const int h0 = g * head_chunk, hc = std::min(head_chunk, heads - h0);
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    a.n_schemes = n_schemes;
    for (int sc = 0; sc < n_schemes; ++sc) a.geo[sc] = make_geo(schemes[sc]);
    a.heads = hc; a.d = d; a.text_tokens = text_tokens; a.N = N; a.dt = dt;
    for (int h = 0; h < hc; ++h) {
      a.head[h].scheme = table[h0 + h].scheme;
      a.head[h].nb = a.geo[table[h0 + h].scheme].nb;
      a.head[h].dense = table[h0 + h].dense;
    }
    if ((st = check_attention(a)) != SPADE_OK) return st;
  }
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return fail(SPADE_ERR_CUDA, "no current CUDA device");
  HostPipe& P = host_pipe(dev);
  std::lock_guard<std::mutex> lock(P.mu);
  const int G = H.n_groups, ns = std::min(kHostSlots, G);
  cudaError_t e = host_pipe_setup(P, (size_t)3 * G + 1 + 2 + kHostComputes);
  if (e != cudaSuccess) return cuda_fail(e, "stream/event set-up");
  cudaEvent_t* loaded = P.ev.data();
  cudaEvent_t* done = loaded + G;
  cudaEvent_t* returned = done + G;
  cudaEvent_t* joins = returned + G;            // [0] entry, [1] up, [2] down, [3..] computes
  const cudaStream_t caller = as_cuda(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t rows = (int64_t)N + text_tokens;
  const void* src[3] = {q_host, k_host, v_host};
  // everything below is ordered after the caller's stream at this point
  if ((e = cudaEventRecord(joins[0], caller)) != cudaSuccess) return cuda_fail(e, "event record");
  cudaStreamWaitEvent(P.up, joins[0], 0);
  cudaStreamWaitEvent(P.down, joins[0], 0);
  for (int c = 0; c < kHostComputes; ++c) cudaStreamWaitEvent(P.comp[c], joins[0], 0);
  auto slot_buf = [&](int g, int which) { return ws + ((size_t)(g % ns) * 4 + which) * H.slot_bytes; };
  auto load = [&](int g) -> spade_status {
    const int h0 = g * head_chunk, hc = std::min(head_chunk, heads - h0);
    if (g >= ns) cudaStreamWaitEvent(P.up, returned[g - ns], 0);   // the slot's previous group is back
    for (int t = 0; t < 3; ++t) {
      spade_status s2 = spade_copy_head_slice(slot_buf(g, t), const_cast<void*>(src[t]), rows, heads, h0, hc, d, dt,
                                              1, reinterpret_cast<spade_stream_t>(P.up));
      if (s2 != SPADE_OK) return s2;
    }
    const cudaError_t e2 = cudaEventRecord(loaded[g], P.up);
    return e2 == cudaSuccess ? SPADE_OK : cuda_fail(e2, "event record");
  };
  for (int g = 0; g < ns - 1; ++g)
    if ((st = load(g)) != SPADE_OK) return st;
  for (int g = 0; g < G; ++g) {
    if (g + ns - 1 < G && (st = load(g + ns - 1)) != SPADE_OK) return st;
    const int h0 = g * head_chunk, hc = std::min(head_chunk, heads - h0);
    const cudaStream_t comp = P.comp[g % kHostComputes];
    cudaStreamWaitEvent(comp, loaded[g], 0);
    st = spade_grouped_attn(slot_buf(g, 0), slot_buf(g, 1), slot_buf(g, 2), slot_buf(g, 3), schemes, n_schemes,
                            table + h0, hc, d, text_tokens, dt, ws + H.ws_off + (size_t)(g % kHostComputes) * H.ws_bytes,
                            H.ws_bytes, reinterpret_cast<spade_stream_t>(comp));
    if (st != SPADE_OK) return st;
    if ((e = cudaEventRecord(done[g], comp)) != cudaSuccess) return cuda_fail(e, "event record");
    cudaStreamWaitEvent(P.down, done[g], 0);
    st = spade_copy_head_slice(slot_buf(g, 3), out_host, rows, heads, h0, hc, d, dt, 0,
                               reinterpret_cast<spade_stream_t>(P.down));
    if (st != SPADE_OK) return st;
    if ((e = cudaEventRecord(returned[g], P.down)) != cudaSuccess) return cuda_fail(e, "event record");
  }
  // the caller's stream waits for every stream of the call
  cudaEventRecord(joins[1], P.up);
  cudaEventRecord(joins[2], P.down);
  cudaStreamWaitEvent(caller, joins[1], 0);
  cudaStreamWaitEvent(caller, joins[2], 0);
  for (int c = 0; c < kHostComputes; ++c) {
    cudaEventRecord(joins[3 + c], P.comp[c]);
    cudaStreamWaitEvent(caller, joins[3 + c], 0);
  }
  e = cudaGetLastError();
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "host-to-host layer");
}

// ---- row passes around the attention ----

spade_status spade_rope_axes(spade_rope* rope, const int32_t pairs[3], const double theta[3], const double scale[3],
                             spade_rope_style style, int shared_ladder) {
  if (!rope || !pairs || !theta || !scale) return fail(SPADE_ERR_INVALID, "null pointer");
  if (style != SPADE_ROPE_INTERLEAVED && style != SPADE_ROPE_HALF)
    return fail(SPADE_ERR_INVALID, "rotation style %d", (int)style);
  long long total = 0;
  for (int a = 0; a < 3; ++a) {
    if (pairs[a] < 0) return fail(SPADE_ERR_INVALID, "axis %d: %d pairs", a, pairs[a]);
    if (!(theta[a] > 0.0) || !std::isfinite(theta[a]) || !std::isfinite(scale[a]))
      return fail(SPADE_ERR_INVALID, "axis %d: theta %g, scale %g", a, theta[a], scale[a]);
    total += pairs[a];
  }
  if (total > SPADE_ROPE_MAX_PAIRS)
    return fail(SPADE_ERR_UNSUPPORTED, "%lld rotated pairs (up to %d)", total, SPADE_ROPE_MAX_PAIRS);
  spade_rope r;
  memset(&r, 0, sizeof(r));
  r.style = style;
  for (int a = 0; a < 3; ++a)
    for (int i = 0; i < pairs[a]; ++i) {
      const double base = shared_ladder ? theta[0] : theta[a];
      const double at = shared_ladder ? (double)r.pairs / (double)total : (double)i / (double)pairs[a];
      r.axis[r.pairs] = a;
      r.freq[r.pairs] = scale[a] * pow(base, -at);
      ++r.pairs;
    }
  *rope = r;
  return SPADE_OK;
}

size_t spade_qk_norm_rope_bwd_workspace_bytes(const spade_qk_desc* desc) {
  QkArgs a;
  if (plan_qk(desc, nullptr, nullptr, a) != SPADE_OK) return 0;
  return a.rows ? qk_bwd_floats(a) * sizeof(float) : 0;
}

spade_status spade_qk_norm_rope(const spade_qk_desc* desc, const spade_rope* rope, const int32_t* positions,
                                const void* q, const void* k, const void* q_weight, const void* k_weight, void* q_out,
                                void* k_out, spade_stream_t stream) {
  if (!rope) return fail(SPADE_ERR_INVALID, "null rotation");
  QkArgs a;
  spade_status st = plan_qk(desc, rope, positions, a);
  if (st != SPADE_OK) return st;
  const void* x[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const void* w[2] = {q_weight, k_weight};
  if ((st = bind_qk(desc, a, x, nullptr, w, out, nullptr, nullptr, 0)) != SPADE_OK) return st;
  if (!a.rows) return SPADE_OK;
  const cudaError_t e = launch_qk_fwd(a, desc->dt == SPADE_BF16, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "qk_norm_rope");
}

spade_status spade_qk_norm_rope_bwd(const spade_qk_desc* desc, const spade_rope* rope, const int32_t* positions,
                                    const void* dq_out, const void* dk_out, const void* q, const void* k,
                                    const void* q_weight, const void* k_weight, void* dq, void* dk, float* dq_weight,
                                    float* dk_weight, void* workspace, size_t ws_bytes, spade_stream_t stream) {
  if (!rope) return fail(SPADE_ERR_INVALID, "null rotation");
  QkArgs a;
  spade_status st = plan_qk(desc, rope, positions, a);
  if (st != SPADE_OK) return st;
  const bool normed = a.norm != SPADE_QK_NORM_NONE;
  const void* x[2] = {normed ? q : nullptr, normed ? k : nullptr};
  const void* dout[2] = {dq_out, dk_out};
  void* out[2] = {dq, dk};
  const void* w[2] = {q_weight, k_weight};
  float* dw[2] = {dq_weight, dk_weight};
  if (!normed && (dq_weight || dk_weight)) return fail(SPADE_ERR_INVALID, "weight gradient without a norm");
  const size_t need = (dq_weight || dk_weight) && a.rows ? qk_bwd_floats(a) * sizeof(float) : 0;
  if ((st = check_scratch(workspace, ws_bytes, need)) != SPADE_OK) return st;
  if ((st = bind_qk(desc, a, x, dout, w, out, dw, workspace, need)) != SPADE_OK) return st;
  const cudaStream_t s = as_cuda(stream);
  if (!a.rows) {
    for (int t = 0; t < 2; ++t)
      if (dw[t]) {
        const cudaError_t e = cudaMemsetAsync(dw[t], 0, sizeof(float) * qk_weight_len(a, t), s);
        if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope_bwd");
      }
    return SPADE_OK;
  }
  if (need) a.part = static_cast<float*>(workspace);
  const cudaError_t e = launch_qk_bwd(a, desc->dt == SPADE_BF16, s);
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "qk_norm_rope_bwd");
}

spade_status spade_norm_modulate(const spade_row_desc* desc, const spade_row_params* params, const void* x, void* h,
                                 spade_stream_t stream) {
  return run_row_fwd(desc, params, x, nullptr, nullptr, h, false, true, as_cuda(stream), "norm_modulate");
}

spade_status spade_gate_residual(const spade_row_desc* desc, const spade_row_params* params, const void* x,
                                 const void* y, void* x_out, spade_stream_t stream) {
  return run_row_fwd(desc, params, x, y, x_out, nullptr, true, false, as_cuda(stream), "gate_residual");
}

spade_status spade_gate_residual_norm(const spade_row_desc* desc, const spade_row_params* params, const void* x,
                                      const void* y, void* x_out, void* h, spade_stream_t stream) {
  return run_row_fwd(desc, params, x, y, x_out, h, true, true, as_cuda(stream), "gate_residual_norm");
}

size_t spade_row_bwd_workspace_bytes(const spade_row_desc* desc) {
  RowArgs a;
  if (plan_row(desc, nullptr, true, a) != SPADE_OK || !a.rows) return 0;
  return plan_row_bwd(a.rows, a.groups, a.dim, true).floats * sizeof(float);
}

spade_status spade_norm_modulate_bwd(const spade_row_desc* desc, const spade_row_params* params, const void* dh,
                                     const void* dres, const void* x, void* dx, const spade_row_grads* grads,
                                     void* workspace, size_t ws_bytes, spade_stream_t stream) {
  return run_row_bwd(desc, params, dres, dh, x, nullptr, dx, nullptr, grads, workspace, ws_bytes, false, true,
                     as_cuda(stream), "norm_modulate_bwd");
}

spade_status spade_gate_residual_bwd(const spade_row_desc* desc, const spade_row_params* params, const void* dx_out,
                                     const void* y, void* dy, const spade_row_grads* grads, void* workspace,
                                     size_t ws_bytes, spade_stream_t stream) {
  return run_row_bwd(desc, params, dx_out, nullptr, nullptr, y, nullptr, dy, grads, workspace, ws_bytes, true, false,
                     as_cuda(stream), "gate_residual_bwd");
}

spade_status spade_gate_residual_norm_bwd(const spade_row_desc* desc, const spade_row_params* params,
                                          const void* dx_out, const void* dh, const void* x, const void* y, void* dx,
                                          void* dy, const spade_row_grads* grads, void* workspace, size_t ws_bytes,
                                          spade_stream_t stream) {
  return run_row_bwd(desc, params, dx_out, dh, x, y, dx, dy, grads, workspace, ws_bytes, true, true, as_cuda(stream),
                     "gate_residual_norm_bwd");
}

spade_status spade_last_device_status(spade_stream_t stream) {
  cudaError_t e = cudaStreamSynchronize(as_cuda(stream));
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  int v = 0;
  e = cudaMemcpyFromSymbol(&v, g_spade_status, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "read status");
  const int zero = 0;
  e = cudaMemcpyToSymbol(g_spade_status, &zero, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "clear status");
  return static_cast<spade_status>(v);
}

spade_status spade_selftest_bounded_wait(int64_t timeout_ns, spade_stream_t stream) {
  if (timeout_ns <= 0 || timeout_ns > 10000000000LL) return fail(SPADE_ERR_INVALID, "timeout_ns out of range");
  int* sp = status_ptr();
  if (!sp) return fail(SPADE_ERR_CUDA, "device status word unavailable");
  cudaError_t e = launch_bounded_wait_selftest(sp, timeout_ns, as_cuda(stream));
  return e == cudaSuccess ? SPADE_OK : cuda_fail(e, "bounded-wait self test");
}

}  // extern "C"
