// Internal interface between the C-ABI layer (spade_api.cu) and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spade.h"

#define SPADE_MAX_SCHEMES 4
#define SPADE_MAX_HEADS 128
#define SPADE_ROW_MAX_DIM 16384
#define SPADE_SELECT_MAX_NB 1024
#define SPADE_SELECT_MAX_HEADS 1024
#define SPADE_ESTIMATE_MAX_NB 2048
#define SPADE_WORKLIST_MAX_COST 4096
#define SPADE_TC_MAX_LIST 1280   // tensor-core path: key blocks per item (nb + text blocks)

namespace spade {

// Geometry of one blocking scheme, with derived block counts.
struct Geo {
  int T, H, W, bt, bh, bw;
  int nbt, nbh, nbw, nb, bs;
};

__host__ __device__ inline int cdiv(int a, int b) { return (a + b - 1) / b; }

__host__ __device__ inline Geo make_geo(const spade_geom& g) {
  Geo r;
  r.T = g.T; r.H = g.H; r.W = g.W; r.bt = g.bt; r.bh = g.bh; r.bw = g.bw;
  r.nbt = cdiv(g.T, g.bt); r.nbh = cdiv(g.H, g.bh); r.nbw = cdiv(g.W, g.bw);
  r.nb = r.nbt * r.nbh * r.nbw;
  r.bs = g.bt * g.bh * g.bw;
  return r;
}

// Origin (t0, y0, x0) and clipped extents (et, eh, ew) of block b.
__host__ __device__ inline void block_box(const Geo& g, int b, int& t0, int& y0, int& x0, int& et, int& eh,
                                          int& ew) {
  const int bk = b % g.nbw;
  const int bj = (b / g.nbw) % g.nbh;
  const int bi = b / (g.nbw * g.nbh);
  t0 = bi * g.bt; y0 = bj * g.bh; x0 = bk * g.bw;
  et = min(g.bt, g.T - t0); eh = min(g.bh, g.H - y0); ew = min(g.bw, g.W - x0);
}

// Per-head row of the attention launch.
struct HeadInfo {
  int scheme;      // index into the launch's scheme table
  int nb;          // blocks of that scheme
  int dense;       // attends every key block
  int cnt_off;     // element offset of this head's cnt[nb] from AttnArgs::cnt
  long long idx_off;  // element offset of this head's idx[nb][nb] from AttnArgs::idx
};

// Everything an attention launch needs (both kernel paths).
struct AttnArgs {
  const void* q; const void* k; const void* v; void* out;
  int n_schemes;
  Geo geo[SPADE_MAX_SCHEMES];
  int heads;           // total heads in the Q/K/V layout
  int d;
  int text_tokens;
  int N;               // video tokens = T*H*W (same for every scheme)
  HeadInfo head[SPADE_MAX_HEADS];
  const int* cnt;      // base of the kept counts
  const int* idx;      // base of the kept ids
  int* work;           // [n_items] work list (built on device)
  int* ticket;         // one int next to the work list: dynamic work hand-out
  int n_items;
  spade_dtype dt;
  int* status;         // device status word
};

// Items per head: one per query block of the head's scheme, plus the text
// query blocks (128 text tokens each).
__host__ __device__ inline int text_blocks(int text_tokens) { return (text_tokens + 127) / 128; }

// ---- launchers (return the CUDA error of the launch) ----
cudaError_t launch_tile3d(const void* x, void* xt, const Geo& g, int heads, int d, spade_dtype dt,
                          cudaStream_t s);
cudaError_t launch_summarize(const void* x, float* out, const Geo& g, int heads_total, int h0, int hc, int d,
                             spade_dtype dt, int mode, cudaStream_t s);
// Q and K with the same reduce, in one launch.
cudaError_t launch_summarize_pair(const void* q, const void* k, float* qout, float* kout, const Geo& g,
                                  int heads_total, int h0, int hc, int d, spade_dtype dt, int mode, cudaStream_t s);
// probs = false: out = the scaled pooled scores; true: their row softmax.
cudaError_t launch_estimate_tc(const float* qm, const float* km, float* out, int heads, int nb, int d, int* status,
                               bool probs, cudaStream_t s);
cudaError_t launch_estimate(const float* qm, const float* km, float* prob, int heads, int nb, int d,
                            cudaStream_t s);
// scores = true: `in` holds scaled pooled scores and the kernel forms the
// softmax itself; false: `in` holds probabilities.
cudaError_t launch_select(const float* in, const float* tau_host, int* cnt, int* idx, int heads, int nb,
                          cudaStream_t s, const int* radius_host = nullptr, const Geo* g = nullptr,
                          bool scores = false);
cudaError_t launch_worklist(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_simt(const AttnArgs& a, cudaStream_t s);
// Returns cudaErrorNotSupported if the shape is not for the tensor-core path.
bool attn_tc_supported(const AttnArgs& a);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s, const char** why);
cudaError_t launch_bounded_wait_selftest(int* status, long long timeout_ns, cudaStream_t s);
size_t sics_workspace_floats(const Geo* cand, int n_cand, int heads);
cudaError_t launch_sics(const void* q, const void* k, const Geo* cand, int n_cand, int heads, int d, spade_dtype dt,
                        float* ws, float* scores, int* choice, cudaStream_t s);

// One row pass of the residual stream (k_row.cu).  Null pointers: no
// such operand (parameters: the identity); strides in elements.
struct RowArgs {
  long long rows, groups, rows_per_group, chunks;
  int dim, norm, post_norm;
  float eps, post_eps, residual_scale, inv_dim;
  bool x_bf16, branch_bf16, param_bf16;
  const void *x, *y;                                  // forward inputs (x also backward)
  void *x_out, *h;                                    // forward outputs
  const void *dx_out, *dh;                            // gradients coming in
  void *dx, *dy;                                      // gradients going out
  const void *gate, *post_weight, *weight, *bias, *scale, *shift;
  float *dgate, *dpost_weight, *dweight, *dbias, *dscale, *dshift;
  long long x_stride, y_stride, x_out_stride, h_stride, dx_out_stride, dh_stride, dx_stride, dy_stride;
  long long gate_stride, scale_stride, shift_stride;
  float* part;                                        // column sums of the backward units
};
struct RowPlan {
  long long chunks;     // units a modulation group is cut into
  int grid;
  size_t floats;        // workspace
};
RowPlan plan_row_bwd(long long rows, long long groups, int dim, bool weights);
cudaError_t launch_row_fwd(const RowArgs& a, cudaStream_t s);
cudaError_t launch_row_bwd(const RowArgs& a, int grid, cudaStream_t s);

// Norm and rotation of Q and K (k_qk_rope.cu).  Index 0 is Q, 1 is K; a
// tensor without heads is absent.
struct QkArgs {
  long long rows, video_rows;
  struct Divisor {                 // n / by = n * mul >> shift for n below 2^31
    unsigned by, mul, shift;
  };
  int tok0;                        // grid token of row 0 (no positions given)
  Divisor H, W;
  int heads[2], d, lanes;          // lanes: threads per head, a power of two
  int norm;
  float eps;
  float inv_count[2];              // 1 / the values that a norm runs over
  bool weight_bf16, half;
  const void* x[2];                // raw rows
  const void* dout[2];             // backward: gradient coming in
  void* out[2];                    // forward: result; backward: gradient going out
  const void* weight[2];
  float* dweight[2];
  long long x_stride[2], dout_stride[2], out_stride[2];
  const int* positions;            // [rows, 3] or null
  float* part;
  int pairs;
  uint8_t axis[SPADE_ROPE_MAX_PAIRS];
  double turn[SPADE_ROPE_MAX_PAIRS];   // turns per unit of position
};
size_t qk_bwd_floats(const QkArgs& a);
cudaError_t launch_qk_fwd(const QkArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_qk_bwd(const QkArgs& a, bool bf16, cudaStream_t s);

int num_sms();                               // SM count of the current device
long long device_wait_timeout_ns();          // limit for every bounded device wait

}  // namespace spade
