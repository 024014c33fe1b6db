// Row passes of the residual stream around a block: the norm with modulation
// that opens it, the gated update that ends it, both in one pass, and their
// gradients (spade_norm_modulate, spade_gate_residual,
// spade_gate_residual_norm and the _bwd calls).
//
//   x' = x + r * gate_g * P(y)          P: none, rms or layer norm * weight
//   h  = (N(x') * w + b) * (1 + scale_g) + shift_g
//
// with g the row's modulation group.  Backward, with A_g = sum of dh and
// B_g = sum of dh * xhat over the rows of group g, C_g = sum of dx' * yhat:
//   dshift = A, dscale = w B + b A, dw = sum_g (1 + scale_g) B_g,
//   db = sum_g (1 + scale_g) A_g, dgate = r pw C, dpw = r sum_g gate_g C_g,
// so three column sums serve every parameter, and
//   u = dh (1 + scale) w,  dx = dx' + rstd (u - mean(u) - xhat mean(u xhat))
// (the mean(u) term for the layer norm only), dy likewise through P.
//
// One block per row at a time, every thread owning the same columns of every
// row it meets, so the modulation stays in registers while the group lasts
// and the column sums of the backward pass stay in registers until a
// (group, chunk of rows) unit ends.  A unit's sums go to the workspace and a
// second small launch adds them in a fixed order, in float64: no atomics, the
// same result on every run.  All passes are bound by memory: each row is read
// and written once.
#include "row_io.cuh"
#include "spade_internal.cuh"

namespace spade {
namespace {

using namespace rowio;

enum { kNone = SPADE_NORM_NONE, kRms = SPADE_NORM_RMS, kLayer = SPADE_NORM_LAYER };

// Which columns a thread owns: vectors of eight neighbours, or (rows whose
// length, stride or address does not allow 16-byte accesses) single columns a
// block apart.
template <bool VEC>
__device__ __forceinline__ int column(int i, int e) {
  return VEC ? ((i * (int)blockDim.x + (int)threadIdx.x) * 8 + e)
             : ((i * 8 + e) * (int)blockDim.x + (int)threadIdx.x);
}

template <bool VEC, typename T>
__device__ __forceinline__ void load_row(float (&v)[8], const T* p, int i, int dim) {
  if (VEC) {
    const int c = column<true>(i, 0);
    Raw8<T> r;
    if (c < dim) load_raw(r, p + c);
    else clear_raw(r);
    unpack(v, r);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(i, e);
      v[e] = c < dim ? to_float(p[c]) : 0.f;
    }
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[8], int i, int dim) {
  if (VEC) {
    const int c = column<true>(i, 0);
    if (c < dim) store_vec(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(i, e);
      if (c < dim) store_one(p + c, v[e]);
    }
  }
}
// A parameter row in either type; absent ones read as `none`.
template <bool VEC>
__device__ __forceinline__ void load_param(float (&v)[8], const void* p, long long off, bool bf16, float none, int i,
                                           int dim) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = none;
  } else if (bf16) {
    load_row<VEC>(v, static_cast<const __nv_bfloat16*>(p) + off, i, dim);
  } else {
    load_row<VEC>(v, static_cast<const float*>(p) + off, i, dim);
  }
}

struct Shared {
  SumScratch<2> sum;
  float2 moment[2][32];
  float count[32];     // columns each warp owns
};

// Mean (0 for the rms norm) and reciprocal deviation of a row held in
// registers.  The layer norm's second moment is taken about each warp's own
// mean and the warps' moments are merged (Chan, Golub and LeVeque, 1979), so
// a row far from zero loses nothing and one barrier is enough.
template <bool VEC, int NV>
__device__ __forceinline__ void row_stats(const float (&v)[NV][8], int kind, float eps, int dim, float inv_dim,
                                          Shared& sh, int& half, int& mhalf, int nwarps, float& mean, float& rstd) {
  if (kind == kRms) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[i][e] * v[i][e];
    block_sum(s, sh.sum, half, nwarps);
    mean = 0.f;
    rstd = rsqrtf(s[0] * inv_dim + eps);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const float n = sh.count[warp];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v[i][e];
  const float m = n > 0.f ? warp_sum(s) / n : 0.f;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = column<VEC>(i, e) < dim ? v[i][e] - m : 0.f;
      q += t * t;
    }
  q = warp_sum(q);
  if (nwarps > 1) {
    if ((threadIdx.x & 31) == 0) sh.moment[mhalf][warp] = make_float2(m, q);
    __syncthreads();
    float total = 0.f;
    for (int w = 0; w < nwarps; ++w) total += sh.count[w] * sh.moment[mhalf][w].x;
    mean = total * inv_dim;
    q = 0.f;
    for (int w = 0; w < nwarps; ++w) {
      const float2 p = sh.moment[mhalf][w];
      q += p.y + sh.count[w] * (p.x - mean) * (p.x - mean);
    }
    mhalf ^= 1;
  } else {
    mean = m;
  }
  rstd = rsqrtf(q * inv_dim + eps);
}

template <bool VEC, int NV>
__device__ __forceinline__ void count_columns(Shared& sh, int dim) {
  float c = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) c += column<VEC>(i, e) < dim ? 1.f : 0.f;
  c = warp_sum(c);
  if ((threadIdx.x & 31) == 0) sh.count[threadIdx.x >> 5] = c;
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ const T* row_in(const void* p, long long row, long long stride) {
  return static_cast<const T*>(p) + row * stride;
}
template <typename T>
__device__ __forceinline__ T* row_out(void* p, long long row, long long stride) {
  return static_cast<T*>(p) + row * stride;
}

// ---------------------------------------------------------------- forward --
template <typename XT, typename BT, bool VEC, int NV, bool RES, bool NORM>
__global__ void __launch_bounds__(1024, 1) row_fwd_kernel(const __grid_constant__ RowArgs a) {
  __shared__ Shared sh;
  const int dim = a.dim, nwarps = blockDim.x >> 5;
  const float inv_dim = 1.f / (float)dim;
  count_columns<VEC, NV>(sh, dim);
  int half = 0, mhalf = 0;
  const long long r0 = a.rows * blockIdx.x / gridDim.x, r1 = a.rows * (blockIdx.x + 1) / gridDim.x;
  long long group_end = r0;      // first row of the next modulation group
  float gate[NV][8], mul[NV][8], add[NV][8];
  for (long long r = r0; r < r1; ++r) {
    if (r >= group_end) {
      const long long g = r / a.rows_per_group;
      group_end = (g + 1) * a.rows_per_group;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (RES) {
          float pw[8];
          load_param<VEC>(gate[i], a.gate, g * a.gate_stride, a.param_bf16, 1.f, i, dim);
          load_param<VEC>(pw, a.post_weight, 0, a.param_bf16, 1.f, i, dim);
#pragma unroll
          for (int e = 0; e < 8; ++e) gate[i][e] *= a.residual_scale * pw[e];
        }
        if (NORM) {
          // (n w + b)(1 + s) + t = n (w (1 + s)) + (b (1 + s) + t)
          float w[8], b[8];
          load_param<VEC>(mul[i], a.scale, g * a.scale_stride, a.param_bf16, 0.f, i, dim);
          load_param<VEC>(add[i], a.shift, g * a.shift_stride, a.param_bf16, 0.f, i, dim);
          load_param<VEC>(w, a.weight, 0, a.param_bf16, 1.f, i, dim);
          load_param<VEC>(b, a.bias, 0, a.param_bf16, 0.f, i, dim);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float s1 = 1.f + mul[i][e];
            add[i][e] += b[e] * s1;
            mul[i][e] = w[e] * s1;
          }
        }
      }
    }
    float x[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_row<VEC>(x[i], row_in<XT>(a.x, r, a.x_stride), i, dim);
    if (RES) {
      float y[NV][8];
#pragma unroll
      for (int i = 0; i < NV; ++i) load_row<VEC>(y[i], row_in<BT>(a.y, r, a.y_stride), i, dim);
      float m = 0.f, s = 1.f;
      if (a.post_norm != kNone)
        row_stats<VEC, NV>(y, a.post_norm, a.post_eps, dim, inv_dim, sh, half, mhalf, nwarps, m, s);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] += gate[i][e] * ((y[i][e] - m) * s);
        store_row<VEC>(row_out<XT>(a.x_out, r, a.x_out_stride), x[i], i, dim);
      }
    }
    if (NORM) {
      if (RES && !VEC) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (column<VEC>(i, e) >= dim) x[i][e] = 0.f;
      } else if (RES) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (column<VEC>(i, 0) >= dim) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
          }
      }
      float m, s;
      row_stats<VEC, NV>(x, a.norm, a.eps, dim, inv_dim, sh, half, mhalf, nwarps, m, s);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = (x[i][e] - m) * s * mul[i][e] + add[i][e];
        store_row<VEC>(row_out<BT>(a.h, r, a.h_stride), x[i], i, dim);
      }
    }
  }
}

// --------------------------------------------------------------- backward --
// A unit is chunk c of group g: rows [g R + R c / C, g R + R (c + 1) / C) of a
// group of R rows cut into C chunks.  With C > 1 the unit's sums A, B, C go to
// `part` [unit][3][dim] and row_reduce_kernel makes every parameter gradient
// of them.  With C = 1 a unit is a whole group: its modulation gradients are
// final and written here, and the weights' sums run on over the block's units
// (WACC) and go to `part` [block][3][dim].
template <typename XT, typename BT, bool VEC, int NV, bool RES, bool NORM, bool WACC>
__global__ void __launch_bounds__(NV == 1 ? 640 : 1024, 1) row_bwd_kernel(const __grid_constant__ RowArgs a) {
  __shared__ Shared sh;
  const int dim = a.dim, nwarps = blockDim.x >> 5;
  const float inv_dim = 1.f / (float)dim;
  count_columns<VEC, NV>(sh, dim);
  int half = 0, mhalf = 0;
  const bool layer = a.norm == kLayer, post_layer = a.post_norm == kLayer;
  float wacc[WACC ? NV : 1][3][8];
  if (WACC) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) wacc[i][k][e] = 0.f;
  }
  const long long units = a.groups * a.chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long g = u / a.chunks, c = u - g * a.chunks;
    const long long base = g * a.rows_per_group;
    const long long r0 = base + a.rows_per_group * c / a.chunks, r1 = base + a.rows_per_group * (c + 1) / a.chunks;
    float gate[NV][8], mul[NV][8];     // r gate pw, and (1 + s) w
    float A[NV][8], B[NV][8], C[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float t[8];
      if (RES) {
        load_param<VEC>(gate[i], a.gate, g * a.gate_stride, a.param_bf16, 1.f, i, dim);
        load_param<VEC>(t, a.post_weight, 0, a.param_bf16, 1.f, i, dim);
#pragma unroll
        for (int e = 0; e < 8; ++e) gate[i][e] *= a.residual_scale * t[e];
      }
      if (NORM) {
        load_param<VEC>(mul[i], a.scale, g * a.scale_stride, a.param_bf16, 0.f, i, dim);
        load_param<VEC>(t, a.weight, 0, a.param_bf16, 1.f, i, dim);
#pragma unroll
        for (int e = 0; e < 8; ++e) mul[i][e] = (1.f + mul[i][e]) * t[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) A[i][e] = B[i][e] = C[i][e] = 0.f;
    }
    for (long long r = r0; r < r1; ++r) {
      float gr[NV][8], y[NV][8];       // the gradient of x', and yhat
      float ys = 1.f;
      if (a.dx_out) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_row<VEC>(gr[i], row_in<XT>(a.dx_out, r, a.dx_out_stride), i, dim);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) gr[i][e] = 0.f;
      }
      if (RES) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_row<VEC>(y[i], row_in<BT>(a.y, r, a.y_stride), i, dim);
        if (a.post_norm != kNone) {
          float m;
          row_stats<VEC, NV>(y, a.post_norm, a.post_eps, dim, inv_dim, sh, half, mhalf, nwarps, m, ys);
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = column<VEC>(i, e) < dim ? (y[i][e] - m) * ys : 0.f;
        }
      }
      if (NORM) {
        float x[NV][8], dh[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          load_row<VEC>(x[i], row_in<XT>(a.x, r, a.x_stride), i, dim);
          load_row<VEC>(dh[i], row_in<BT>(a.dh, r, a.dh_stride), i, dim);
          if (RES) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (column<VEC>(i, e) < dim) x[i][e] += gate[i][e] * y[i][e];
          }
        }
        float m, s;
        row_stats<VEC, NV>(x, a.norm, a.eps, dim, inv_dim, sh, half, mhalf, nwarps, m, s);
        float t[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[i][e] = (x[i][e] - m) * s;
            A[i][e] += dh[i][e];
            B[i][e] += dh[i][e] * x[i][e];
            dh[i][e] *= mul[i][e];
            t[0] += dh[i][e];
            t[1] += dh[i][e] * x[i][e];
          }
        block_sum(t, sh.sum, half, nwarps);
        const float m0 = layer ? t[0] * inv_dim : 0.f, m1 = t[1] * inv_dim;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) gr[i][e] += s * (dh[i][e] - m0 - x[i][e] * m1);
          store_row<VEC>(row_out<XT>(a.dx, r, a.dx_stride), gr[i], i, dim);
        }
      }
      if (RES) {
        float t[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (column<VEC>(i, e) >= dim) gr[i][e] = 0.f;
            C[i][e] += gr[i][e] * y[i][e];
            gr[i][e] *= gate[i][e];
            t[0] += gr[i][e];
            t[1] += gr[i][e] * y[i][e];
          }
        if (a.post_norm != kNone) {
          block_sum(t, sh.sum, half, nwarps);
          const float m0 = post_layer ? t[0] * inv_dim : 0.f, m1 = t[1] * inv_dim;
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) gr[i][e] = ys * (gr[i][e] - m0 - y[i][e] * m1);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) store_row<VEC>(row_out<BT>(a.dy, r, a.dy_stride), gr[i], i, dim);
      }
    }
    if (a.chunks > 1) {
      float* p = a.part + u * 3 * dim;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (NORM) {
          store_row<VEC>(p, A[i], i, dim);
          store_row<VEC>(p + dim, B[i], i, dim);
        }
        if (RES) store_row<VEC>(p + 2 * (long long)dim, C[i], i, dim);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float t[8], w[8], b[8];
        if (NORM) {
          load_param<VEC>(w, a.weight, 0, a.param_bf16, 1.f, i, dim);
          load_param<VEC>(b, a.bias, 0, a.param_bf16, 0.f, i, dim);
          if (a.dshift) store_row<VEC>(a.dshift + g * dim, A[i], i, dim);
          if (a.dscale) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = w[e] * B[i][e] + b[e] * A[i][e];
            store_row<VEC>(a.dscale + g * dim, t, i, dim);
          }
          if (WACC) {
            load_param<VEC>(t, a.scale, g * a.scale_stride, a.param_bf16, 0.f, i, dim);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              wacc[i][0][e] += (1.f + t[e]) * A[i][e];
              wacc[i][1][e] += (1.f + t[e]) * B[i][e];
            }
          }
        }
        if (RES) {
          load_param<VEC>(w, a.post_weight, 0, a.param_bf16, 1.f, i, dim);
          if (a.dgate) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = a.residual_scale * w[e] * C[i][e];
            store_row<VEC>(a.dgate + g * dim, t, i, dim);
          }
          if (WACC) {
            load_param<VEC>(t, a.gate, g * a.gate_stride, a.param_bf16, 1.f, i, dim);
#pragma unroll
            for (int e = 0; e < 8; ++e) wacc[i][2][e] += a.residual_scale * t[e] * C[i][e];
          }
        }
      }
    }
  }
  if (WACC) {
    float* p = a.part + (long long)blockIdx.x * 3 * dim;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 3; ++k) store_row<VEC>(p + (long long)k * dim, wacc[i][k], i, dim);
  }
}

// Adds the units' column sums in a fixed order, in float64, and forms the
// parameter gradients.  A block takes 32 columns; its 32 warps take the
// groups in turn, or, with few groups, slices of every group's chunks.
__device__ __forceinline__ float param_at(const void* p, long long i, bool bf16, float none) {
  if (!p) return none;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__global__ void __launch_bounds__(1024) row_reduce_kernel(const __grid_constant__ RowArgs a, int blocks) {
  __shared__ double sh[3][32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, dim = a.dim;
  const bool in = col < dim;
  double wsum[3] = {0.0, 0.0, 0.0};
  if (a.chunks == 1) {
    for (int b = warp; in && b < blocks; b += 32)
      for (int k = 0; k < 3; ++k) wsum[k] += (double)a.part[((long long)b * 3 + k) * dim + col];
  } else {
    const bool sliced = a.groups < 16;        // every warp on every group
    const float w = in ? param_at(a.weight, col, a.param_bf16, 1.f) : 0.f;
    const float b = in ? param_at(a.bias, col, a.param_bf16, 0.f) : 0.f;
    const float pw = in ? param_at(a.post_weight, col, a.param_bf16, 1.f) : 0.f;
    for (long long g0 = 0; g0 < a.groups; g0 += sliced ? 1 : 32) {
      const long long g = sliced ? g0 : g0 + warp;
      double s[3] = {0.0, 0.0, 0.0};
      if (in && g < a.groups)
        for (long long c = sliced ? warp : 0; c < a.chunks; c += sliced ? 32 : 1)
          for (int k = 0; k < 3; ++k) s[k] += (double)a.part[((g * a.chunks + c) * 3 + k) * dim + col];
      if (sliced) {
        for (int k = 0; k < 3; ++k) sh[k][warp][lane] = s[k];
        __syncthreads();
        if (warp == 0)
          for (int v = 1; v < 32; ++v)
            for (int k = 0; k < 3; ++k) s[k] += sh[k][v][lane];
        __syncthreads();
      }
      if (in && g < a.groups && (!sliced || warp == 0)) {
        if (a.dshift) a.dshift[g * dim + col] = (float)s[0];
        if (a.dscale) a.dscale[g * dim + col] = (float)(w * s[1] + b * s[0]);
        if (a.dgate) a.dgate[g * dim + col] = (float)(a.residual_scale * pw * s[2]);
        const double s1 = 1.0 + param_at(a.scale, g * a.scale_stride + col, a.param_bf16, 0.f);
        wsum[0] += s1 * s[0];
        wsum[1] += s1 * s[1];
        wsum[2] += (double)a.residual_scale * param_at(a.gate, g * a.gate_stride + col, a.param_bf16, 1.f) * s[2];
      }
    }
  }
  for (int k = 0; k < 3; ++k) sh[k][warp][lane] = wsum[k];
  __syncthreads();
  if (warp < 3 && in) {
    double s = 0.0;
    for (int v = 0; v < 32; ++v) s += sh[warp][v][lane];
    float* out = warp == 0 ? a.dbias : (warp == 1 ? a.dweight : a.dpost_weight);
    if (out) out[col] = (float)s;
  }
}

// ----------------------------------------------------------------- launch --
bool vec_ok(const void* p, long long stride, int esz) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * esz % 16 == 0);
}

// Every row of every operand starts on a 16-byte boundary and holds whole
// vectors of eight.
bool vectors(const RowArgs& a) {
  const int ex = a.x_bf16 ? 2 : 4, eb = a.branch_bf16 ? 2 : 4, ep = a.param_bf16 ? 2 : 4;
  return a.dim % 8 == 0 && vec_ok(a.x, a.x_stride, ex) && vec_ok(a.y, a.y_stride, eb) &&
         vec_ok(a.x_out, a.x_out_stride, ex) && vec_ok(a.h, a.h_stride, eb) &&
         vec_ok(a.dx_out, a.dx_out_stride, ex) && vec_ok(a.dh, a.dh_stride, eb) && vec_ok(a.dx, a.dx_stride, ex) &&
         vec_ok(a.dy, a.dy_stride, eb) && vec_ok(a.gate, a.gate_stride, ep) && vec_ok(a.scale, a.scale_stride, ep) &&
         vec_ok(a.shift, a.shift_stride, ep) && vec_ok(a.weight, 0, ep) && vec_ok(a.bias, 0, ep) &&
         vec_ok(a.post_weight, 0, ep) && vec_ok(a.dscale, 0, 4) && vec_ok(a.dshift, 0, 4) && vec_ok(a.dgate, 0, 4);
}

int row_threads(int dim, int nv) {
  const int t = (dim + 8 * nv - 1) / (8 * nv);
  return (t + 31) / 32 * 32;
}

template <typename XT, typename BT, bool VEC, int NV>
cudaError_t fwd(const RowArgs& a, cudaStream_t s) {
  const int threads = row_threads(a.dim, NV);
  const long long resident = (long long)num_sms() * (threads >= 1024 ? 1 : 1024 / threads > 16 ? 16 : 1024 / threads);
  const int grid = (int)(a.rows < resident ? a.rows : resident);
  if (a.y && a.h) row_fwd_kernel<XT, BT, VEC, NV, true, true><<<grid, threads, 0, s>>>(a);
  else if (a.y) row_fwd_kernel<XT, BT, VEC, NV, true, false><<<grid, threads, 0, s>>>(a);
  else row_fwd_kernel<XT, BT, VEC, NV, false, true><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename XT, typename BT, bool VEC, int NV, bool WACC>
cudaError_t bwd(const RowArgs& a, int grid, cudaStream_t s) {
  const int threads = row_threads(a.dim, NV);
  if (a.dy && a.dh) row_bwd_kernel<XT, BT, VEC, NV, true, true, WACC><<<grid, threads, 0, s>>>(a);
  else if (a.dy) row_bwd_kernel<XT, BT, VEC, NV, true, false, WACC><<<grid, threads, 0, s>>>(a);
  else row_bwd_kernel<XT, BT, VEC, NV, false, true, WACC><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename F>
cudaError_t by_type(const RowArgs& a, F f) {
  if (a.x_bf16) return f((__nv_bfloat16*)nullptr, (__nv_bfloat16*)nullptr);
  if (a.branch_bf16) return f((float*)nullptr, (__nv_bfloat16*)nullptr);
  return f((float*)nullptr, (float*)nullptr);
}

}  // namespace

// The blocks of a backward launch and the chunks each group is cut into: of
// the cuts that fill the resident blocks once to eight times, the one whose
// busiest block has the fewest rows (the first such, for the smallest
// workspace).
RowPlan plan_row_bwd(long long rows, long long groups, int dim, bool weights) {
  RowPlan p;
  const int threads = row_threads(dim, dim > 5120 ? 2 : 1);
  const long long resident = (long long)num_sms() * (threads > 320 ? 1 : (threads > 160 ? 2 : (threads > 64 ? 4 : 8)));
  const long long per = groups > 0 ? rows / groups : 0;
  p.chunks = 1;
  long long best = ((groups + resident - 1) / resident) * per;
  for (long long k = 1; k <= 8 && per > 1; ++k) {
    const long long fill = k * resident / (groups > 0 ? groups : 1);
    const long long c = fill < 1 ? 1 : (fill < per ? fill : per);
    const long long cost = ((groups * c + resident - 1) / resident) * ((per + c - 1) / c);
    if (cost < best) {
      best = cost;
      p.chunks = c;
    }
  }
  const long long units = groups * p.chunks;
  p.grid = (int)(units < resident ? units : resident);
  p.floats = p.chunks > 1 ? (size_t)units * 3 * dim : (weights ? (size_t)p.grid * 3 * dim : 0);
  return p;
}

cudaError_t launch_row_fwd(const RowArgs& a, cudaStream_t s) {
  const bool vec = vectors(a);
  return by_type(a, [&](auto* x, auto* b) {
    using XT = std::remove_pointer_t<decltype(x)>;
    using BT = std::remove_pointer_t<decltype(b)>;
    if (vec) return a.dim <= 8192 ? fwd<XT, BT, true, 1>(a, s) : fwd<XT, BT, true, 2>(a, s);
    return a.dim <= 8192 ? fwd<XT, BT, false, 1>(a, s) : fwd<XT, BT, false, 2>(a, s);
  });
}

cudaError_t launch_row_bwd(const RowArgs& a, int grid, cudaStream_t s) {
  const bool vec = vectors(a);
  const bool weights = a.dweight || a.dbias || a.dpost_weight;
  const bool wacc = weights && a.chunks == 1;
  cudaError_t e = by_type(a, [&](auto* x, auto* b) {
    using XT = std::remove_pointer_t<decltype(x)>;
    using BT = std::remove_pointer_t<decltype(b)>;
    if (a.dim <= 5120) {
      if (vec) return wacc ? bwd<XT, BT, true, 1, true>(a, grid, s) : bwd<XT, BT, true, 1, false>(a, grid, s);
      return wacc ? bwd<XT, BT, false, 1, true>(a, grid, s) : bwd<XT, BT, false, 1, false>(a, grid, s);
    }
    if (vec) return wacc ? bwd<XT, BT, true, 2, true>(a, grid, s) : bwd<XT, BT, true, 2, false>(a, grid, s);
    return wacc ? bwd<XT, BT, false, 2, true>(a, grid, s) : bwd<XT, BT, false, 2, false>(a, grid, s);
  });
  if (e != cudaSuccess) return e;
  if (a.chunks > 1 || weights) {
    row_reduce_kernel<<<(a.dim + 31) / 32, 1024, 0, s>>>(a, grid);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace spade
