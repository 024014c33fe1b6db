// Row passes: choice of the kernels by type, the backward plan, and the sums of
// the parameter gradients.  The kernels are in row_fwd.cuh and row_bwd.cuh,
// compiled once for each pair of types (k_row_*.cu).
#include "row_pass.cuh"

namespace spade {

template <typename XT, typename BT> cudaError_t row_fwd(const RowArgs& a, cudaStream_t s);
template <typename XT, typename BT> cudaError_t row_bwd(const RowArgs& a, int grid, bool weights, cudaStream_t s);

namespace {

using namespace rowpass;

// Adds the units' column sums in a fixed order, in float64, and forms the
// parameter gradients.  A block takes 32 columns; its 32 warps take the
// groups in turn, or, with few groups, slices of every group's chunks.
__device__ __forceinline__ float param_at(const void* p, long long i, bool is_bf16, float none) {
  if (!p) return none;
  return is_bf16 ? __bfloat162float(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Column sums of `n` units, `step` floats apart, that start at p: all loads of
// a round are in flight together.
template <int K0, int K1>
__device__ __forceinline__ void sum_units(double (&s)[3], const float* __restrict__ p, long long n, long long step, int dim) {
  constexpr int R = K1 - K0 == 1 ? 16 : 8;
  for (long long c = 0; c < n; c += R) {
    float v[R][3];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = K0; k < K1; ++k) v[i][k] = c + i < n ? p[(c + i) * step + (long long)k * dim] : 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = K0; k < K1; ++k) s[k] += (double)v[i][k];
  }
}

// K0, K1: the sums that the pass has, A and B with a norm, C with a residual.
template <int K0, int K1>
__global__ void __launch_bounds__(1024) row_reduce_kernel(const __grid_constant__ RowArgs a, int blocks) {
  __shared__ double sh[3][32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, dim = a.dim;
  const long long unit = 3LL * dim;
  const bool in = col < dim;
  cudaGridDependencySynchronize();
  double wsum[3] = {0.0, 0.0, 0.0};
  if (a.chunks == 1) {
    if (in && warp < blocks) sum_units<K0, K1>(wsum, a.part + warp * unit + col, (blocks - warp + 31) / 32, 32 * unit, dim);
  } else {
    const bool sliced = a.groups < 16;        // every warp on every group
    const float w = in ? param_at(a.weight, col, a.param_bf16, 1.f) : 0.f;
    const float b = in ? param_at(a.bias, col, a.param_bf16, 0.f) : 0.f;
    const float pw = in ? param_at(a.post_weight, col, a.param_bf16, 1.f) : 0.f;
    for (long long g0 = 0; g0 < a.groups; g0 += sliced ? 1 : 32) {
      const long long g = sliced ? g0 : g0 + warp;
      double s[3] = {0.0, 0.0, 0.0};
      if (in && g < a.groups) {
        const float* p = a.part + g * a.chunks * unit + col;
        if (!sliced) sum_units<K0, K1>(s, p, a.chunks, unit, dim);
        else if (warp < a.chunks) sum_units<K0, K1>(s, p + warp * unit, (a.chunks - warp + 31) / 32, 32 * unit, dim);
      }
      if (sliced) {
#pragma unroll
        for (int k = K0; k < K1; ++k) sh[k][warp][lane] = s[k];
        __syncthreads();
        if (warp == 0)
#pragma unroll 8
          for (int v = 1; v < 32; ++v)
#pragma unroll
            for (int k = K0; k < K1; ++k) s[k] += sh[k][v][lane];
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
  if (!a.dbias && !a.dweight && !a.dpost_weight) return;
#pragma unroll
  for (int k = K0; k < K1; ++k) sh[k][warp][lane] = wsum[k];
  __syncthreads();
  if (warp >= K0 && warp < K1 && in) {
    double s = 0.0;
#pragma unroll 8
    for (int v = 0; v < 32; ++v) s += sh[warp][v][lane];
    float* out = warp == 0 ? a.dbias : (warp == 1 ? a.dweight : a.dpost_weight);
    if (out) out[col] = (float)s;
  }
}

}  // namespace

// The blocks of a backward launch and the chunks each group is cut into: of
// the cuts that fill the resident blocks once to eight times, the one whose
// busiest block has the fewest rows (the first such, for the smallest
// workspace).
RowPlan plan_row_bwd(long long rows, long long groups, int dim, bool weights) {
  RowPlan p;
  const long long resident = (long long)num_sms() * bwd_blocks(dim);
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
  if (a.x_bf16) return row_fwd<bf16, bf16>(a, s);
  return a.branch_bf16 ? row_fwd<float, bf16>(a, s) : row_fwd<float, float>(a, s);
}

cudaError_t launch_row_bwd(const RowArgs& a, int grid, cudaStream_t s) {
  const bool weights = a.dweight || a.dbias || a.dpost_weight;
  cudaError_t e;
  if (a.x_bf16) e = row_bwd<bf16, bf16>(a, grid, weights, s);
  else e = a.branch_bf16 ? row_bwd<float, bf16>(a, grid, weights, s) : row_bwd<float, float>(a, grid, weights, s);
  if (e != cudaSuccess) return e;
  if (a.part) {
    const int cols = (a.dim + 31) / 32;
    const auto kernel = a.dh && a.dy ? row_reduce_kernel<0, 3> : (a.dh ? row_reduce_kernel<0, 2> : row_reduce_kernel<2, 3>);
    e = launch_behind(kernel, cols, 1024, s, a, grid);
  }
  return e;
}

}  // namespace spade
