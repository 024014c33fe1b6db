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

__global__ void __launch_bounds__(1024) row_reduce_kernel(const __grid_constant__ RowArgs a, int blocks) {
  __shared__ double sh[3][32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, dim = a.dim;
  const bool in = col < dim;
  // the sums that the pass has: A and B with a norm, C with a residual
  const int k0 = a.dh ? 0 : 2, k1 = a.dy ? 3 : 2;
  double wsum[3] = {0.0, 0.0, 0.0};
  if (a.chunks == 1) {
    for (int b = warp; in && b < blocks; b += 32)
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k >= k0 && k < k1) wsum[k] += (double)a.part[((long long)b * 3 + k) * dim + col];
  } else {
    const bool sliced = a.groups < 16;        // every warp on every group
    const float w = in ? param_at(a.weight, col, a.param_bf16, 1.f) : 0.f;
    const float b = in ? param_at(a.bias, col, a.param_bf16, 0.f) : 0.f;
    const float pw = in ? param_at(a.post_weight, col, a.param_bf16, 1.f) : 0.f;
    for (long long g0 = 0; g0 < a.groups; g0 += sliced ? 1 : 32) {
      const long long g = sliced ? g0 : g0 + warp;
      double s[3] = {0.0, 0.0, 0.0};
      if (in && g < a.groups) {
#pragma unroll 4
        for (long long c = sliced ? warp : 0; c < a.chunks; c += sliced ? 32 : 1)
#pragma unroll
          for (int k = 0; k < 3; ++k)
            if (k >= k0 && k < k1) s[k] += (double)a.part[((g * a.chunks + c) * 3 + k) * dim + col];
      }
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
  if (a.chunks > 1 || weights) {
    row_reduce_kernel<<<(a.dim + 31) / 32, 1024, 0, s>>>(a, grid);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace spade
