// Row passes of the residual stream around a block: the norm with modulation
// that opens it, the gated update that ends it, and both in one pass
// (spade_norm_modulate, spade_gate_residual, spade_gate_residual_norm).
//
//   x' = x + r * gate_g * P(y)          P: none, rms or layer norm * weight
//   h  = (N(x') * w + b) * (1 + scale_g) + shift_g
//
// with g the row's modulation group.  A block walks a run of rows, K at a
// time: their sums share a barrier, and the modulation stays in registers
// while the group lasts.  Bound by memory: each row is read and written once.
#pragma once
#include "row_pass.cuh"

namespace spade {
namespace {

using namespace rowpass;

template <typename XT, typename BT, int P, bool RING, int NV, int K, bool RES, bool NORM>
__global__ void __launch_bounds__(NV == 1 ? 640 : 512, 1) row_fwd_kernel(const __grid_constant__ RowArgs a, int depth) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Shared<K> sh;
  const int dim = a.dim, nwarps = blockDim.x >> 5;
  Stream<XT, P, RING, NV> sx{static_cast<const XT*>(a.x), a.x_stride, 0};
  Stream<BT, P, RING, NV> sy{static_cast<const BT*>(a.y), a.y_stride, slot_bytes(blockDim.x, NV, sizeof(XT))};
  const uint32_t slot = sy.at + (RES ? slot_bytes(blockDim.x, NV, sizeof(BT)) : 0);
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  const long long r0 = a.rows * blockIdx.x / gridDim.x, r1 = a.rows * (blockIdx.x + 1) / gridDim.x;

  // the next row to copy and its slot; the slot of the next row to use
  long long fr = r0;
  int fs = 0, us = 0;
  auto fetch = [&]() {
    if (fr < r1) {
      sx.fetch(ring_at + fs * slot, fr, dim);
      if (RES) sy.fetch(ring_at + fs * slot, fr, dim);
    }
    commit_async();
    ++fr;
    fs = fs + 1 == depth ? 0 : fs + 1;
  };
  if (RING) {
    for (int d = 0; d < depth; ++d) {
      sx.clear(ring + d * slot, dim);
      if (RES) sy.clear(ring + d * slot, dim);
      fetch();
    }
  }
  count_columns<P, NV>(sh.count, dim);
  int half = 0;
  long long group_end = r0;      // first row of the next modulation group
  Eight gate[NV], times[NV], plus[NV];
  for (long long r = r0; r < r1;) {
    if (r >= group_end) {
      const long long g = r / a.rows_per_group;
      group_end = (g + 1) * a.rows_per_group;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (RES) {
          Eight pw;
          load_param<P>(gate[i], a.gate, g * a.gate_stride, a.param_bf16, 1.f, i, dim);
          load_param<P>(pw, a.post_weight, 0, a.param_bf16, 1.f, i, dim);
#pragma unroll
          for (int q = 0; q < 4; ++q) gate[i].p[q] = mul(gate[i].p[q], mul(both(a.residual_scale), pw.p[q]));
        }
        if (NORM) {
          // (n w + b)(1 + s) + t = n (w (1 + s)) + (b (1 + s) + t)
          Eight w, b;
          load_param<P>(times[i], a.scale, g * a.scale_stride, a.param_bf16, 0.f, i, dim);
          load_param<P>(plus[i], a.shift, g * a.shift_stride, a.param_bf16, 0.f, i, dim);
          load_param<P>(w, a.weight, 0, a.param_bf16, 1.f, i, dim);
          load_param<P>(b, a.bias, 0, a.param_bf16, 0.f, i, dim);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 s1 = add(both(1.f), times[i].p[q]);
            plus[i].p[q] = fma(b.p[q], s1, plus[i].p[q]);
            times[i].p[q] = mul(w.p[q], s1);
          }
        }
      }
    }
    const long long end = r1 < group_end ? r1 : group_end;
    const int n = end - r < K ? (int)(end - r) : K;
    if (RING) wait_async_upto(depth - K);
    const unsigned char* at[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int s = us + k >= depth ? us + k - depth : us + k;
      at[k] = ring + s * slot;
    }
    Eight x[K][NV];
    if (RES) {
      float m[K], s[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (k < n) sy.get(x[k][i], at[k], r + k, i, dim);
          else x[k][i].fill(0.f);
        }
      if (a.post_norm != kNone) {
        row_stats<P, NV, K>(x, a.post_norm, a.post_eps, dim, sh, half, nwarps, m, s);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) x[k][i].p[q] = mul(add(x[k][i].p[q], both(-m[k])), both(s[k]));
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          Eight v;
          sx.get(v, at[k], r + k, i, dim);
#pragma unroll
          for (int q = 0; q < 4; ++q) x[k][i].p[q] = fma(gate[i].p[q], x[k][i].p[q], v.p[q]);
          store8<P>(static_cast<XT*>(a.x_out) + (r + k) * a.x_out_stride, x[k][i], i, dim);
          if (NORM) {
#pragma unroll
            for (int q = 0; q < 4; ++q) x[k][i].p[q] = present<P>(x[k][i].p[q], i, q, dim);
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (k < n) sx.get(x[k][i], at[k], r + k, i, dim);
          else x[k][i].fill(0.f);
        }
    }
    if (RING) {                 // everything of these rows is in registers: their slots are free
      for (int k = 0; k < n; ++k) fetch();
      us = us + n >= depth ? us + n - depth : us + n;
    }
    if (NORM) {
      float m[K], s[K];
      row_stats<P, NV, K>(x, a.norm, a.eps, dim, sh, half, nwarps, m, s);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            x[k][i].p[q] = fma(mul(add(x[k][i].p[q], both(-m[k])), both(s[k])), times[i].p[q], plus[i].p[q]);
          store8<P>(static_cast<BT*>(a.h) + (r + k) * a.h_stride, x[k][i], i, dim);
        }
      }
    }
    r += n;
  }
  if (RING) wait_async<0>();
}

// ----------------------------------------------------------------- launch --
template <typename XT, typename BT, int P, bool RING, int NV, bool RES, bool NORM>
cudaError_t run(const RowArgs& a, cudaStream_t s) {
  constexpr int K = NV == 1 ? 4 : (NV == 2 ? 2 : 1);
  const auto kernel = row_fwd_kernel<XT, BT, P, RING, NV, K, RES, NORM>;
  const int threads = row_threads(a.dim, NV);
  // blocks of an SM: by registers (96 a thread), then the ring takes what shared memory is left
  int blocks = 640 / threads < 16 ? 640 / threads : 16;
  if (blocks < 1) blocks = 1;
  const long long resident = (long long)num_sms() * blocks;
  const int grid = (int)(a.rows < resident ? a.rows : resident);
  int depth = 0;
  size_t smem = 0;
  if (RING) {
    const size_t slot = slot_bytes(threads, NV, sizeof(XT)) + (RES ? slot_bytes(threads, NV, sizeof(BT)) : 0);
    const size_t room = kSmemSm / blocks - 1024 - sizeof(Shared<K>);
    const long long rows = (a.rows + grid - 1) / grid;
    depth = (int)(room / slot < kDepthMax ? room / slot : kDepthMax);
    if (rows < depth) depth = (int)(rows > K ? rows : K);
    smem = depth * slot;
    if (smem > 32 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
  }
  kernel<<<grid, threads, smem, s>>>(a, depth);
  return cudaGetLastError();
}

template <typename XT, typename BT, int P, bool RING, int NV>
cudaError_t by_op(const RowArgs& a, cudaStream_t s) {
  if (a.y && a.h) return run<XT, BT, P, RING, NV, true, true>(a, s);
  if (a.y) return run<XT, BT, P, RING, NV, true, false>(a, s);
  return run<XT, BT, P, RING, NV, false, true>(a, s);
}

// Rows above 8192 elements are read where they are used.
template <typename XT, typename BT, int P, bool RING>
cudaError_t by_width(const RowArgs& a, cudaStream_t s) {
  switch (row_nv(a.dim)) {
    case 1: return by_op<XT, BT, P, RING, 1>(a, s);
    case 2: return by_op<XT, BT, P, RING, 2>(a, s);
    default: return by_op<XT, BT, P == 2 ? 1 : P, false, 4>(a, s);
  }
}

}  // namespace

template <typename XT, typename BT>
cudaError_t row_fwd(const RowArgs& a, cudaStream_t s) {
  const int p = piece_of(a);
  if constexpr (sizeof(XT) == 2) {
    if (p == 8) return by_width<XT, BT, 8, true>(a, s);
    return p > 1 ? by_width<XT, BT, 2, true>(a, s) : by_width<XT, BT, 1, false>(a, s);
  } else {
    return p == 4 ? by_width<XT, BT, 4, true>(a, s) : by_width<XT, BT, 1, sizeof(BT) == 4>(a, s);
  }
}

}  // namespace spade
