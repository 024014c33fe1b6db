// Row passes of the residual stream around a block: the norm with modulation
// that opens it, the gated update that ends it, and both in one pass
// (spade_norm_modulate, spade_gate_residual, spade_gate_residual_norm).
//
//   x' = x + r * gate_g * P(y)          P: none, rms or layer norm * weight
//   h  = (N(x') * w + b) * (1 + scale_g) + shift_g
//
// with g the row's modulation group.  A block walks its rows K at a time:
// their sums share a barrier, and the modulation stays in registers while the
// group lasts.
//
// Bound by memory: each row is read and written once.  On 75600 rows of 5120
// (bfloat16), different cards: h alone 250 to 276 us, 5.6 to 6.2 TB/s of the 6.55
// that a copy reaches; x' and h 491 to 552 us, 5.6 to 6.3 TB/s.  Steps of h alone,
// on one card: 1131 us with one row to a block and a load when it was needed, 352
// with the ring, 302 with paired arithmetic and whole batches without per-row
// branches, 278 with the moments merged without divisions, 251 with the blocks
// taking turns.
//
// With one modulation a row the batch is one row and its parameters are loaded
// where they are used: 162 us for h of 32760 rows of 1536 (float32 stream), 1.5
// times their bytes.  Narrow pieces: h of 32760 rows of 1540 bfloat16 in pieces
// of two 71 us, of 1537 in single elements 108, where 1536 take 31 of bytes.
#pragma once
#include "row_pass.cuh"

namespace spade {
namespace {

using namespace rowpass;

// POST: the branch has a norm (0 no, 1 yes, 2 as the call says).
template <typename XT, typename BT, class L, int K, bool RES, bool NORM, int POST>
__global__ void __maxnreg__(L::NV <= 2 ? 96 : 128) row_fwd_kernel(const __grid_constant__ RowArgs a, int depth) {
  constexpr int NV = L::NV;
  constexpr bool RING = L::RING;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Shared<K> sh;
  const int dim = a.dim, nwarps = blockDim.x >> 5;
  // With one modulation group the blocks take turns, K rows each, so that all of
  // them read and write one stretch of memory; with several a block keeps to a
  // run of rows and so to few groups.
  const bool turns = a.groups == 1;
  const long long tiles = (a.rows + K - 1) / K, hop = turns ? (gridDim.x - 1LL) * K : 0;      // rows of the others
  const long long r0 = turns ? (long long)blockIdx.x * K : a.rows * blockIdx.x / gridDim.x;
  const long long r1 = a.rows * (blockIdx.x + 1) / gridDim.x;
  Stream<XT, L> sx;
  Stream<BT, L> sy;
  sx.seek(a.x, a.x_stride, r0);
  sx.at = 0;
  sy.at = slot_bytes(blockDim.x, NV, sizeof(XT));
  if (RES) sy.seek(a.y, a.y_stride, r0);
  XT* xo = RES ? static_cast<XT*>(a.x_out) + r0 * a.x_out_stride : nullptr;
  BT* ho = NORM ? static_cast<BT*>(a.h) + r0 * a.h_stride : nullptr;
  const uint32_t slot = sy.at + (RES ? slot_bytes(blockDim.x, NV, sizeof(BT)) : 0), ring_bytes = depth * slot;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);

  int left = (int)(r1 - r0);                   // rows to use, and to copy
  if (turns) {
    left = (int)((tiles - blockIdx.x + gridDim.x - 1) / gridDim.x) * K;
    if ((tiles - 1) % gridDim.x == blockIdx.x) left -= (int)(tiles * K - a.rows);
  }
  int to_copy = left, of_turn = K;
  uint32_t fs = 0, us = 0;                     // slot of the next row to copy, of the next to use
  auto fetch = [&]() {
    if (to_copy > 0) {
      sx.fetch(ring_at + fs, dim);
      if (RES) sy.fetch(ring_at + fs, dim);
      long long step = 1;
      if (--of_turn == 0) {
        of_turn = K;
        step += hop;
      }
      sx.p += step * a.x_stride;
      if (RES) sy.p += step * a.y_stride;
    }
    commit_async();
    --to_copy;
    fs = fs + slot == ring_bytes ? 0 : fs + slot;
  };
  if (RING) {
    for (int d = 0; d < depth; ++d) {
      sx.clear(ring + d * slot, dim);
      if (RES) sy.clear(ring + d * slot, dim);
      fetch();
    }
  }
  count_columns<L>(sh, dim);
  int half = 0;
  long long g = turns ? -1 : r0 / a.rows_per_group - 1;
  int of_group = 0;              // rows until the next modulation group
  Eight gate[NV], times[NV], plus[NV];
  while (left > 0) {
    if (of_group == 0) {
      ++g;
      const long long end = (g + 1) * a.rows_per_group;
      of_group = turns ? left : (int)((end < r1 ? end : r1) - (r1 - left));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (RES) {
          Eight pw;
          load_param<L>(gate[i], a.gate, g * a.gate_stride, a.param_bf16, 1.f, i, dim);
          load_param<L>(pw, a.post_weight, 0, a.param_bf16, 1.f, i, dim);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            gate[i].p[q] = present<L>(mul(gate[i].p[q], mul(both(a.residual_scale), pw.p[q])), i, q, dim);
        }
        if (NORM) {
          // (n w + b)(1 + s) + t = n (w (1 + s)) + (b (1 + s) + t)
          Eight w, b;
          load_param<L>(times[i], a.scale, g * a.scale_stride, a.param_bf16, 0.f, i, dim);
          load_param<L>(plus[i], a.shift, g * a.shift_stride, a.param_bf16, 0.f, i, dim);
          load_param<L>(w, a.weight, 0, a.param_bf16, 1.f, i, dim);
          load_param<L>(b, a.bias, 0, a.param_bf16, 0.f, i, dim);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 s1 = add(both(1.f), times[i].p[q]);
            plus[i].p[q] = fma(b.p[q], s1, plus[i].p[q]);
            times[i].p[q] = mul(w.p[q], s1);
          }
        }
      }
    }
    // N rows of one group at once
    auto rows = [&](auto count) {
      constexpr int N = decltype(count)::value;
      const unsigned char* at[N];
#pragma unroll
      for (int k = 0; k < N; ++k) at[k] = ring + (us + k * slot >= ring_bytes ? us + k * slot - ring_bytes : us + k * slot);
      Eight x[N][NV];              // 0 past the row's end
      if (RES) {
        float m[N], s[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            sy.get(x[k][i], at[k], k * a.y_stride, i, dim);
          }
        if (POST == 2 ? a.post_norm != kNone : POST == 1) {
          row_stats<L, N>(x, a.post_norm, a.post_eps, a.inv_dim, dim, sh, half, nwarps, m, s);
#pragma unroll
          for (int k = 0; k < N; ++k)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q) x[k][i].p[q] = mul(add(x[k][i].p[q], both(-m[k])), both(s[k]));
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            Eight v;
            sx.get(v, at[k], k * a.x_stride, i, dim);
#pragma unroll
            for (int q = 0; q < 4; ++q) x[k][i].p[q] = fma(gate[i].p[q], x[k][i].p[q], v.p[q]);
            store8<L>(xo, x[k][i], i, dim);
          }
          xo += a.x_out_stride;
        }
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            sx.get(x[k][i], at[k], k * a.x_stride, i, dim);
          }
      }
      if (RING) {                 // everything of these rows is in registers: their slots are free
        #pragma unroll
        for (int k = 0; k < N; ++k) fetch();
        us = us + N * slot >= ring_bytes ? us + N * slot - ring_bytes : us + N * slot;
      } else {
        sx.p += N * a.x_stride;
        if (RES) sy.p += N * a.y_stride;
      }
      if (NORM) {
        float m[N], s[N];
        row_stats<L, N>(x, a.norm, a.eps, a.inv_dim, dim, sh, half, nwarps, m, s);
#pragma unroll
        for (int k = 0; k < N; ++k) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              x[k][i].p[q] = fma(mul(add(x[k][i].p[q], both(-m[k])), both(s[k])), times[i].p[q], plus[i].p[q]);
            store8<L>(ho, x[k][i], i, dim);
          }
          ho += a.h_stride;
        }
      }
    };
    const int n = of_group < K ? of_group : K;
    if (RING) wait_async_upto(depth - K);
    if (n == K) {
      rows(std::integral_constant<int, K>());
    } else {
      for (int k = 0; k < n; ++k) rows(std::integral_constant<int, 1>());
    }
    if (!RING) {
      sx.p += hop * a.x_stride;
      if (RES) sy.p += hop * a.y_stride;
    }
    if (RES) xo += hop * a.x_out_stride;
    if (NORM) ho += hop * a.h_stride;
    left -= n;
    of_group -= n;
  }
  if (RING) wait_async<0>();
}

// ----------------------------------------------------------------- launch --
template <typename XT, typename BT, class L, bool RES, bool NORM, int POST>
cudaError_t run(const RowArgs& a, cudaStream_t s) {
  constexpr int K = L::NV == 1 ? (POST == 1 ? 2 : 4) : (L::NV == 2 ? 2 : 1);
  const auto kernel = row_fwd_kernel<XT, BT, L, K, RES, NORM, POST>;
  const int threads = row_threads(a.dim, L::NV);
  // blocks of an SM: by registers (96 a thread), then the ring takes what shared memory is left
  int blocks = 640 / threads < 16 ? 640 / threads : 16;
  if (blocks < 1) blocks = 1;
  const long long resident = (long long)num_sms() * blocks;
  const long long most = a.groups == 1 ? (a.rows + K - 1) / K : a.rows;
  const int grid = (int)(most < resident ? most : resident);
  int depth = 0;
  size_t smem = 0;
  if (L::RING) {
    const size_t slot = slot_bytes(threads, L::NV, sizeof(XT)) + (RES ? slot_bytes(threads, L::NV, sizeof(BT)) : 0);
    const size_t room = kSmemSm / blocks - 1024 - sizeof(Shared<K>);
    const long long rows = (a.rows + grid - 1) / grid;
    depth = (int)(room / slot < kDepthMax ? room / slot : kDepthMax);
    if (rows < depth) depth = (int)(rows > K ? rows : K);
    smem = depth * slot;
    if (smem > 32 * 1024) {      // one value for all launches: callers on other threads may be between theirs and this
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kSmemSm - 1024 - (int)sizeof(Shared<K>));
      if (e != cudaSuccess) return e;
    }
  }
  kernel<<<grid, threads, smem, s>>>(a, depth);
  return cudaGetLastError();
}

template <typename XT, typename BT, class L>
cudaError_t by_op(const RowArgs& a, cudaStream_t s) {
  if (a.y && a.h)
    return a.post_norm == kNone ? run<XT, BT, L, true, true, 0>(a, s)
                                : run<XT, BT, L, true, true, 1>(a, s);
  if (a.y) return run<XT, BT, L, true, false, 2>(a, s);
  return run<XT, BT, L, false, true, 0>(a, s);
}

// Sixteen columns a thread above 2560, so that two blocks share an SM and one
// works while the other waits at a barrier.  Narrow pieces have kernels up to
// 5120 elements; longer rows, and rows above 8192, are read where they are
// used (x' and h of 16384 x 8192 bfloat16 193 us, 1.2 times their bytes; of
// 8192 x 16384, as many bytes, 294).
template <typename XT, typename BT>
cudaError_t by_width(const RowArgs& a, cudaStream_t s) {
  constexpr int P = sizeof(XT) == 2 ? 8 : 4;
  const int p = piece_of(a);
  const bool wide = p == P;
  if (wide && a.dim <= 2560)
    return a.dim % 256 == 0 ? by_op<XT, BT, Layout<P, true, true, 1>>(a, s) : by_op<XT, BT, Layout<P, false, true, 1>>(a, s);
  if (wide && a.dim <= 8192)
    return a.dim % 512 == 0 ? by_op<XT, BT, Layout<P, true, true, 2>>(a, s) : by_op<XT, BT, Layout<P, false, true, 2>>(a, s);
  if (a.dim <= 5120) {
    if constexpr (sizeof(XT) == 2) {
      if (p > 1) return by_op<XT, BT, Layout<2, false, true, 1>>(a, s);
    }
    return by_op<XT, BT, Layout<1, false, sizeof(BT) == 4, 1>>(a, s);
  }
  return wide ? by_op<XT, BT, Layout<P, false, false, 4>>(a, s) : by_op<XT, BT, Layout<1, false, false, 4>>(a, s);
}

}  // namespace

template <typename XT, typename BT>
cudaError_t row_fwd(const RowArgs& a, cudaStream_t s) {
  return by_width<XT, BT>(a, s);
}

}  // namespace spade
