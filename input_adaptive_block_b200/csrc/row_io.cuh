// Row access and reductions shared by the row passes around the attention
// (k_qk_rope.cu, k_row_norm.cu): eight-element loads and stores of float32 or
// bfloat16 rows, and block-wide sums and moments in float32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace spade {
namespace rowio {

// Eight elements as they lie in memory: 16 bytes of bfloat16, 32 of float32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
};
template <>
struct Raw8<float> {
  float4 a, b;
};

__device__ __forceinline__ void load_raw(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p) {
  r.u = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void load_raw(Raw8<float>& r, const float* p) {
  r.a = *reinterpret_cast<const float4*>(p);
  r.b = *reinterpret_cast<const float4*>(p + 4);
}
__device__ __forceinline__ void clear_raw(Raw8<__nv_bfloat16>& r) { r.u = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void clear_raw(Raw8<float>& r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }

// bfloat16 is the upper half of a float32: the low element of a word shifts
// up, the high one is masked.
__device__ __forceinline__ void unpack(float (&v)[8], const Raw8<__nv_bfloat16>& r) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(float (&v)[8], const Raw8<float>& r) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}

__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store_vec(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Scratch of block_sum for up to M values at once, in two halves.
template <int M>
struct SumScratch {
  float v[2][M * 32];
};

// Sums of K values over the block, the same in every thread.  Calls on one
// scratch alternate its halves, whatever their K, so one barrier per call is
// enough: a half is written again only after the next call's barrier, which
// every thread reaches after its reads of this one.  One-warp blocks need no
// barrier.
template <int K, int M>
__device__ __forceinline__ void block_sum(float (&v)[K], SumScratch<M>& buf, int& half, int nwarps) {
  static_assert(K <= M, "scratch too small");
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (nwarps == 1) return;
  float* b = buf.v[half];
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) b[k * 32 + (threadIdx.x >> 5)] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float s = 0.f;
    for (int w = 0; w < nwarps; ++w) s += b[k * 32 + w];
    v[k] = s;
  }
  half ^= 1;
}

}  // namespace rowio
}  // namespace spade
