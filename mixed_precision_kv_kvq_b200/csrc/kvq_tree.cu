// kvq_tree.cu -- attention of a tree of drafted tokens over the packed cache
// and over one another (kvq_tree_attn).
//
// One CTA per (query row, stream): its warps take the cached and the drafted
// tokens in turn, each lane four channels, with an online softmax per warp;
// the warps' states are joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_decode_common.cuh"
#include "kvq_view.cuh"

namespace kvq {
namespace {

constexpr int kTreeWarps = 8;

__device__ __forceinline__ float lo16(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float hi16(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

struct State {
  float m, l, o[4];
};
__device__ __forceinline__ void step(State& st, const float (&q)[4], const float (&k)[4], const float (&v)[4]) {
  float d = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
  for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  const float m = fmaxf(st.m, d), f = exp2f(st.m - m), p = exp2f(d - m);
  st.m = m;
  st.l = st.l * f + p;
#pragma unroll
  for (int i = 0; i < 4; i++) st.o[i] = st.o[i] * f + p * v[i];
}

__global__ void __launch_bounds__(kTreeWarps * 32) tree_kernel(const TreeArgs a) {
  const CacheView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.y, b = s / c.kv_heads, j = s - b * c.kv_heads;
  const int node = blockIdx.x / a.group, h = j * a.group + blockIdx.x % a.group;
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_b + node * a.q_t + h * a.q_h + 4 * lane;
  float qd[4], qc[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    qd[i] = __bfloat162float(qp[i]) * a.qscale;
    qc[i] = qd[i] * (c.lam ? c.lam[j * kHeadDim + 4 * lane + i] : 1.f);
  }
  State st{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
  for (int seg = 0; seg < 2; seg++) {
    const int n = seg == 0 ? (int)c.n_prog : c.n_win;
    const int bits = seg == 0 ? c.bits : 16;
    const float inv = 1.0f / (float)((1u << bits) - 1u);
    for (int i = warp; i < n; i += kTreeWarps) {
      const Place pl = seg == 0 ? place_of(c.ep, i) : Place{i / slots_per_tile(16), i % slots_per_tile(16)};
      const size_t tile = (size_t)s * (seg == 0 ? c.nt : kWindowTiles) + pl.tile;
      const uint8_t* gb = (seg == 0 ? c.codes : c.wcodes) + tile * kTileBytes + (size_t)(pl.slot >> 4) * group_bytes(bits);
      const uint32_t* mt = (seg == 0 ? c.meta : c.wmeta) + (tile * (seg == 0 ? c.pf : slots_per_tile(16)) + pl.slot) * 2;
      float k[4], v[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int ch = 4 * lane + e;
        uint32_t km = mt[0];
        if (seg == 0 && c.kmc) km = c.kmc[((size_t)s * c.blocks_max + i / kKeyBlock) * kHeadDim + ch];
        k[e] = hi16(km) + (float)key_code(gb, bits, pl.slot & 15, ch) * (lo16(km) * inv);
        v[e] = hi16(mt[1]) + (float)value_code(gb, bits, pl.slot & 15, ch) * (lo16(mt[1]) * inv);
      }
      step(st, qc, k, v);
    }
  }
  for (int i = warp; i < a.n; i += kTreeWarps) {
    const bool seen = a.mask ? a.mask[b * a.mask_b + (long long)node * a.n + i] != 0 : i <= node;
    if (!seen) continue;
    float k[4], v[4];
    const long long ko = b * a.k_b + i * a.k_t + j * a.k_h + 4 * lane, vo = b * a.v_b + i * a.v_t + j * a.v_h + 4 * lane;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      k[e] = a.f32 ? static_cast<const float*>(a.k)[ko + e] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.k)[ko + e]);
      v[e] = a.f32 ? static_cast<const float*>(a.v)[vo + e] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.v)[vo + e]);
    }
    step(st, qd, k, v);
  }
  __shared__ float sm[kTreeWarps], sl[kTreeWarps], so[kTreeWarps][kHeadDim];
  if (lane == 0) {
    sm[warp] = st.m;
    sl[warp] = st.l;
  }
#pragma unroll
  for (int e = 0; e < 4; e++) so[warp][4 * lane + e] = st.o[e];
  __syncthreads();
  if (threadIdx.x < kHeadDim) {
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int w = 0; w < kTreeWarps; w++) m = fmaxf(m, sm[w]);
    for (int w = 0; w < kTreeWarps; w++) {
      const float f = sl[w] > 0.f ? exp2f(sm[w] - m) : 0.f;
      l += f * sl[w];
      o += f * so[w][threadIdx.x];
    }
    static_cast<__nv_bfloat16*>(a.out)[(((long long)b * a.n + node) * a.q_heads + h) * kHeadDim + threadIdx.x] =
        __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
  }
}

}  // namespace

size_t tree_workspace(int num_sms) { return (size_t)num_sms * 16; }

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  tree_kernel<<<dim3(a.n * a.group, a.c.batch * a.c.kv_heads), kTreeWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
