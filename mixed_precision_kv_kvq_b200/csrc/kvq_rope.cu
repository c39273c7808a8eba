// kvq_rope.cu -- rotary positions for queries and Keys, one launch for both.
//
// A pair (x0, x1) of one head at position m is turned by the angle m w_p, w_p
// the pair's frequency (radians per position):
//   y0 = (x0 cos - x1 sin) mag,   y1 = (x1 cos + x0 sin) mag.
// Pairs are (p, p + rot_dim / 2) (KVQ_ROPE_HALF) or (2p, 2p + 1)
// (KVQ_ROPE_INTERLEAVED); channels from rot_dim on pass unchanged.
//
// Angles.  At position 10^6 an fp32 product m w_p is off by ~0.06 rad, so the
// phase is kept as an integer: the host turns w_p into 2^64 w_p / (2 pi)
// modulo 2^64, rounded once, and m times that, modulo 2^64, is the fraction of a
// turn up to |m| 2^-65 of a turn, whatever the frequency.  Its top 32 bits become
// the angle in half turns, in [-1, 1), for sincospif: 2 pi 2^-26 rad more (one
// rounding to fp32) and that function's own error.
//
// The kernel is bound by HBM (each value read once and written once).  A CTA
// takes four tokens, or one where there are few (RopeArgs::tokens_per_cta): its
// threads first form the tokens' cos and sin, one pair each, in shared memory --
// every head of a token shares them -- and then walk the rows (token, head), a
// thread always at the same chunk of the head, with 16-byte accesses (8 bytes
// where rot_dim / 2 or the rows' alignment allows no more; single elements, or
// pairs, for any other).  Measured on a B200 (copy peak 6.46 TB/s): 8 x 4096
// tokens of 64 + 8 heads, bf16, 202 us, 5.98 TB/s; 3 x 1001 tokens of 40 + 8
// heads, fp32, half of each head turned, 32 us, 4.60 TB/s; one token of 16
// sequences, 28 + 4 heads, 2.9 us in a graph (launch latency).
#include <cuda_bf16.h>

#include "kvq_rope.cuh"

namespace kvq {
namespace {

constexpr int kRopeThreads = 256;

template <int V, typename T>
struct alignas(V * sizeof(T)) Pack {
  T v[V];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// A chunk of a head: V channels (INTER: V/2 neighbouring pairs) or V pairs (the
// channels c .. c+V-1 and those rot_dim/2 further on), or as many that pass.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];  // [tokens of the CTA][rot_dim / 2]
  const int half = a.rot_dim >> 1;
  const long long tok0 = (long long)blockIdx.x * a.tokens_per_cta;
  const int nt = (int)min((long long)a.tokens_per_cta, a.tokens - tok0);
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tt = i / half, p = i - tt * half;
    const long long tok = tok0 + tt, b = tok / a.n, t = tok - b * a.n;
    const long long at = b * a.pos_b + t * a.pos_t;
    const long long m = a.pos64 ? static_cast<const long long*>(a.pos)[at] : (long long)static_cast<const int*>(a.pos)[at];
    const unsigned long long phase = (unsigned long long)m * a.turn[p];
    float s, c;
    sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
    cs[i] = make_float2(c * a.mag, s * a.mag);
  }
  __syncthreads();
  // A thread keeps its chunk of the head and walks the rows (token, head).  One
  // row in flight a thread and eight CTAs an SM: two or four rows a thread cost
  // registers and so CTAs (a 1.2 GB bf16 call: 248 and 397 us against 214).
  constexpr int kPer = INTER ? V : 2 * V;  // channels per chunk
  const int turned = a.rot_dim / kPer, chunks = kHeadDim / kPer;  // kPer divides rot_dim (launch_t)
  const int heads = a.q.heads + a.k.heads, rows = nt * heads, step = kRopeThreads / chunks;
  const int ch = threadIdx.x % chunks;
  if ((int)threadIdx.x / chunks >= step) return;
  // the chunk's two packs: channels c0 .. and c1 .. (one pack of pairs: c1 = c0)
  const bool turn = ch < turned;
  const int c0 = turn ? ch * V : a.rot_dim + (ch - turned) * kPer;
  const int c1 = INTER ? c0 : turn ? c0 + half : c0 + V;
  for (int r = threadIdx.x / chunks; r < rows; r += step) {
    const int tt = r / heads, hh = r - tt * heads;
    const bool is_k = hh >= a.q.heads;
    const RopeRows& x = is_k ? a.k : a.q;
    const int h = is_k ? hh - a.q.heads : hh;
    const long long tok = tok0 + tt, b = tok / a.n, t = tok - b * a.n;
    const T* src = static_cast<const T*>(x.in) + b * x.in_b + t * x.in_t + h * x.in_h;
    T* dst = static_cast<T*>(x.out) + b * x.out_b + t * x.out_t + h * x.out_h;
    Pack<V, T> y0 = *reinterpret_cast<const Pack<V, T>*>(src + c0), y1;
    if constexpr (!INTER) y1 = *reinterpret_cast<const Pack<V, T>*>(src + c1);
    if (turn) {
      const float2* w = cs + tt * half;
      if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float2 f = w[(c0 + e) >> 1];
          const float x0 = to_f(y0.v[e]), x1 = to_f(y0.v[e + 1]);
          from_f(x0 * f.x - x1 * f.y, y0.v[e]);
          from_f(x1 * f.x + x0 * f.y, y0.v[e + 1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; e++) {
          const float2 f = w[c0 + e];
          const float x0 = to_f(y0.v[e]), x1 = to_f(y1.v[e]);
          from_f(x0 * f.x - x1 * f.y, y0.v[e]);
          from_f(x1 * f.x + x0 * f.y, y1.v[e]);
        }
      }
    }
    *reinterpret_cast<Pack<V, T>*>(dst + c0) = y0;
    if constexpr (!INTER) *reinterpret_cast<Pack<V, T>*>(dst + c1) = y1;
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch_v(const RopeArgs& a, cudaStream_t s) {
  const long long ctas = (a.tokens + a.tokens_per_cta - 1) / a.tokens_per_cta;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t smem = (size_t)a.tokens_per_cta * (a.rot_dim / 2) * sizeof(float2);
  rope_kernel<T, V, INTER><<<(unsigned)ctas, kRopeThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, bool inter, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);  // elements of a 16-byte access
  // the widest pack that every row's alignment and the pairs' layout allow
  const int fit = inter ? a.rot_dim : a.rot_dim / 2;
  if (a.align % 16 == 0 && fit % W == 0) return inter ? launch_v<T, W, true>(a, s) : launch_v<T, W, false>(a, s);
  if (a.align % 8 == 0 && fit % (W / 2) == 0) return inter ? launch_v<T, W / 2, true>(a, s) : launch_v<T, W / 2, false>(a, s);
  if (inter && a.align % (2 * (int)sizeof(T)) == 0) return launch_v<T, 2, true>(a, s);
  if (inter) return cudaErrorInvalidValue;  // the entry point asks for pairs on their own alignment
  return launch_v<T, 1, false>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool inter, bool f32, cudaStream_t s) {
  return f32 ? launch_t<float>(a, inter, s) : launch_t<__nv_bfloat16>(a, inter, s);
}

}  // namespace kvq
