// kvq_read.cu -- the cache read back as values, in the order of arrival:
//   v = Z + q (R / (2^b - 1)), Keys times lambda,
// each step rounded to fp32, the result to the output's type.
//
// Bound by HBM: 2 (16 b + 4) bytes in and 256 values out per token and head,
// so by the writes at every width.  One warp takes one 16-token group (its
// tokens are 16 consecutive ones of the progressive cache, or 16 slots of the
// window), loads its lane units whole -- lane L the 64 Key and 64 Value codes of
// unit L, contiguous over the warp -- and dequantises in registers.  A Key
// quad is four consecutive channels of one token; Value pairs hold one channel
// of two tokens and are transposed code by code with movmatrix, so every
// lane then holds channels of tokens g and g + 8 for Keys and Values alike and
// needs two (R, Z) pairs.  The 16 rows go through the warp's own shared memory
// (rows padded by 16 bytes: no bank conflicts) and leave as whole rows of
// 16-byte stores.  Measured on a B200 (copy peak 6.46 TB/s): 16 x 32768 tokens of
// 4 heads from 2 bits to bf16 246 us, 4.98 TB/s (issue: ~1000 instructions a group,
// half of the time); 8 x 9001 tokens of 8 heads from 4 bits to fp32 122 us, 5.48
// TB/s.  Codes turned to floats by an OR and a subtraction instead of the
// integer conversion took 266 us, ten CTAs an SM at fewer registers the same.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_decode_common.cuh"
#include "kvq_view.cuh"

namespace kvq {
namespace {

constexpr int kReadWarps = 4;

template <typename T>
__host__ __device__ constexpr int row_pitch() {  // bytes of a row in shared memory
  return kHeadDim * (int)sizeof(T) + 16;
}

template <int N>
__device__ __forceinline__ void put(uint8_t* at, const float (&x)[N], float) {
  if constexpr (N == 4)
    *reinterpret_cast<float4*>(at) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<float2*>(at) = make_float2(x[0], x[1]);
}
template <int N>
__device__ __forceinline__ void put(uint8_t* at, const float (&x)[N], __nv_bfloat16) {
#pragma unroll
  for (int i = 0; i < N; i += 2)
    reinterpret_cast<__nv_bfloat162*>(at)[i / 2] = __floats2bfloat162_rn(x[i], x[i + 1]);
}

__device__ __forceinline__ float low_half(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float high_half(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

// Member i (0..3) of quad p (0..7) of token half x in a Key unit.
template <int BITS>
__device__ __forceinline__ uint32_t key_member(const uint32_t (&u)[2 * BITS], int x, int p, int i) {
  if constexpr (BITS == 16) {
    return (u[x * 16 + 2 * p + (i >> 1)] >> (16 * (i & 1))) & 0xffffu;
  } else {
    constexpr int qpw = 8 / BITS;
    return (u[x * BITS + p / qpw] >> (8 * i + BITS * (p % qpw))) & ((1u << BITS) - 1u);
  }
}
// Pair p (0..15) of token half x in a Value unit, as two 16-bit integers.
template <int BITS>
__device__ __forceinline__ uint32_t value_pair(const uint32_t (&u)[2 * BITS], int x, int p) {
  constexpr int ppw = 16 / BITS;
  constexpr uint32_t m = BITS == 16 ? 0xffffu : (1u << BITS) - 1u;
  return (u[x * BITS + p / ppw] >> (BITS * (p % ppw))) & (m | (m << 16));
}

template <int BITS>
__device__ __forceinline__ void load_unit(uint32_t (&u)[2 * BITS], const uint8_t* part, int lane) {
#pragma unroll
  for (int i = 0; i < 2 * BITS; i += 4) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(part + lane * unit_bytes(BITS)) + i / 4);
    u[i] = w.x; u[i + 1] = w.y; u[i + 2] = w.z; u[i + 3] = w.w;
  }
}

// The warp's 16 rows leave: row i to dst + tok[i] stride, where tok[i] is this
// group's i-th token relative to the range (skipped outside [0, n)).
template <typename T>
__device__ __forceinline__ void flush_rows(const uint8_t* sm, T* dst, long long stride, int n, long long rel, int lane) {
  constexpr int kLanes = kHeadDim * (int)sizeof(T) / 16;  // lanes of a row
#pragma unroll
  for (int i0 = 0; i0 < kGroupTokens; i0 += 32 / kLanes) {
    const int i = i0 + lane / kLanes, c = lane % kLanes;
    const long long r = __shfl_sync(0xffffffffu, rel, i);
    if (r >= 0 && r < n)
      __stcs(reinterpret_cast<uint4*>(dst + r * stride) + c, *reinterpret_cast<const uint4*>(sm + i * row_pitch<T>() + 16 * c));
  }
}

// One group: gbase its codes, meta its 16 (K, V) words, kmc the block's
// per-channel Key words or null; rel: lane i < 16 the place of token i in the
// range (outside: not written).
template <int BITS, typename T>
__device__ __forceinline__ void read_group(const ReadArgs& a, const uint8_t* gbase, const uint32_t* meta, const uint32_t* kmc,
                                           int b, int j, long long rel, uint8_t* sm, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const float qmax = (float)((1u << BITS) - 1u);
  const uint2 m[2] = {__ldg(reinterpret_cast<const uint2*>(meta) + g), __ldg(reinterpret_cast<const uint2*>(meta) + g + 8)};
  uint32_t ku[2 * BITS], vu[2 * BITS];
  if (a.k) load_unit<BITS>(ku, gbase, lane);
  if (a.v) load_unit<BITS>(vu, gbase + part_bytes(BITS), lane);
  if (a.k) {
    float z[2], s[2];
#pragma unroll
    for (int x = 0; x < 2; x++) {
      z[x] = high_half(m[x].x);
      s[x] = __fdiv_rn(low_half(m[x].x), qmax);
    }
    const float4* lam = a.c.lam ? reinterpret_cast<const float4*>(a.c.lam + (size_t)j * kHeadDim) : nullptr;
#pragma unroll
    for (int p = 0; p < 8; p++) {
      const int c = 16 * p + 4 * t;  // 32 s + 16 r + 4 t with p = 2 s + r
      const float4 lv = lam ? __ldg(lam + c / 4) : make_float4(1.f, 1.f, 1.f, 1.f);
      const float l[4] = {lv.x, lv.y, lv.z, lv.w};
      float zc[4], scl[4];
      if (kmc) {
        const uint4 w4 = __ldg(reinterpret_cast<const uint4*>(kmc + c));
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
          zc[i] = high_half(w[i]);
          scl[i] = __fdiv_rn(low_half(w[i]), qmax);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; x++) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float q = (float)key_member<BITS>(ku, x, p, i);
          y[i] = __fmul_rn(__fadd_rn(__fmul_rn(q, kmc ? scl[i] : s[x]), kmc ? zc[i] : z[x]), l[i]);
        }
        put(sm + (g + 8 * x) * row_pitch<T>() + c * sizeof(T), y, T());
      }
    }
    __syncwarp();
    flush_rows(sm, static_cast<T*>(a.k) + b * a.k_b + j * a.k_h, a.k_t, a.n, rel, lane);
    __syncwarp();
  }
  if (a.v) {
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const float z = high_half(m[x].y), s = __fdiv_rn(low_half(m[x].y), qmax);
#pragma unroll
      for (int p = 0; p < 16; p++) {
        const uint32_t w = movmatrix_t(value_pair<BITS>(vu, x, p));  // token g + 8 x, channels 8 p + 2 t, + 1
        const float y[2] = {__fadd_rn(__fmul_rn((float)(w & 0xffffu), s), z), __fadd_rn(__fmul_rn((float)(w >> 16), s), z)};
        put(sm + (g + 8 * x) * row_pitch<T>() + (8 * p + 2 * t) * sizeof(T), y, T());
      }
    }
    __syncwarp();
    flush_rows(sm, static_cast<T*>(a.v) + b * a.v_b + j * a.v_h, a.v_t, a.n, rel, lane);
  }
}

// Groups [g0, g0 + n) of every stream's progressive cache (in the order of
// arrival), or (WIN) of the window or the staged block.  Heads run fastest over
// the warps: neighbouring warps write neighbouring rows of the output.
template <int BITS, typename T, bool WIN>
__global__ void __launch_bounds__(kReadWarps * 32) read_kernel(const ReadArgs a, int g0, int n) {
  __shared__ __align__(16) uint8_t smem[kReadWarps][kGroupTokens * row_pitch<T>()];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kReadWarps + warp;
  const int per = n * a.c.kv_heads;
  if (unit >= (long long)a.c.batch * per) return;
  const int b = (int)(unit / per), rest = (int)(unit - (long long)b * per), u = rest / a.c.kv_heads, j = rest - u * a.c.kv_heads;
  const int s = b * a.c.kv_heads + j;
  const long long shift = a.c.window ? 1 : 0;  // progressive token i is token i + 1 after the sink
  if constexpr (!WIN) {
    const int i0 = kGroupTokens * (g0 + u);
    const Place pl = place_of(a.c.ep, i0);
    const size_t tile = (size_t)s * a.c.nt + pl.tile;
    const uint32_t* kmc =
        a.c.kmc ? a.c.kmc + ((size_t)s * a.c.blocks_max + (size_t)(i0 / kKeyBlock)) * kHeadDim : nullptr;
    const long long i = i0 + lane;
    const long long rel = lane < kGroupTokens && i < a.c.n_prog ? i + shift - a.start : -1;
    read_group<BITS, T>(a, a.c.codes + tile * kTileBytes + (size_t)(pl.slot >> 4) * group_bytes(BITS),
                        a.c.meta + (tile * a.c.pf + pl.slot) * 2, kmc, b, j, rel, smem[warp], lane);
  } else {
    constexpr int kGroups = slots_per_tile(16) / kGroupTokens;  // groups of a 16-bit tile
    const int slot = kGroupTokens * u + lane;
    const size_t tile = (size_t)s * kWindowTiles + u / kGroups;
    const int first = kGroupTokens * (u % kGroups);
    const long long tok = a.c.window ? window_token(a.c.n_all, slot) : a.c.n_prog + slot;
    const long long rel = lane < kGroupTokens && slot < a.c.n_win ? tok - a.start : -1;
    read_group<16, T>(a, a.c.wcodes + tile * kTileBytes + (size_t)(u % kGroups) * group_bytes(16),
                      a.c.wmeta + (tile * slots_per_tile(16) + first) * 2, nullptr, b, j, rel, smem[warp], lane);
  }
}

template <int BITS, bool WIN>
cudaError_t launch_bits(const ReadArgs& a, int g0, int n, cudaStream_t s) {
  const long long units = (long long)a.c.batch * a.c.kv_heads * n;
  if (units == 0) return cudaSuccess;
  const long long ctas = (units + kReadWarps - 1) / kReadWarps;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.f32)
    read_kernel<BITS, float, WIN><<<(unsigned)ctas, kReadWarps * 32, 0, s>>>(a, g0, n);
  else
    read_kernel<BITS, __nv_bfloat16, WIN><<<(unsigned)ctas, kReadWarps * 32, 0, s>>>(a, g0, n);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, cudaStream_t s) {
  // progressive tokens of the range, in whole groups
  const long long shift = a.c.window ? 1 : 0;
  long long p0 = a.start - shift, p1 = a.start + a.n - shift;
  if (p0 < 0) p0 = 0;
  if (p1 > a.c.n_prog) p1 = a.c.n_prog;
  int g0 = 0, pg = 0;
  if (p0 < p1) {
    g0 = (int)(p0 / kGroupTokens);
    pg = (int)((p1 + kGroupTokens - 1) / kGroupTokens) - g0;
  }
  // the window holds token 0 and the latest ones; staged tokens follow the progressive ones
  const bool tail = a.c.n_win > 0 && (a.start + a.n > a.c.n_prog + shift || (a.c.window && a.start == 0));
  const int wg = tail ? (a.c.n_win + kGroupTokens - 1) / kGroupTokens : 0;
  if (cudaError_t e = launch_bits<16, true>(a, 0, wg, s)) return e;
  switch (a.c.bits) {
    case 2: return launch_bits<2, false>(a, g0, pg, s);
    case 4: return launch_bits<4, false>(a, g0, pg, s);
    case 8: return launch_bits<8, false>(a, g0, pg, s);
    case 16: return launch_bits<16, false>(a, g0, pg, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
