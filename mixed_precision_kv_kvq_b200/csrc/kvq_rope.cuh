// kvq_rope.cuh -- launch interface of the rotary kernel (kvq_rope.cu).
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

// One tensor [batch][n][heads][128]: strides in elements, in and out.
struct RopeRows {
  const void* in;
  void* out;
  int heads;  // 0: absent
  long long in_b, in_t, in_h, out_b, out_t, out_h;
};

struct RopeArgs {
  RopeRows q, k;
  const void* pos;  // int32 or int64 positions at [b pos_b + t pos_t]
  bool pos64;
  long long pos_b, pos_t;
  long long n, tokens;  // tokens per sequence; batch * n
  int rot_dim, tokens_per_cta;
  int align;  // largest power of two (at most 16) that divides every row's address
  float mag;
  unsigned long long turn[kHeadDim / 2];  // 2^64 w_p / (2 pi) modulo 2^64
};

cudaError_t launch_rope(const RopeArgs& a, bool interleaved, bool f32, cudaStream_t s);

}  // namespace kvq
