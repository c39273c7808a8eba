// kvq_view.cuh -- read-only view of one block's cache for the kernels that
// walk it token by token (kvq_read.cu, kvq_tree.cu), and the way from a token's
// place in the order of arrival to its slot.
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

struct CacheView {
  const uint8_t* codes;    // progressive cache: [streams][nt][16 KiB]
  const uint32_t* meta;    // [streams][nt][pf][2]
  const uint32_t* kmc;     // per-channel Key groups: [streams][blocks_max][128], else null
  const uint8_t* wcodes;   // sink + window, or staged block: [streams][kWindowTiles][16 KiB], else null
  const uint32_t* wmeta;
  const float* lam;        // [kv_heads][128] or null
  const float* lam_inv;
  int nt, pf, bits, blocks_max;
  int batch, kv_heads;
  long long n_prog;        // tokens in the progressive cache
  int n_win;               // tokens in the window (sink + latest) or staged
  long long n_all;
  bool window;             // sink + window (progressive token i is token i + 1); else staged tokens follow the progressive ones
  Epochs ep;               // of the progressive cache
};

// Slot of progressive token i (order of arrival).
struct Place {
  int tile, slot;
};
__device__ __forceinline__ Place place_of(const Epochs& ep, int i) {
  int e = 0;
  while (e + 1 < ep.n && i >= ep.start[e + 1]) e++;
  const int m = i - ep.start[e], lg = ep.lg_ee[e];
  return Place{m >> lg, ep.h[e] + (m & ((1 << lg) - 1))};
}
// Token (order of arrival, all tokens) in window slot s, with n tokens in all:
// slot 0 is the sink, slot s >= 1 the latest token t with (t - 1) % 128 = s - 1.
__device__ __forceinline__ long long window_token(long long n, int s) {
  if (s == 0) return 0;
  const long long last = n - 2;  // (t - 1) of the latest token
  return last - ((last - (s - 1)) & (kWindowTokens - 1)) + 1;
}

struct ReadArgs {
  CacheView c;
  long long start;
  int n;
  bool f32;
  void* k;  // may be null
  void* v;
  long long k_b, k_t, k_h, v_b, v_t, v_h;
};
cudaError_t launch_read(const ReadArgs& a, cudaStream_t s);

constexpr int kTreeMaxNodes = 1024;
struct TreeArgs {
  CacheView c;
  const void* q;  // bf16
  const void* k;  // drafted Keys, bf16 or f32
  const void* v;
  long long q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h;
  bool f32;
  const unsigned char* mask;  // null: a chain
  long long mask_b;
  int n, q_heads, group;
  float qscale;  // sm_scale * log2(e)
  void* out;     // bf16 [batch][n][q_heads][128]
  ErrWord err;
  void* ws;
  int num_sms;
};
size_t tree_workspace(int num_sms, int rows);
// Few rows (n group <= kTreeNarrowRows) go through the decode kernel: this launch
// lays their queries out as a decode call's, [batch][kv_heads][n group][128],
// leaves the drafted tokens' partial as the last of each stream's nparts and
// takes its ticket (so counters need no clearing before).
constexpr int kTreeNarrowRows = 8;
struct TreeNarrow {
  void* q;        // bf16
  float* parts;
  int* counters;  // [streams]
  int nparts;
};
size_t tree_narrow_bytes(int n_streams, int rows);  // queries and counters
cudaError_t launch_tree_draft(const TreeArgs& a, const TreeNarrow& t, cudaStream_t s);
cudaError_t launch_tree(const TreeArgs& a, const Fill& f, cudaStream_t s);

}  // namespace kvq
