// kvq_tree.cu -- tree attention, host side: how a call's work is divided
// (kvq_tree.cuh has the kernel), and the kernel that joins partial results.
#include "kvq_tree.cuh"

namespace kvq {

extern template cudaError_t launch_tree_bits<2>(const TreePlan& p, cudaStream_t s);
extern template cudaError_t launch_tree_bits<4>(const TreePlan& p, cudaStream_t s);
extern template cudaError_t launch_tree_bits<8>(const TreePlan& p, cudaStream_t s);
extern template cudaError_t launch_tree_bits<16>(const TreePlan& p, cudaStream_t s);

namespace {

// Joins the partial records of one block of rows: a CTA per (stream, block of
// rows, 4 rows), a thread per tensor-memory row (channel).  Every record's max
// and sum come first, all in flight at once; then the weights; then the outputs.
constexpr int kMergeRows = 4;
constexpr int kMergeRecords = 256;  // more than CTAs of a launch
__global__ void __launch_bounds__(kHeadDim) tree_merge_kernel(const __grid_constant__ TreePlan p) {
  __shared__ float wt[kMergeRows][kMergeRecords], ls[kMergeRows][kMergeRecords], sum[kMergeRows];
  __shared__ __align__(16) __nv_bfloat16 sh[kMergeRows][kHeadDim];
  const TreeArgs& a = p.a;
  const int x = blockIdx.x, s = x / p.blocks, block = x - s * p.blocks;
  const int c0 = cta_of(p, x, 0), c1 = cta_of(p, x, p.tiles - 1);
  const int b = s / a.c.kv_heads, j = s - b * a.c.kv_heads;
  const int first = cta_begin(p, c0) == x * p.tiles ? 0 : 1;  // the record of CTA c0
  const float* p0 = p.parts + ((size_t)c0 * 2 + first) * p.rec;
  const float* p1 = p.parts + (size_t)(c0 + 1) * 2 * p.rec;  // record k >= 1 at p1 + (k - 1) 2 rec
  const int nrec = c1 - c0 + 1, rb = blockIdx.y * kMergeRows;
  const int rows = min(kMergeRows, min(p.block_rows, p.rows - block * p.block_rows) - rb);
  pdl_wait();
  if (nrec == 1 || rows <= 0) return;
  auto record = [&](int k) { return k == 0 ? p0 : p1 + (size_t)(k - 1) * 2 * p.rec; };
  for (int i = threadIdx.x; i < nrec * kMergeRows; i += kHeadDim) {
    const int k = i / kMergeRows, r = i % kMergeRows;
    wt[r][k] = r < rows ? __ldcg(record(k) + rb + r) : 0.f;
    ls[r][k] = r < rows ? __ldcg(record(k) + p.block_rows + rb + r) : 0.f;
  }
  __syncthreads();
  {  // warp r: row r
    const int r = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f;
    for (int k = lane; k < nrec; k += 32)
      if (ls[r][k] != 0.f) m = fmaxf(m, wt[r][k]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int k = lane; k < nrec; k += 32) {
      const float w = ls[r][k] != 0.f ? ex2(wt[r][k] - m) : 0.f;
      wt[r][k] = w;
      l = fmaf(w, ls[r][k], l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) sum[r] = l != 0.f ? 1.0f / (value_scale_of(a.c.bits) * l) : 0.f;
  }
  __syncthreads();
  const int ch = channel_of(threadIdx.x);
  float acc[kMergeRows] = {0.f, 0.f, 0.f, 0.f};
  // a record's O is uninitialised where its sum is zero (no tile of the half, or no row)
#pragma unroll 4
  for (int k = 0; k < nrec; k++) {
    const float* o = record(k) + 2 * p.block_rows + rb * kHeadDim + threadIdx.x;
#pragma unroll
    for (int r = 0; r < kMergeRows; r++) {
      const float v = r < rows ? __ldcg(o + r * kHeadDim) : 0.f;
      acc[r] += wt[r][k] != 0.f ? wt[r][k] * v : 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < kMergeRows; r++) sh[r][ch] = __float2bfloat16_rn(acc[r] * sum[r]);
  __syncthreads();
  if (threadIdx.x < kMergeRows * 16) {
    const int i = threadIdx.x >> 4, q = threadIdx.x & 15;
    if (i < rows) {
      const int row = block * p.block_rows + rb + i, node = row / a.group, g = row - node * a.group;
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                               (((long long)b * a.n + node) * a.q_heads + j * a.group + g) * kHeadDim)[q] =
          reinterpret_cast<const uint4*>(sh[i])[q];
    }
  }
}
static_assert(kMergeRows * 32 == kHeadDim, "a warp per row");

// Few rows: the drafted tokens' share of a stream, and its queries for the decode
// kernel.  One CTA per stream: the n R <= 64 scores by warps (a lane four
// channels), then a thread per channel for the output.
__global__ void __launch_bounds__(kHeadDim) tree_draft_kernel(const __grid_constant__ TreeArgs a, const TreeNarrow t) {
  constexpr int kN = kTreeNarrowRows;  // rows, and nodes
  __shared__ float sc[kN][kN];         // score, then weight, of row r and node i
  __shared__ float ml[2][kN];
  __shared__ float nan_of[kN];         // NaN for a row whose query holds one or an infinity, else 0
  const int s = blockIdx.x, b = s / a.c.kv_heads, j = s - b * a.c.kv_heads;
  const int R = a.n * a.group, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();  // the decode launch waits for this kernel before it touches what it writes
  if (threadIdx.x == 0) t.counters[s] = 1;  // this partial's ticket
  // Values beyond what the tree kernel's binary16 operands hold end there too.
  auto limit = [](float x) { return fminf(fmaxf(x, -131008.f), 131008.f); };
  auto load4 = [&](const void* x, long long at, float (&y)[4], bool f32) {
    if (f32) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
      y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x) + at);
      y[0] = __uint_as_float(v.x << 16); y[1] = __uint_as_float(v.x & 0xffff0000u);
      y[2] = __uint_as_float(v.y << 16); y[3] = __uint_as_float(v.y & 0xffff0000u);
    }
  };
  for (int r = warp; r < R; r += 4) {
    const int node = r / a.group, g = r - node * a.group;
    const long long at = b * a.q_b + node * a.q_t + (long long)(j * a.group + g) * a.q_h + 4 * lane;
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(t.q) + ((size_t)s * R + r) * kHeadDim)[lane] =
        *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + at);
    float q[4];
    load4(a.q, at, q, false);
    const float z = ((q[0] + q[1]) + (q[2] + q[3])) * 0.f;
    const bool nan = __any_sync(0xffffffffu, isnan(z));
    if (lane == 0) nan_of[r] = nan ? __int_as_float(0x7fffffff) : 0.f;
    for (int i = 0; i < a.n; i++) {
      const bool see = a.mask ? a.mask[b * a.mask_b + (long long)node * a.n + i] != 0 : i <= node;
      float d = 0.f;
      if (see) {
        float k[4];
        load4(a.k, b * a.k_b + i * a.k_t + j * a.k_h + 4 * lane, k, a.f32);
        d = q[0] * limit(k[0]) + q[1] * limit(k[1]) + q[2] * limit(k[2]) + q[3] * limit(k[3]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (lane == 0) sc[r][i] = see ? d * a.qscale : -INFINITY;
    }
  }
  __syncthreads();
  if (threadIdx.x < kN) {
    const int r = threadIdx.x;
    float m = -INFINITY, l = 0.f;
    if (r < R) {
      for (int i = 0; i < a.n; i++) m = fmaxf(m, sc[r][i]);
      for (int i = 0; i < a.n; i++) {
        const float w = m > -INFINITY ? ex2(sc[r][i] - m) : 0.f;
        sc[r][i] = w;
        l += w;
      }
      l += nan_of[r];  // reaches the joined sum whatever this partial's weight
    }
    ml[0][r] = m;
    ml[1][r] = l;
  }
  __syncthreads();
  float o[kN] = {};
  for (int i = 0; i < a.n; i++) {
    const long long at = b * a.v_b + i * a.v_t + j * a.v_h + threadIdx.x;
    const float v = limit(a.f32 ? static_cast<const float*>(a.v)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.v)[at]));
#pragma unroll
    for (int r = 0; r < kN; r++)
      if (r < R && sc[r][i] != 0.f) o[r] = fmaf(sc[r][i], v, o[r]);  // what a row does not see may be anything
  }
  float* rec = t.parts + ((size_t)s * t.nparts + t.nparts - 1) * kPartFloats;
  if (threadIdx.x < kN) {
    rec[threadIdx.x] = ml[0][threadIdx.x];
    rec[kMaxGroup + threadIdx.x] = ml[1][threadIdx.x];
  }
#pragma unroll
  for (int r = 0; r < kN; r += 4)
    *reinterpret_cast<float4*>(rec + 2 * kMaxGroup + threadIdx.x * kMaxGroup + r) = make_float4(o[r], o[r + 1], o[r + 2], o[r + 3]);
}
static_assert(kTreeNarrowRows == kMaxGroup, "a decode call's query heads per KV head");

}  // namespace

size_t tree_narrow_bytes(int n_streams, int rows) {
  return (size_t)n_streams * rows * kHeadDim * 2 + ((size_t)n_streams * 4 + 15) / 16 * 16;
}

cudaError_t launch_tree_draft(const TreeArgs& a, const TreeNarrow& t, cudaStream_t s) {
  return launch_pdl(tree_draft_kernel, dim3(a.c.batch * a.c.kv_heads), dim3(kHeadDim), 0, s, a, t);
}

size_t tree_workspace(int num_sms, int rows) {
  const int block = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  return (size_t)num_sms * 2 * block * (2 + kHeadDim) * sizeof(float);
}

cudaError_t launch_tree(const TreeArgs& a, const Fill& f, cudaStream_t s) {
  TreePlan p{};
  p.a = a;
  p.f = f;
  p.rows = a.n * a.group;
  p.block_rows = p.rows <= 16 ? 16 : p.rows <= 32 ? 32 : p.rows <= 64 ? 64 : 128;
  p.blocks = (p.rows + p.block_rows - 1) / p.block_rows;
  p.part_group = -1;
  if (a.c.n_prog > 0) {
    p.groups = (int)(a.c.kmc ? a.c.n_prog / kGroupTokens : f.gps);  // per-channel groups: whole blocks, all full
    p.tp = (p.groups + kTileGroups - 1) / kTileGroups;
    if (!a.c.kmc && f.k < f.nt && (f.h + f.r) % kGroupTokens) {  // tile k's last group
      p.part_group = f.k * f.gpt + f.gk - 1;
      p.part_valid = (f.h + f.r) % kGroupTokens;
    }
  }
  p.tw = (a.c.n_win + kTile - 1) / kTile;
  p.td = (a.n + kTile - 1) / kTile;
  p.tiles = p.tp + p.tw + p.td;
  p.extra = kDraftExtra * p.td;
  const long long units = (long long)a.c.batch * a.c.kv_heads * p.blocks * (p.tiles + p.extra);
  if (units > 0x7fffffffLL || a.num_sms < 1) return cudaErrorInvalidValue;
  p.units = (int)units;
  p.grid = (int)std::min<long long>(units, std::min(a.num_sms, kMergeRecords));
  // Two tiles a block of rows (a short context): a CTA takes whole blocks, as
  // joining partial results costs more than the second tile (17.8 against 20.3 us).
  if (p.tiles <= 2 && units / (p.tiles + p.extra) <= a.num_sms) p.grid = (int)(units / (p.tiles + p.extra));
  p.rec = p.block_rows * (2 + kHeadDim);
  p.parts = static_cast<float*>(a.ws);
  cudaError_t e;
  switch (a.c.bits) {
    case 2: e = launch_tree_bits<2>(p, s); break;
    case 4: e = launch_tree_bits<4>(p, s); break;
    case 8: e = launch_tree_bits<8>(p, s); break;
    case 16: e = launch_tree_bits<16>(p, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || p.units % p.grid == 0 && (p.units / p.grid) % (p.tiles + p.extra) == 0) return e;  // every share whole blocks of rows
  return launch_pdl(tree_merge_kernel, dim3((unsigned)(p.units / (p.tiles + p.extra)), (unsigned)((p.block_rows + kMergeRows - 1) / kMergeRows)),
                    dim3(kHeadDim), 0, s, p);
}

}  // namespace kvq
