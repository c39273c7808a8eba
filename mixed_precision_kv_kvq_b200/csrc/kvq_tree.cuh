// kvq_tree.cuh -- attention of a tree of drafted tokens over the packed cache
// and over one another (kvq_tree_attn).
//
// For one (sequence, KV head) stream the n nodes' G query heads are R = n G
// rows r, and with s the scores in log2 units
//   s[t][r] = (q_r lambda sm_scale log2 e) . k^_t          (cached token t)
//   out_r   = sum_t 2^(s[t][r] - m_r) v^_t / sum_t 2^(s[t][r] - m_r),
// the drafted tokens being further tokens t that a mask hides from some rows.
//
// Products on tcgen05, tokens as rows.  A tile is 128 tokens.  Both products
// take their left operand from tensor memory and a narrow right operand from
// shared memory, so their cost follows the number of query rows (16, 32 or 64
// columns a half, below) and not a fixed 128:
//   S[token][row]   = K[token][channel]   Q[row][channel]^T
//   O[channel][row] += V[token][channel]^T P[token][row]
// The cache's lane units are what tcgen05.st takes: lane 4g + t of a warp
// holds tokens g, g + 8 and four neighbouring channels of each Key quad
// (16x256b: rows lane / 4 and + 8, two columns a lane), and one channel of two
// neighbouring tokens in each Value pair (16x128b, one column a lane), so
// codes are widened in registers and stored once, with no transposition.
// Codes become val = (c - 2^(b-1)) 2^(1-b), exact in fp16 at 8 bits and fewer
// (rounded to 11 bits at 16).  With rk = R 2^(b-1) / (2^b - 1) a Key is
// (Z + rk) + rk val, and the score
//   s = rk (q' . val + a sum(q')) - m,   a = (Z + rk) / rk.
// Keys go in as val, and a sum(q') by one more k-step (below); rk and -m are
// applied in fp32 by the thread that owns the token.  (Keys rounded to fp16 as
// whole values took the bf16 output from 0.17% to 0.28% off where outlier
// channels dominate: their errors differ from token to token, while the
// query's are common to the tokens that matter.)  Drafted Keys and those of
// per-channel groups go in as fp16 values, rk a constant and a = 0.
// Values go in as one fma from val: x g = val R/4 + (Z g + R/4), g = (1 - 2^-b) / 2:
// with this g R/4 is exact, the value is rounded twice (its centre Z g + R/4,
// then itself), and nothing in binary16's range overflows.
// S has a token per tensor-memory lane: a thread owns one token and walks the
// rows, so a token's rk and whether it counts are registers, P is written row by
// row as the K-slices that an MN-major operand wants (16-byte stores, 128-byte
// swizzle), and row sums are per-thread partial sums until the end.  The extra
// k-step of the scores multiplies (a, a, a's low part) with (sum(q'), its low
// part, sum(q')), fp16 pairs of 22 bits, so that a row's only term at the softmax is
// -m, four rows an LDS.128 (with sum(q') there too, the loads took ~1000 cycles
// of a tile's 3800).  The running maximum m of a row is shared by the 128
// threads; it moves only when some score exceeds it by more than 2^8 (one vote
// per 32 rows), and only then are column maxima formed and O rescaled in
// tensor memory.
//
// Roles (one CTA per SM, which holds all 512 tensor-memory columns): 8 or 16
// softmax warps, groups of four widening warps, one warp streaming packed tiles
// with bulk copies, two issuing MMAs.  The softmax warps form two halves, each
// with an issuer, S, P, Q and O of its own.  With up to 64 rows the halves take
// alternate tiles of the same rows (two independent softmax states, joined at
// the end); above, each takes 64 of 128 rows of every tile.  Two widened tiles
// fit beside S and O; the widening warps of a buffer (four, or eight that share
// a tile's groups where few rows leave them more of the work) take every second
// tile whole, so the fixed cost of a tile (waits, fences) falls on few warps.
//
// Phases.  A wait tells apart only two successive phases of a barrier, so every
// waiter has to see each phase of the barriers it waits on: the ring is one
// ring per buffer (its slots are never read by the other buffer's warps), and
// in alternate tiles a buffer belongs to one half.
//
// Work split: the (stream, block of rows, tile) units form one line that is cut
// evenly over the grid; a CTA writes the rows it covers whole, and leaves a
// partial (max, sum, O) of at most two others in the workspace, which
// tree_merge_kernel joins.
//
// Every block of up to 128 rows streams and widens the stream's cache again.
// Measured on a B200 (graph replay): 16 nodes of 7 heads over 16 x 32768 2-bit
// tokens of 4 heads 206 us, 585 TFLOP/s; 63 nodes of 8 heads over 8 x 16383 8-bit
// tokens of 8 heads 439 us, 620 TFLOP/s (four blocks of rows; 495 us in a run of
// many, under the power cap); 4 nodes of 7 heads over 16 x 32701 4-bit tokens of 4
// heads 158 us; 5 nodes of 5 heads over 4 x 4999 16-bit tokens of 8 heads 50 us, 1.7
// TB/s (84 MB, of which L2 may hold a part from one replay to the next); one tile
// a CTA 14 us (query set-up, cold instructions, the drafted tile's scattered loads).
// A 128 x 128 tile takes ~2700 cycles, against ~1300 of MMA and 1024 of ex2 at
// 16 an SM and cycle.  A half's loop is its score product (~1800 cycles from its
// issue until it is in, the other half's products between), 220 until it is in
// registers and S is free, and ~500 until the next is issued; S is single, as
// tensor memory is full.  (S held until the maxima were agreed on: 220 us where it
// is 206; of those 220, 208 were left without any widening at all.)
// At 16 bits a tile is 64 KiB and two ring stages are what fits.  Every wait is bounded: a wait that gives up raises
// the cache's error flag and the CTA's abort flag, after which all waits return
// at once and the loops run out.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_decode_common.cuh"
#include "kvq_view.cuh"

namespace kvq {

struct TreePlan {
  TreeArgs a;
  Fill f;               // progressive cache (group order)
  int groups;           // groups of a stream's progressive cache
  int part_group, part_valid;  // the one group that may be partial, and its tokens
  int rows, block_rows, blocks;  // query rows of a stream, rows per block, blocks
  int tp, tw, td, tiles;         // progressive, window and drafted tiles of a stream
  int extra, units, grid;
  int rec;              // floats of one partial record
  float* parts;         // [grid][2][rec]: m[block_rows], l[block_rows], O[block_rows][128]
};

// A CTA's share.  The line's units are the tiles of every (stream, block of rows),
// drafted tiles counting 1 + kDraftExtra each (their scattered rows and mask words
// cost about four packed tiles; at the end of their block): units
// are cut evenly, a cut inside a drafted tile moves to the block's end, and
// tile_at gives it as a tile of the line, block * tiles + tile.
constexpr int kDraftExtra = 3;
__host__ __device__ __forceinline__ int cta_begin(const TreePlan& p, int i) {
  const int per = p.tiles + p.extra, v = (int)((long long)p.units * i / p.grid), x = v / per;
  const int t = v - x * per;
  return x * p.tiles + (t < p.tiles ? t : p.tiles);
}
__host__ __device__ __forceinline__ int cta_of(const TreePlan& p, int block, int tile) {
  const long long v = (long long)block * (p.tiles + p.extra) + tile;
  return (int)(((v + 1) * p.grid - 1) / p.units);
}

// The kernel for caches of BITS bits (kvq_tree_<BITS>.cu).
template <int BITS>
cudaError_t launch_tree_bits(const TreePlan& p, cudaStream_t s);

namespace {

constexpr int kTile = 128;           // tokens per tile
constexpr int kTileGroups = kTile / kGroupTokens;
constexpr int kMaxStages = 8;
constexpr int kHalfRows = 64;        // rows of a half's operands in shared memory
constexpr int kQBytes = kHalfRows * kHeadDim * 2;  // one half's Q: two 64-channel slabs of [64][128 B]
constexpr int kPBytes = kTile * 128;               // one half's P: [128 tokens][64 rows] fp16
// -m of a row with no token yet (0 - m is never -0)
constexpr uint32_t kUnsetBits = 0x80000000u;
__device__ __forceinline__ bool unset(float neg) { return __float_as_uint(neg) == kUnsetBits; }

// How the warps are divided, the registers of each kind (setmaxnreg from what the
// launch gives) and tensor memory's columns.  With 64 rows a half (128 rows a
// CTA, or 64 in alternate tiles) a half's rows are divided over two
// warpgroups: 32 rows a thread is what its registers hold.
template <int COLS>
struct Split {
  static constexpr int kSoft = COLS == 64 ? 16 : 8;       // softmax warps
  static constexpr int kShare = COLS == 64 ? 1 : 2;       // widening groups that share a tile
  static constexpr int kWiden = 8 * kShare;               // widening warps: groups of 4 for each of the two buffers
  static constexpr int kWarps = kSoft + kWiden + 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kSubs = kSoft / 8;                 // softmax warpgroups per half
  static constexpr int kCols = COLS / kSubs;              // rows per softmax thread
  static constexpr int kRegs = 72;                        // at launch
  static constexpr int kSoftRegs = COLS == 64 ? 88 : COLS == 32 ? 96 : 80;
  static constexpr int kWidenRegs = COLS == 64 ? 64 : COLS == 32 ? 72 : 80;
  static constexpr int kCtlRegs = 24;
  static_assert(kWarps == 28 && 65536 / kThreads / 8 * 8 == kRegs);
  static_assert(32 * (kSoft * kSoftRegs + kWiden * kWidenRegs + 4 * kCtlRegs) <= kThreads * kRegs);
  static constexpr uint32_t kStep = COLS == 64 ? 64 : 32;  // columns of one half's S or O
  static constexpr uint32_t kColS = 0, kColO = 2 * kStep, kColK = 4 * kStep, kColV = kColK + 128;
  static_assert(kColV + 128 <= 512);
};
constexpr int kCentreBytes = kTile * 32;           // a of one buffer's tokens: [128][16] fp16
constexpr int kSumBytes = kHalfRows * 32;          // sum(q') of one half's rows: [64][16] fp16
constexpr float kSumScale = 16.0f;                 // sum(q') / 16 and 16 a: up to 10^6 and 4000
constexpr float kCentreMax = 4000.0f;

struct Small {
  float rk[4][kTile];                // of the tokens of tile t, ring of 4
  float neg[2][kHalfRows];           // per half: -m
  float alpha[2][kHalfRows];         // factor of the last rescaling
  float shift[2][kHalfRows];         // what it added to -m
  float red[2][4][kHalfRows];        // per warp: column maxima, then row sums
  float2 ml[2][kHalfRows];           // final (m, l)
  uint32_t seen[4][kTile][4];        // drafted tile t: bit i of word w: the row sees token 32 w + i
  uint64_t ring_full[kMaxStages], ring_free[kMaxStages];
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t q_full[2], s_full[2], s_free[2], p_full[2], pv_done[2], drain[2];
  uint32_t tmem;
  volatile int abort;
};
constexpr int kSmallBytes = (sizeof(Small) + 1023) / 1024 * 1024;
constexpr int kSmemMax = 227 * 1024 - 1024;  // the base is aligned by hand

// Shared memory: Q of both halves, P of both, the operands of the extra k-step,
// Small, the ring.  (A second P buffer a half, so that a tile's
// probabilities need not wait for the product of the tile before, gained
// nothing: 211 against 207 us for 112 rows over 32K 2-bit tokens.)
template <int BITS>
struct Layout {
  static constexpr int kP = 2 * kQBytes;
  static constexpr int kCentre = kP + 2 * kPBytes;
  static constexpr int kSum = kCentre + 2 * kCentreBytes;
  static constexpr int kSmall = kSum + 2 * kSumBytes;
  static constexpr int kRing = kSmall + kSmallBytes;
  static constexpr int kStage = kTileGroups * (group_bytes(BITS) + 128) + 4 * kHeadDim;
  static constexpr int kFit = (kSmemMax - kRing) / kStage;
  static constexpr int kStages = (kFit < kMaxStages ? kFit : kMaxStages) / 2 * 2;  // one ring per buffer
  static constexpr int kBytes = kRing + kStages * kStage + 1024;
  static_assert(kStages >= 2);
};

// ------------------------------------------------------------------ PTX

// Up to 64 tests, each of which may suspend the warp for a while.  A loop of two
// instructions: waiting warps share the schedulers with working ones.
__device__ __forceinline__ bool mbar_try_many(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 64;\n"
      "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra done;\n"
      " add.u32 n, n, -1;\n setp.ne.u32 q, n, 0;\n @q bra again;\n"
      "done:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Whether a phase is complete, without suspending.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait: gives up after kWaitNs or once another wait of the CTA has.
__device__ __forceinline__ void tree_wait(uint32_t bar, uint32_t parity, const ErrWord& err, volatile int* abort) {
  if (mbar_try_many(bar, parity)) return;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_many(bar, parity)) {
    if (*abort) return;
    if (global_ns() - t0 > kWaitNs) {
      *abort = 1;
      atomicExch(err.at, err.code);
      return;
    }
  }
}
// One lane of a converged warp.  MMAs and copies are issued under this
// predicate by warps that run their loops whole: with `if (lane == 0)` instead,
// every tcgen05.mma took ~108 cycles to issue (operands moved to uniform
// registers lane by lane) whatever its size; so it is 30-40.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// Also after an abort: what is in flight lands before the CTA ends.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = global_ns();
  while (!mbar_try(bar, parity))
    if (global_ns() - t0 > kWaitNs) break;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}
// One 128 x N x 16 step: A [128][16] fp16 in tensor memory, B in shared memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// The same with A in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// Instruction descriptor: fp16 A and B, fp32 D, M = 128; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// Shared-memory descriptor: 128-byte swizzle, 1024 bytes between the 8-row
// groups (rows of Q along N, tokens of P along K); one 64-element atom wide.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}

// [rows][16] fp16, K-major without swizzle: 8 x 16-byte core matrices, the two
// along K 128 bytes apart, 256 bytes between 8-row groups.
__device__ __forceinline__ uint64_t narrow_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(256 >> 4) << 32) | ((uint64_t)1 << 46);
}
__host__ __device__ constexpr int narrow_at(int row) { return (row >> 3) * 256 + (row & 7) * 16; }  // elements 0 .. 7

#define KVQ_R4(r, i) "r"((r)[i]), "r"((r)[(i) + 1]), "r"((r)[(i) + 2]), "r"((r)[(i) + 3])
#define KVQ_R16(r, i) KVQ_R4(r, i), KVQ_R4(r, (i) + 4), KVQ_R4(r, (i) + 8), KVQ_R4(r, (i) + 12)
#define KVQ_W4(r, i) "=r"((r)[i]), "=r"((r)[(i) + 1]), "=r"((r)[(i) + 2]), "=r"((r)[(i) + 3])
#define KVQ_W16(r, i) KVQ_W4(r, i), KVQ_W4(r, (i) + 4), KVQ_W4(r, (i) + 8), KVQ_W4(r, (i) + 12)

// 16 rows x 32 columns (64 channels of the Keys of a group).
__device__ __forceinline__ void tc_st_16x256_x4(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::KVQ_R16(r, 0),
      "r"(t)
      : "memory");
}
// 16 rows x 16 columns (16 channels of the Values of two groups).
__device__ __forceinline__ void tc_st_16x128_x4(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::KVQ_R4(r, 0), KVQ_R4(r, 4),
               "r"(t)
               : "memory");
}
template <int N>
__device__ __forceinline__ void tc_ld(uint32_t (&r)[N], uint32_t t) {
  static_assert(N == 8 || N == 16 || N == 32);
  if constexpr (N == 8)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : KVQ_W4(r, 0), KVQ_W4(r, 4)
        : "r"(t)
        : "memory");
  else if constexpr (N == 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : KVQ_W16(r, 0), KVQ_W16(r, 16)
        : "r"(t)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : KVQ_W16(r, 0)
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::KVQ_R4(r, 0), KVQ_R4(r, 4), "r"(t)
               : "memory");
}
// Where a group lies: a stage of the ring (shared memory) or the window's
// tiles (global memory).
struct FromRing {
  uint32_t at;
  __device__ __forceinline__ FromRing operator+(int o) const { return FromRing{at + (uint32_t)o}; }
  __device__ __forceinline__ uint32_t u32() const {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at));
    return x;
  }
  __device__ __forceinline__ uint2 u64() const {
    uint2 x;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at));
    return x;
  }
  __device__ __forceinline__ uint4 u128() const {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
    return x;
  }
};
struct FromGlobal {
  const uint8_t* at;
  __device__ __forceinline__ FromGlobal operator+(int o) const { return FromGlobal{at + o}; }
  __device__ __forceinline__ uint2 u64() const { return *reinterpret_cast<const uint2*>(at); }
  __device__ __forceinline__ uint4 u128() const { return *reinterpret_cast<const uint4*>(at); }
};

// --------------------------------------------------------------- widening

__host__ __device__ constexpr uint32_t splat_h(uint32_t h) { return h | (h << 16); }
// fp16 bits of 2^e (normal)
__host__ __device__ constexpr uint32_t pow2_h(int e) { return (uint32_t)(15 + e) << 10; }
__device__ __forceinline__ uint32_t hadd2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Codes at bits [E, E + BITS) of both half-words -> (c - 2^(BITS-1)) 2^(1-BITS),
// exact: the code lands in the mantissa of 2^X (1 + c 2^(E-10)) with
// X = 11 - E - BITS, i.e. 2^X + c 2^(1-BITS); 2^X + 1 comes off.
template <int BITS, int E>
__device__ __forceinline__ uint32_t code_val(uint32_t w) {
  constexpr int X = 11 - E - BITS;
  static_assert(X >= 0 && X <= 9, "the code lies in the mantissa");
  constexpr uint32_t m = ((1u << BITS) - 1u) << E;
  // -(2^X + 1) in fp16: mantissa bit 10 - X (X = 0: -2)
  constexpr uint32_t off = X == 0 ? 0xc000u : (0x8000u | pow2_h(X) | (1u << (10 - X)));
  return hadd2_u(lop_and_or(w, splat_h(m), splat_h(pow2_h(X))), splat_h(off));
}
// Two 16-bit codes -> fp16((c - 2^15) 2^-15), rounded once.
__device__ __forceinline__ uint32_t code_val16(uint32_t w) {
  const uint32_t hi = lop_and_or(w >> 8, 0x00ff00ffu, splat_h(pow2_h(3)));  // 8 + hi / 128
  const uint32_t lo = lop_and_or(w, 0x00ff00ffu, splat_h(pow2_h(3)));       // 8 + lo / 128
  // hi / 128 - 1 - 2^-5 is exact; (8 + lo / 128) 2^-8 adds 2^-5 + lo 2^-15
  return hfma2_u(lo, splat_h(pow2_h(-8)), hadd2_u(hi, splat_h(0xc884u)));  // - 9.03125
}
// g = (1 - 2^-b) / 2, as fp16 and fp32 (16 bits: 1/2, off by 2^-16)
template <int BITS>
__host__ __device__ constexpr uint32_t value_scale_h() {
  return BITS == 2 ? 0x3600u : BITS == 4 ? 0x3780u : BITS == 8 ? 0x37f8u : 0x3800u;
}
template <int BITS>
__host__ __device__ constexpr float value_scale() {
  return BITS == 16 ? 0.5f : 0.5f - 0.5f / (float)(1 << BITS);
}
__device__ __forceinline__ float value_scale_of(int bits) {
  return bits == 16 ? 0.5f : 0.5f - 0.5f / (float)(1 << bits);
}
__device__ __forceinline__ uint32_t sat_h2(float lo, float hi) {
  return pack_h2(fminf(fmaxf(lo, -65504.f), 65504.f), fminf(fmaxf(hi, -65504.f), 65504.f));
}

// Quad position p (channels 16 p + 4 t .. + 3) of one token: the pairs (members
// 0, 2) and (members 1, 3).  u: the words of the token's half of the lane unit
// from quad position p0 on.
template <int BITS>
__device__ __forceinline__ void key_pairs(const uint32_t* u, int p, uint32_t& a, uint32_t& b) {
  if constexpr (BITS == 16) {
    a = code_val16(__byte_perm(u[2 * p], u[2 * p + 1], 0x5410));
    b = code_val16(__byte_perm(u[2 * p], u[2 * p + 1], 0x7632));
  } else {
    constexpr int qpw = 8 / BITS;
    const uint32_t w = u[p / qpw], w8 = w >> 8;
    switch (p % qpw) {  // a constant after unrolling
      case 0: a = code_val<BITS, 0>(w); b = code_val<BITS, 0>(w8); break;
      case 1: if constexpr (qpw > 1) { a = code_val<BITS, BITS>(w); b = code_val<BITS, BITS>(w8); } break;
      case 2: if constexpr (qpw > 2) { a = code_val<BITS, 2 * BITS>(w); b = code_val<BITS, 2 * BITS>(w8); } break;
      default: if constexpr (qpw > 2) { a = code_val<BITS, 3 * BITS>(w); b = code_val<BITS, 3 * BITS>(w8); } break;
    }
  }
}

// Factors of a token's group from its (R, Z) word at the cache's width: R/4 and
// Z g + R/4, for two tokens or twice for one.
template <int BITS>
__device__ __forceinline__ void group_factors(uint32_t m0, uint32_t m1, uint32_t& rc, uint32_t& zc) {
  rc = hmul2_u(__byte_perm(m0, m1, 0x5410), splat_h(pow2_h(-2)));
  zc = hfma2_u(__byte_perm(m0, m1, 0x7632), splat_h(value_scale_h<BITS>()), rc);
}
// The same for 16-bit codes in a cache of another width: R g / 2 is not exact
// then, so the centre is formed in fp32.
template <int BITS>
__device__ __forceinline__ void window_factors(uint32_t m0, uint32_t m1, uint32_t& rc, uint32_t& zc) {
  constexpr float g = value_scale<BITS>(), f = g * (32768.0f / 65535.0f);
  const uint32_t r2 = __byte_perm(m0, m1, 0x5410), z2 = __byte_perm(m0, m1, 0x7632);
  const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&r2));
  const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&z2));
  rc = pack_h2(r.x * f, r.y * f);
  zc = pack_h2(fmaf(r.x, f, z.x * g), fmaf(r.y, f, z.y * g));
}

// Keys of one group into 16 tensor-memory rows, 64 channels at a time.  part:
// the group's Key part.  CHAN: per-channel groups, their (R, Z) words at kmc (the
// cache's width): values times g; otherwise val, or (SHARE) val times share[x], the
// fp16 pairs of the lane's tokens g and g + 8 (key_terms).
template <int BITS, bool CHAN, bool SHARE, typename From>
__device__ __forceinline__ void widen_keys(From part, FromRing kmc, uint32_t taddr, int lane, const uint32_t* share = nullptr) {
  constexpr int kHalfWords = BITS / 2;  // words of 4 quad positions of one token
  const From unit = part + lane * unit_bytes(BITS);
#pragma unroll
  for (int hf = 0; hf < 2; hf++) {
    uint32_t u[2][kHalfWords], r[16];
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const From at = unit + 4 * (x * BITS + hf * kHalfWords);
      if constexpr (kHalfWords == 1) {
        u[x][0] = at.u32();
      } else if constexpr (kHalfWords == 2) {
        const uint2 w = at.u64();
        u[x][0] = w.x; u[x][1] = w.y;
      } else {
#pragma unroll
        for (int i = 0; i < kHalfWords; i += 4) {
          const uint4 w = (at + 4 * i).u128();
          u[x][i] = w.x; u[x][i + 1] = w.y; u[x][i + 2] = w.z; u[x][i + 3] = w.w;
        }
      }
    }
#pragma unroll
    for (int p = 0; p < 4; p++) {
      uint32_t ra[2], za[2];  // CHAN: of members (0, 2) and (1, 3)
      if constexpr (CHAN) {
        const uint4 w = (kmc + 4 * (16 * (4 * hf + p) + 4 * (lane & 3))).u128();
        group_factors<BITS>(w.x, w.z, ra[0], za[0]);
        group_factors<BITS>(w.y, w.w, ra[1], za[1]);
      }
#pragma unroll
      for (int x = 0; x < 2; x++) {
        uint32_t& k0 = r[4 * p + 2 * x];
        uint32_t& k1 = r[4 * p + 2 * x + 1];
        key_pairs<BITS>(u[x], p, k0, k1);
        if constexpr (CHAN) {
          k0 = hfma2_u(k0, ra[0], za[0]);
          k1 = hfma2_u(k1, ra[1], za[1]);
        }
        if constexpr (SHARE) {
          k0 = hmul2_u(k0, share[x]);
          k1 = hmul2_u(k1, share[x]);
        }
      }
    }
    tc_st_16x256_x4(taddr + 32 * hf, r);
  }
}

// Values of one group and this warp's 32 channels.  The warp takes the channels
// of lane units g = 2 w and 2 w + 1 (h = 0, 1): tensor-memory row 16 h + 8 r +
// g' holds channel 16 g' + 8 r + 2 w + h, so every unit is read by one warp only;
// lane (g', t) turns pairs 2 g', 2 g' + 1 (r = 0, 1) of unit (2 w + h, t).
// out[h][2 u + r]: rows g' + 8 r, column 4 u + t of the group's eight.
// rc, zc: half2 of (R, Z) factors of tokens 2t, 2t + 1 (+ 8 u).
template <int BITS, typename From>
__device__ __forceinline__ void widen_values(From part, const uint32_t (&rc)[2], const uint32_t (&zc)[2], int w, int lane,
                                             uint32_t (&out)[2][4]) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const From unit = part + (4 * (2 * w + h) + t) * unit_bytes(BITS);
#pragma unroll
    for (int u = 0; u < 2; u++) {
      uint32_t v0, v1;
      if constexpr (BITS == 16) {
        const uint2 x = (unit + 4 * (u * 16 + 2 * g)).u64();
        v0 = code_val16(x.x);
        v1 = code_val16(x.y);
      } else {
        constexpr int ppw = 16 / BITS;  // pairs per word
        const uint32_t x = (unit + 4 * (u * BITS + 2 * g / ppw)).u32() >> (2 * BITS * (g % (ppw / 2)));
        v0 = code_val<BITS, 0>(x);
        if constexpr (BITS == 8)
          v1 = code_val<8, 0>(x >> 8);
        else
          v1 = code_val<BITS, BITS>(x);
      }
      out[h][2 * u] = hfma2_u(v0, rc[u], zc[u]);
      out[h][2 * u + 1] = hfma2_u(v1, rc[u], zc[u]);
    }
  }
}
// Channel of tensor-memory row rho of V and O.
__device__ __forceinline__ int channel_of(int rho) {
  return 16 * (rho & 7) + 8 * ((rho >> 3) & 1) + 2 * (rho >> 5) + ((rho >> 4) & 1);
}
// ------------------------------------------------------------------ roles

// Shared address of barrier i of an array in Small, from that of Small (sb).
#define KVQ_BAR(array, i) (sb + (uint32_t)offsetof(Small, array) + 8u * (uint32_t)(i))

// One CTA's walk over its share: segments (a stream's block of rows), tiles.
struct Walk {
  int u, end;               // units left
  int s, block, t0, t1;     // current segment
  __device__ __forceinline__ bool next(const TreePlan& p) {
    if (u >= end) return false;
    const int x = u / p.tiles;
    t0 = u - x * p.tiles;
    t1 = min(p.tiles, t0 + end - u);
    s = x / p.blocks;
    block = x - s * p.blocks;
    u += t1 - t0;
    return true;
  }
};

// Whether token tl (0..127) of tile t exists.
__device__ __forceinline__ bool token_valid(const TreePlan& p, int t, int tl) {
  if (t < p.tp) {
    const int v = t * kTileGroups + (tl >> 4);
    return v < p.groups && (v != p.part_group || (tl & 15) < p.part_valid);
  }
  if (t < p.tp + p.tw) return (t - p.tp) * kTile + tl < p.a.c.n_win;
  return (t - p.tp - p.tw) * kTile + tl < p.a.n;
}

// One buffer's ring: slots buf, buf + 2, ... of the stages, in turn.
struct Slot {
  int i;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Slot(int buf) : i(buf) {}
  __device__ __forceinline__ void step(int stages) {
    i += 2;
    if (i >= stages) {
      i &= 1;
      phase ^= 1;
    }
  }
};

// Producer (one warp): packed progressive tiles into the ring, run by run (groups
// that neighbour in one tile of the cache).
template <int BITS>
__device__ __forceinline__ void produce(const TreePlan& p, Small& sm, uint32_t sb, uint32_t ring, Walk wk) {
  const CacheView& c = p.a.c;
  const Fill& f = p.f;
  using Lay = Layout<BITS>;
  constexpr int gb = group_bytes(BITS);
  const bool chan = c.kmc != nullptr;
  Slot even(0), odd(1);
  uint32_t ct = 0;
  while (wk.next(p)) {
    const uint32_t ct0 = ct;
    ct += wk.t1 - wk.t0;
    if (wk.t0 >= p.tp) continue;
    const uint8_t* sbase = c.codes + (size_t)wk.s * c.nt * kTileBytes;
    const uint32_t* mbase = c.meta + (size_t)wk.s * c.nt * c.pf * 2;
    int tile = 0, grp = 0, groups = 0, e = 0;
    if (!chan) {
      const GroupLoc loc = locate_group(f, (long long)wk.t0 * kTileGroups);
      tile = loc.tile;
      grp = loc.grp;
      groups = loc.tile_groups;
    }
    for (int t = wk.t0; t < min(wk.t1, p.tp); t++) {
      const bool second = (ct0 + (uint32_t)(t - wk.t0)) & 1u;
      const Slot sl = second ? odd : even;
      tree_wait(KVQ_BAR(ring_free, sl.i), sl.phase ^ 1, p.a.err, &sm.abort);
      if (sm.abort) goto out;
      const uint32_t st = ring + (uint32_t)(sl.i * Lay::kStage);
      const uint32_t bar = KVQ_BAR(ring_full, sl.i);
      const int n = min(kTileGroups, p.groups - t * kTileGroups);
      if (elect_one()) {
        mbar_expect_tx(bar, (uint32_t)n * (gb + 128u) + (chan ? 4u * kHeadDim : 0u));
        if (chan)
          bulk_g2s(st + kTileGroups * (gb + 128), c.kmc + ((size_t)wk.s * c.blocks_max + t) * kHeadDim, 4u * kHeadDim, bar);
      }
      __syncwarp();
      for (int g = 0; g < n;) {
        int run;
        if (chan) {  // a block in the order of arrival: whole or partial runs of its epochs
          const int i = t * kTile + g * kGroupTokens;
          while (e + 1 < c.ep.n && i >= c.ep.start[e + 1]) e++;
          const int m = i - c.ep.start[e], lg = c.ep.lg_ee[e], off = m & ((1 << lg) - 1);
          tile = m >> lg;
          grp = (c.ep.h[e] + off) >> 4;
          run = min(n - g, ((1 << lg) - off) >> 4);
        } else {
          run = min(n - g, groups - grp);
        }
        if (elect_one()) {
          bulk_g2s(st + g * gb, sbase + (size_t)tile * kTileBytes + (size_t)(grp * gb), (uint32_t)(run * gb), bar);
          bulk_g2s(st + kTileGroups * gb + g * 128, mbase + ((size_t)tile * c.pf + (size_t)(grp * kGroupTokens)) * 2,
                   (uint32_t)run * 128u, bar);
        }
        __syncwarp();
        g += run;
        if (!chan) {
          grp += run;
          if (grp == groups) {  // the next tile: full, the partial tile k, or half full
            tile++;
            grp = 0;
            groups = tile < f.k ? f.gpt : tile == f.k ? f.gk : f.gh;
          }
        }
      }
      if (second)
        odd.step(Lay::kStages);
      else
        even.step(Lay::kStages);
    }
  }
out:
  if (sm.abort) {  // copies in flight land before the CTA ends: of each slot the last use, if any
    for (int i = 0; i < Lay::kStages; i++) {
      const Slot& r = i & 1 ? odd : even;
      const uint32_t uses_phase = i < r.i ? r.phase : r.phase ^ 1;  // of the slot's last use; the phase before the first reads as done
      drain_wait(KVQ_BAR(ring_full, i), uses_phase);
    }
  }
}

// Group gi (0..7) of window tile t; null if it does not exist.
struct WindowGroup {
  const uint8_t* code;
  const uint32_t* meta;
};
__device__ __forceinline__ WindowGroup window_group(const TreePlan& p, int s, int t, int gi) {
  const int wg = (t - p.tp) * kTileGroups + gi;
  if (wg * kGroupTokens >= p.a.c.n_win) return WindowGroup{nullptr, nullptr};
  constexpr int kPer = slots_per_tile(16) / kGroupTokens;
  const size_t tile = (size_t)s * kWindowTiles + wg / kPer;
  return WindowGroup{p.a.c.wcodes + tile * kTileBytes + (size_t)(wg % kPer) * group_bytes(16),
                     p.a.c.wmeta + (tile * slots_per_tile(16) + kGroupTokens * (wg % kPer)) * 2};
}

// Drafted Keys of a group: a lane's part of tokens g and g + 8 as it is in memory
// (bf16: channels 16 q + 4 t .. + 3 of both halves; fp32: of half hf), so that
// the loads are in flight while something else is done, and into tensor memory
// as k g / lambda.
struct DraftKeys {
  uint4 raw[2][4];
  __device__ __forceinline__ void load(const TreeArgs& a, int b, int h, int j0, int hf, int lane) {
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const int j = j0 + (lane >> 2) + 8 * x;
      const long long at = b * a.k_b + j * a.k_t + h * a.k_h + 4 * (lane & 3);
#pragma unroll
      for (int q = 0; q < 4; q++) {
        raw[x][q] = make_uint4(0u, 0u, 0u, 0u);
        if (j < a.n) {
          if (a.f32) {
            raw[x][q] = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(a.k) + at + 64 * hf + 16 * q));
          } else {
            const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + at + 16 * q;
            const uint2 lo = __ldg(reinterpret_cast<const uint2*>(k)), hi = __ldg(reinterpret_cast<const uint2*>(k + 64));
            raw[x][q] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void store(const TreeArgs& a, int h, int hf, float scale, uint32_t taddr, int lane) const {
    uint32_t r[16];
#pragma unroll
    for (int q = 0; q < 4; q++) {
      float4 l = make_float4(1.f, 1.f, 1.f, 1.f);
      if (a.c.lam_inv)
        l = __ldg(reinterpret_cast<const float4*>(a.c.lam_inv + (size_t)h * kHeadDim + 64 * hf + 16 * q + 4 * (lane & 3)));
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const uint4 w = raw[x][q];
        const uint32_t u0 = hf ? w.z : w.x, u1 = hf ? w.w : w.y;
        const float4 k = a.f32 ? make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w))
                               : make_float4(__uint_as_float(u0 << 16), __uint_as_float(u0 & 0xffff0000u),
                                             __uint_as_float(u1 << 16), __uint_as_float(u1 & 0xffff0000u));
        r[4 * q + 2 * x] = sat_h2(scale * k.x * l.x, scale * k.z * l.z);
        r[4 * q + 2 * x + 1] = sat_h2(scale * k.y * l.y, scale * k.w * l.w);
      }
    }
    tc_st_16x256_x4(taddr + 32 * hf, r);
  }
};
// Drafted Values of a group for this warp's channels (widen_values' layout), times g.
__device__ __forceinline__ void draft_values(const TreePlan& p, int s, int j0, float scale, int w, int lane,
                                             uint32_t (&out)[2][4]) {
  const TreeArgs& a = p.a;
  const int b = s / a.c.kv_heads, h = s - b * a.c.kv_heads;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int u = 0; u < 2; u++) {
#pragma unroll
    for (int r = 0; r < 2; r++) {
      float2 v[2];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int j = j0 + 8 * u + 2 * t + e;
        const long long at = b * a.v_b + j * a.v_t + h * a.v_h + 16 * g + 8 * r + 2 * w;
        v[e] = make_float2(0.f, 0.f);
        if (j < a.n) {
          if (a.f32) {
            v[e] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.v) + at));
          } else {
            const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.v) + at));
            v[e] = make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
          }
        }
      }
      out[0][2 * u + r] = sat_h2(scale * v[0].x, scale * v[1].x);
      out[1][2 * u + r] = sat_h2(scale * v[0].y, scale * v[1].y);
    }
  }
}

// Values of a packed tile in the ring.  CHECK: some of its tokens do not exist
// (n groups do; group part only its first valid tokens): they become zeros, as
// P is zero there and stale codes with a stale range may be anything.
template <int BITS, bool CHECK, int GROUPS>
__device__ __forceinline__ void value_tile(FromRing st, uint32_t ta, int g0, int n, int part, int valid, int w, int lane) {
  constexpr int gb = group_bytes(BITS);
  const int t = lane & 3;
#pragma unroll 2
  for (int g2 = g0; g2 < g0 + GROUPS; g2 += 2) {
    uint32_t o0[8], o1[8];  // rows 0-15 and 16-31, columns 8 g2 .. 8 g2 + 15
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int gi = g2 + i;
      uint32_t rc[2], zc[2], out[2][4];
#pragma unroll
      for (int u = 0; u < 2; u++) {
        uint4 m = (st + (kTileGroups * gb + gi * 128 + 8 * (8 * u + 2 * t))).u128();  // K, V of tokens 2t, 2t + 1 (+ 8u)
        if constexpr (CHECK) {
          const int first = 8 * u + 2 * t, have = gi >= n ? 0 : gi == part ? valid : kGroupTokens;
          if (first >= have) m.y = 0u;
          if (first + 1 >= have) m.w = 0u;
        }
        group_factors<BITS>(m.y, m.w, rc[u], zc[u]);
      }
      widen_values<BITS>(st + (gi * gb + part_bytes(BITS)), rc, zc, w, lane, out);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        o0[4 * i + e] = out[0][e];
        o1[4 * i + e] = out[1][e];
      }
    }
    tc_st_16x128_x4(ta + 8 * g2, o0);
    tc_st_16x128_x4(ta + 8 * g2 + (16u << 16), o1);
  }
}

// Which rows see drafted tokens 32 w .. + 31 of tile t: one word per row.
__device__ __forceinline__ void draft_seen(const TreePlan& p, uint32_t (*seen)[4], int s, int block, int t, int w, int lane) {
  const TreeArgs& a = p.a;
  const int b = s / a.c.kv_heads, j = (t - p.tp - p.tw) * kTile + 32 * w + lane;
  const int r0 = block * p.block_rows, r1 = min(p.rows, r0 + p.block_rows);
  const unsigned char* m = a.mask ? a.mask + b * a.mask_b + j : nullptr;
  constexpr int kBatch = 16;  // mask bytes in flight
  for (int n0 = r0 / a.group; n0 * a.group < r1; n0 += kBatch) {
    bool see[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const int node = n0 + i;
      see[i] = j < a.n && node < a.n;
      if (see[i]) see[i] = m ? m[(long long)node * a.n] != 0 : j <= node;
    }
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      const uint32_t word = __ballot_sync(0xffffffffu, see[i]);
      const int row = (n0 + i) * a.group + lane - r0;
      if (lane < a.group && row >= 0 && row < r1 - r0) seen[row][w] = word;
    }
  }
}

// What a token's score needs beside val: rk for the softmax, a for the extra
// k-step.  A range so small beside its zero that a would leave binary16
// (|Z + rk| > 3999 rk) is taken as |Z + rk| / 3999 by both, and the Key's val counts
// with the share of it that the true range is: rounded once more, by 2^-11 of the
// Key's distance from its group's centre (and by 2^-25 / 3999 of |Z + rk|, below
// what fp32 holds of that).  -> whether the range is such a one.
__device__ __forceinline__ bool key_terms(uint32_t m, float half_codes, float& rk, uint2& centre) {
  const float r = __half2float(__ushort_as_half((unsigned short)(m & 0xffffu))) * half_codes;
  const float mid = __half2float(__ushort_as_half((unsigned short)(m >> 16))) + r;
  rk = fmaxf(r, fabsf(mid) * (1.0f / (kCentreMax - 1.0f)));
  const float a = rk > 0.f ? __fdividef(mid, rk) * kSumScale : 0.f;  // 2 ulp, as fine as the pair
  const float hi = __half2float(__float2half_rn(a));
  centre = make_uint2(pack_h2(hi, hi), pack_h2(a - hi, 0.f));
  return r < rk;
}
// A group's Keys once more, with its tokens' shares.  Few caches have such groups at
// all, so the ordinary way writes every Key first and stays as it is (a choice before
// it took 3-7% of a tree of 14 or 28 rows).  meta: the group's (R, Z) words.
template <int BITS, typename From>
__device__ __forceinline__ void share_keys(From part, From meta, float half_codes, uint32_t taddr, int lane) {
  uint32_t sh[2];
#pragma unroll
  for (int x = 0; x < 2; x++) {
    const uint32_t m = (meta + 8 * (8 * x + (lane >> 2))).u64().x;
    const float r = __half2float(__ushort_as_half((unsigned short)(m & 0xffffu))) * half_codes;
    float rk;
    uint2 centre;
    const float y = key_terms(m, half_codes, rk, centre) ? __fdividef(r, rk) : 1.0f;
    sh[x] = pack_h2(y, y);
  }
  widen_keys<BITS, false, true>(part, FromRing{0}, taddr, lane, sh);
}

// Widening: Keys, then Values of buffer buf's tiles (every second one), and for
// drafted tiles which rows see them.  Warp w of a group writes tensor-memory rows
// 32 w .. + 31: Keys of tokens 32 w .. + 31, Values of the channels of lane units
// 2 w and 2 w + 1; of two groups that share a tile each takes one of the two Key
// groups and half of the Value groups (part).
// KEYS: the cache's Key groups, known here or (kAnyKeys) at run time.
enum { kTokenKeys, kChannelKeys, kAnyKeys };
template <int BITS, int COLS, int KEYS>
__device__ __forceinline__ void widen_role(const TreePlan& p, Small& sm, uint32_t sb, uint32_t ring, Walk wk, int buf, int part,
                                           int w, int lane) {
  using S = Split<COLS>;
  using Lay = Layout<BITS>;
  constexpr int kKeys = 2 / S::kShare, kValues = kTileGroups / S::kShare;
  const int i0 = part * kKeys, v0 = part * kValues;
  const CacheView& c = p.a.c;
  constexpr int gb = group_bytes(BITS);
  constexpr float kHalfCodes = (float)(1u << (BITS - 1)) / (float)((1u << BITS) - 1u), kHalfCodes16 = 32768.0f / 65535.0f;
  const int t4 = lane & 3;
  const uint32_t centre_at = sb - Lay::kSmall + Lay::kCentre + buf * kCentreBytes;
  const uint32_t tk = sm.tmem + ((uint32_t)(32 * w) << 16) + S::kColK + 64 * buf;
  const uint32_t tv = sm.tmem + ((uint32_t)(32 * w) << 16) + S::kColV + 64 * buf;
  uint32_t phase = 1;  // of k_free and v_free
  uint32_t ct = 0;
  Slot sl(buf);
  while (wk.next(p)) {
    for (int t = wk.t0; t < wk.t1; t++, ct++) {
      if ((ct & 1) == (uint32_t)buf) {
        const bool packed = t < p.tp;
        const FromRing st{ring + (uint32_t)(sl.i * Lay::kStage)};
        if (packed) tree_wait(KVQ_BAR(ring_full, sl.i), sl.phase, p.a.err, &sm.abort);
        tree_wait(KVQ_BAR(k_free, buf), phase, p.a.err, &sm.abort);
        tc_after();
        // ---- Keys ----
        const int tl = 32 * w + 16 * i0 + (kKeys == 2 ? lane : lane & 15);  // this lane's token (one group: twice)
        float rk = 0.f;
        uint2 centre = make_uint2(0u, 0u);
        bool small = false;
        if (packed) {
          // groups that do not exist are read as whatever the stage holds: those rows of S are not used
          const uint32_t m = (st + (kTileGroups * gb + 8 * tl)).u32();
          if (KEYS == kChannelKeys || (KEYS == kAnyKeys && c.kmc)) {
#pragma unroll 1
            for (int i = i0; i < i0 + kKeys; i++)
              widen_keys<BITS, true, false>(st + (2 * w + i) * gb, st + kTileGroups * (gb + 128), tk + ((uint32_t)(16 * i) << 16), lane);
            rk = 1.0f / value_scale<BITS>();
          } else {
#pragma unroll 1
            for (int i = i0; i < i0 + kKeys; i++)
              widen_keys<BITS, false, false>(st + (2 * w + i) * gb, st, tk + ((uint32_t)(16 * i) << 16), lane);
            small = key_terms(m, kHalfCodes, rk, centre);
          }
        } else if (t < p.tp + p.tw) {
#pragma unroll 1
          for (int i = i0; i < i0 + kKeys; i++) {
            const WindowGroup wg = window_group(p, wk.s, t, 2 * w + i);
            if (wg.code) widen_keys<16, false, false>(FromGlobal{wg.code}, FromRing{0}, tk + ((uint32_t)(16 * i) << 16), lane);
          }
          const WindowGroup wg = window_group(p, wk.s, t, tl >> 4);
          if (wg.meta) small = key_terms(wg.meta[2 * (tl & 15)], kHalfCodes16, rk, centre);
        } else {
          const int j0 = (t - p.tp - p.tw) * kTile + 32 * w, sb_ = wk.s / c.kv_heads, sh = wk.s - sb_ * c.kv_heads;
          if (c.lam_inv && lane < 4) asm volatile("prefetch.global.L1 [%0];" ::"l"(c.lam_inv + (size_t)sh * kHeadDim + 32 * lane));
          bool told = part != 0;
#pragma unroll 1
          for (int i = i0; i < i0 + kKeys || !told; i++) {
            const bool any = i < i0 + kKeys && j0 + 16 * i < p.a.n;
            const int passes = p.a.f32 ? 2 : 1;
#pragma unroll 1
            for (int ps = 0; ps < passes; ps++) {
              DraftKeys dk;
              if (any) dk.load(p.a, sb_, sh, j0 + 16 * i, ps, lane);
              if (!told) {
                draft_seen(p, sm.seen[ct & 3], wk.s, wk.block, t, w, lane);
                told = true;
              }
              if (any) {
                const uint32_t ti = tk + ((uint32_t)(16 * i) << 16);
                dk.store(p.a, sh, ps, value_scale<BITS>(), ti, lane);
                if (passes == 1) dk.store(p.a, sh, 1, value_scale<BITS>(), ti, lane);
              }
            }
          }
          rk = 1.0f / value_scale<BITS>();
        }
        sm.rk[ct & 3][tl] = rk;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(centre_at + narrow_at(tl)), "r"(centre.x), "r"(centre.y) : "memory");
        if (__builtin_expect(__any_sync(0xffffffffu, small), 0)) {
          tc_wait_st();  // the first writing of these rows
#pragma unroll 1
          for (int i = i0; i < i0 + kKeys; i++) {
            const uint32_t ti = tk + ((uint32_t)(16 * i) << 16);
            if (packed) {
              share_keys<BITS>(st + (2 * w + i) * gb, st + (kTileGroups * gb + 128 * (2 * w + i)), kHalfCodes, ti, lane);
            } else {
              const WindowGroup wg = window_group(p, wk.s, t, 2 * w + i);
              if (wg.code) share_keys<16>(FromGlobal{wg.code}, FromGlobal{reinterpret_cast<const uint8_t*>(wg.meta)}, kHalfCodes16, ti, lane);
            }
          }
        }
        fence_async_smem();
        tc_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(KVQ_BAR(k_full, buf));
        // ---- Values ----
        tree_wait(KVQ_BAR(v_free, buf), phase, p.a.err, &sm.abort);
        tc_after();
        if (packed) {
          const int n = min(kTileGroups, p.groups - t * kTileGroups);
          const int pg = p.part_group - t * kTileGroups;
          if (n == kTileGroups && (unsigned)pg >= (unsigned)kTileGroups)
            value_tile<BITS, false, kValues>(st, tv, v0, n, pg, p.part_valid, w, lane);
          else
            value_tile<BITS, true, kValues>(st, tv, v0, n, pg, p.part_valid, w, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(KVQ_BAR(ring_free, sl.i));
        } else {
#pragma unroll 1
          for (int g2 = v0; g2 < v0 + kValues; g2 += 2) {
            uint32_t o0[8], o1[8];
#pragma unroll
            for (int i = 0; i < 2; i++) {
              uint32_t out[2][4] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
              if (t < p.tp + p.tw) {
                const WindowGroup wg = window_group(p, wk.s, t, g2 + i);
                if (wg.code) {
                  uint32_t rc[2], zc[2];
#pragma unroll
                  for (int u = 0; u < 2; u++) {
                    const uint4 m = *reinterpret_cast<const uint4*>(wg.meta + 2 * (8 * u + 2 * t4));
                    const bool ok0 = token_valid(p, t, 16 * (g2 + i) + 8 * u + 2 * t4);
                    const bool ok1 = token_valid(p, t, 16 * (g2 + i) + 8 * u + 2 * t4 + 1);
                    window_factors<BITS>(ok0 ? m.y : 0u, ok1 ? m.w : 0u, rc[u], zc[u]);
                  }
                  widen_values<16>(FromGlobal{wg.code + part_bytes(16)}, rc, zc, w, lane, out);
                }
              } else {
                const int j0 = (t - p.tp - p.tw) * kTile + 16 * (g2 + i);
                if (j0 < p.a.n) draft_values(p, wk.s, j0, value_scale<BITS>(), w, lane, out);
              }
#pragma unroll
              for (int e = 0; e < 4; e++) {
                o0[4 * i + e] = out[0][e];
                o1[4 * i + e] = out[1][e];
              }
            }
            tc_st_16x128_x4(tv + 8 * g2, o0);
            tc_st_16x128_x4(tv + 8 * g2 + (16u << 16), o1);
          }
        }
        tc_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(KVQ_BAR(v_full, buf));
        phase ^= 1;
        if (packed) sl.step(Lay::kStages);
      }
    }
  }
}

// One warp per half: the MMAs of the half's tiles.  at: shared address of the CTA's data.
template <int BITS, int COLS, bool DUAL>
__device__ __forceinline__ void mma_role(const TreePlan& p, Small& sm, uint32_t sb, uint32_t at, Walk wk, int half) {
  using S = Split<COLS>;
  constexpr uint32_t kDescQk = mma_desc(COLS, false), kDescPv = mma_desc(COLS, true);
  const uint32_t ts = sm.tmem + S::kColS + S::kStep * half, to = sm.tmem + S::kColO + S::kStep * half;
  const uint32_t tk = sm.tmem + S::kColK, tv = sm.tmem + S::kColV;
  using Lay = Layout<BITS>;
  const uint64_t q_desc = smem_desc(at + half * kQBytes);
  const uint64_t p_desc = smem_desc(at + Lay::kP + half * kPBytes);
  const uint64_t centre_desc = narrow_desc(at + Lay::kCentre), sum_desc = narrow_desc(at + Lay::kSum + half * kSumBytes);
  // The two products of a tile are issued each as soon as it is ready: the next
  // tile's scores first where the Keys are early, the output first where they are
  // late (it frees the Values' buffer).
  struct Cursor {
    Walk wk;
    int t = 0;
    uint32_t ct = 0, n = 0, segs = 0;  // before this tile: tiles of the CTA, of the half; segments with tiles of the half, this one included
    bool started = false, fresh = false, first = false, live = false;  // first: of the half in its segment
    __device__ __forceinline__ explicit Cursor(const Walk& w) : wk(w) { wk.t0 = wk.t1 = 0; }
    __device__ __forceinline__ void next(const TreePlan& p, int half) {
      if (started) {
        t++;
        ct++;
        n++;
      }
      first = false;
      while (true) {
        if (!DUAL && t < wk.t1 && (ct & 1) != (uint32_t)half) {
          t++;
          ct++;
        }
        if (t < wk.t1) break;
        if (!wk.next(p)) {
          live = false;
          return;
        }
        t = wk.t0;
        fresh = true;
      }
      if (fresh) {
        fresh = false;
        first = true;
        segs++;
      }
      started = live = true;
    }
  };
  Cursor q(wk), v(wk);
  q.next(p, half);
  v.next(p, half);
  unsigned idle = 0;
  unsigned long long t0 = 0;
  while (v.live) {
    bool did = false;
    if (q.live) {
      const int buf = q.ct & 1;
      if (mbar_test(KVQ_BAR(k_full, buf), (q.ct >> 1) & 1) && mbar_test(KVQ_BAR(s_free, half), (q.n & 1) ^ 1) &&
          (!q.first || mbar_test(KVQ_BAR(q_full, half), (q.segs - 1) & 1))) {
        tc_after();
        if (elect_one()) {
          tc_mma_ss(ts, centre_desc + (kCentreBytes >> 4) * buf, sum_desc, kDescQk, false);  // a sum(q')
#pragma unroll
          for (int k = 0; k < 8; k++)
            tc_mma(ts, tk + 64 * buf + 8 * k, q_desc + (((k >> 2) * (kQBytes / 2) + 32 * (k & 3)) >> 4), kDescQk, true);
          tc_commit(KVQ_BAR(k_free, buf));
          tc_commit(KVQ_BAR(s_full, half));
        }
        __syncwarp();
        q.next(p, half);
        did = true;
      }
    }
    if (!q.live || v.n < q.n) {  // its scores are issued
      const int buf = v.ct & 1;
      if (mbar_test(KVQ_BAR(p_full, half), v.n & 1) && mbar_test(KVQ_BAR(v_full, buf), (v.ct >> 1) & 1)) {
        tc_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; k++)
            tc_mma(to, tv + 64 * buf + 8 * k, p_desc + (2048 >> 4) * k, kDescPv, !(v.first && k == 0));
          tc_commit(KVQ_BAR(v_free, buf));
          tc_commit(KVQ_BAR(pv_done, half));
        }
        __syncwarp();
        v.next(p, half);
        did = true;
      }
    }
    if (did) {
      idle = 0;
      t0 = 0;
    } else if ((++idle & 255u) == 0u) {  // bounded like every wait
      if (sm.abort) break;
      const unsigned long long now = global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitNs) {
        sm.abort = 1;
        atomicExch(p.a.err.at, p.a.err.code);
        break;
      }
    }
  }
  if (elect_one()) tc_commit(KVQ_BAR(drain, half));
  __syncwarp();
  drain_wait(KVQ_BAR(drain, half), 0);
}

// Sum or maximum over the warp's lanes of N values a lane: every exchange halves
// the values a lane carries.  Lane L ends, in v[0], with column L N / 32 (N <= 32).
template <int N, bool MAX>
__device__ __forceinline__ void warp_columns(float (&v)[N], int lane) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int o = 16, len = N; o; o >>= 1) {
    if (len > 1) {
      len /= 2;
#pragma unroll
      for (int i = 0; i < N / 2; i++) {
        if (i < len) {
          const float keep = (lane & o) ? v[i + len] : v[i], send = (lane & o) ? v[i] : v[i + len];
          v[i] = join(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
      }
    } else {
      v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
}

// A warpgroup: softmax of C of the half's columns (from column cb on) in the
// half's tiles, and the segment's results for them.
template <int BITS, int COLS, bool DUAL>
__device__ __forceinline__ void softmax_role(const TreePlan& p, Small& sm, uint32_t sb, uint8_t* base, Walk wk, int wg, int tl) {
  using S = Split<COLS>;
  constexpr int C = S::kCols;
  static_assert(C == 16 || C == 32);
  constexpr int kSoftThreads = 32 * S::kSoft;
  const TreeArgs& a = p.a;
  const int half = wg / S::kSubs, cb = (wg % S::kSubs) * C;
  const int w = tl >> 5, lane = tl & 31;
  const uint32_t lanes = (uint32_t)(32 * w) << 16;
  const uint32_t ts = sm.tmem + S::kColS + S::kStep * half + cb + lanes, to = sm.tmem + S::kColO + S::kStep * half + cb + lanes;
  uint8_t* q_smem = base + half * kQBytes;
  using Lay = Layout<BITS>;
  uint8_t* p_all = base + Lay::kP;
  uint8_t* p_smem = p_all + half * kPBytes;
  uint8_t* sum_smem = base + Lay::kSum + half * kSumBytes;
  // the product of this half's tile i is in
  auto wait_pv = [&](uint32_t i) { tree_wait(KVQ_BAR(pv_done, half), i & 1, p.a.err, &sm.abort); };
  const int id = 1 + wg;  // barriers 1 .. 4: one warpgroup; 5: every softmax thread; 6, 7: one half
  uint32_t ct = 0, n = 0;
  constexpr float out_scale = 1.0f / value_scale<BITS>();
  while (wk.next(p)) {
    const int b = wk.s / a.c.kv_heads, j = wk.s - b * a.c.kv_heads;
    const int r0 = wk.block * p.block_rows + (DUAL ? half * kHalfRows : 0) + cb;  // first row of these columns
    const int nr = min(C, min(p.rows, (wk.block + 1) * p.block_rows) - r0);       // rows that exist (may be <= 0)
    // tiles of this half in the segment
    const int mine = DUAL ? wk.t1 - wk.t0 : (wk.t1 - wk.t0 + ((ct & 1) == (uint32_t)half ? 1 : 0)) >> 1;
    float2 l2[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; i++) l2[i] = make_float2(0.f, 0.f);
    if (mine > 0) {
      // ---- q' = q lambda sm_scale log2(e) as fp16, K-major, channels of a quad in the order 0, 2, 1, 3 ----
      // (Few instructions matter here more than anything: they run once a segment,
      // from cold instruction memory.)
      float4 lam = make_float4(1.f, 1.f, 1.f, 1.f);
      if (a.c.lam) lam = __ldg(reinterpret_cast<const float4*>(a.c.lam + (size_t)j * kHeadDim) + lane);
      const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + b * a.q_b + (long long)(j * a.group) * a.q_h + 4 * lane;
      int node = (r0 + w) / a.group, g = r0 + w - node * a.group;
      uint2 raw[C / 4];
#pragma unroll
      for (int i = 0; i < C / 4; i++) {  // rows w, w + 4, ...
        raw[i] = make_uint2(0u, 0u);
        if (w + 4 * i < nr) raw[i] = *reinterpret_cast<const uint2*>(qp + node * a.q_t + g * a.q_h);
        g += 4;
        while (g >= a.group) {
          g -= a.group;
          node++;
        }
      }
      lam.x *= a.qscale; lam.y *= a.qscale; lam.z *= a.qscale; lam.w *= a.qscale;
      uint8_t* qs = q_smem + (lane >> 4) * (kQBytes / 2) + 8 * (lane & 1);
      float sum[C / 4];  // of the rounded q', as the products see it
#pragma unroll
      for (int i = 0; i < C / 4; i++) {
        const int rs = cb + w + 4 * i;  // row of the half's Q
        const float q0 = __uint_as_float(raw[i].x << 16) * lam.x, q2 = __uint_as_float(raw[i].y << 16) * lam.z;
        const float q1 = __uint_as_float(raw[i].x & 0xffff0000u) * lam.y, q3 = __uint_as_float(raw[i].y & 0xffff0000u) * lam.w;
        const uint32_t h02 = sat_h2(q0, q2), h13 = sat_h2(q1, q3);
        const float2 f02 = __half22float2(*reinterpret_cast<const __half2*>(&h02));
        const float2 f13 = __half22float2(*reinterpret_cast<const __half2*>(&h13));
        // sat_h2 makes numbers of NaN and infinities; the row's sum, and so its scores, become NaN instead
        sum[i] = fmaf(0.f, (q0 + q2) + (q1 + q3), (f02.x + f02.y) + (f13.x + f13.y));
        *reinterpret_cast<uint2*>(qs + rs * 128 + ((((lane & 15) >> 1) ^ (rs & 7)) << 4)) = make_uint2(h02, h13);
      }
      warp_columns<C / 4, false>(sum, lane);
      constexpr int kSumLanes = 128 / C;  // lanes that end with the same row
      if (lane % kSumLanes == 0) {
        const int rs = cb + w + 4 * (lane / kSumLanes);
        const float sc = isnan(sum[0]) ? sum[0] : fminf(fmaxf(sum[0] * (1.0f / kSumScale), -65504.f), 65504.f);
        const float hi = __half2float(__float2half_rn(sc));
        *reinterpret_cast<uint4*>(sum_smem + narrow_at(rs)) = make_uint4(pack_h2(hi, sc - hi), pack_h2(hi, 0.f), 0u, 0u);
        *reinterpret_cast<uint4*>(sum_smem + narrow_at(rs) + 128) = make_uint4(0u, 0u, 0u, 0u);
        sm.neg[half][rs] = __uint_as_float(kUnsetBits);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(KVQ_BAR(q_full, half));
      bar_sync(id, 128);  // neg
    }
    int done = 0;
    for (int t = wk.t0; t < wk.t1; t++, ct++) {
      if (!DUAL && (ct & 1) != (uint32_t)half) continue;
      // which columns' rows do not see this thread's token
      uint32_t hide = 0u;
      if (t >= p.tp || t * kTileGroups + kTileGroups > p.groups || (unsigned)(p.part_group - t * kTileGroups) < (unsigned)kTileGroups)
        hide = token_valid(p, t, tl) ? 0u : 0xffffffffu;
      tree_wait(KVQ_BAR(s_full, half), n & 1, a.err, &sm.abort);
      tc_after();
      if (t >= p.tp + p.tw && hide == 0u) {
        const uint32_t(*seen)[4] = sm.seen[ct & 3] + (DUAL ? half * kHalfRows : 0) + cb;
#pragma unroll
        for (int i = 0; i < C; i++) hide |= (seen[i][w] >> lane & 1u) ? 0u : 1u << i;
      }
      const float rk = sm.rk[ct & 3][tl];
      float2 x[C / 2];
      {  // scores less the running maxima (of a row that has none: as they are)
        uint32_t d[C];
        tc_ld(d, ts);
        tc_before();  // S is in registers: the next tile's product may start
        __syncwarp();
        if (lane == 0) mbar_arrive(KVQ_BAR(s_free, half));
#pragma unroll
        for (int i = 0; i < C; i += 4) {
          const float4 neg = *reinterpret_cast<const float4*>(&sm.neg[half][cb + i]);
          x[i / 2] = fma2(splat2(rk), make_float2(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), make_float2(neg.x, neg.y));
          x[i / 2 + 1] = fma2(splat2(rk), make_float2(__uint_as_float(d[i + 2]), __uint_as_float(d[i + 3])), make_float2(neg.z, neg.w));
        }
      }
      if (hide) {
#pragma unroll
        for (int i = 0; i < C / 2; i++) {
          if (hide >> (2 * i) & 1u) x[i].x = -INFINITY;
          if (hide >> (2 * i + 1) & 1u) x[i].y = -INFINITY;
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < C / 2; i++) mx[i & 3] = fmaxf(mx[i & 3], fmaxf(x[i].x, x[i].y));
      // Every row sees some token of a cached tile, so only the first tile and the
      // drafted ones meet rows without a maximum.
      const bool some_unset = done == 0 || t >= p.tp + p.tw;
      if (bar_or(id, 128, some_unset || fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) > kRebase)) {
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += 8) {  // column maxima, of the scores themselves; eight columns are what registers hold
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 neg = *reinterpret_cast<const float2*>(&sm.neg[half][cb + c0 + i]);
            v[i] = x[(c0 + i) / 2].x - neg.x;
            v[i + 1] = x[(c0 + i) / 2].y - neg.y;
          }
          warp_columns<8, true>(v, lane);
          if ((lane & 3) == 0) sm.red[half][w][cb + c0 + (lane >> 2)] = v[0];
        }
        bar_sync(id, 128);
        if (tl < C) {
          const int c = cb + tl;
          const float old = sm.neg[half][c];
          float m = fmaxf(fmaxf(sm.red[half][0][c], sm.red[half][1][c]), fmaxf(sm.red[half][2][c], sm.red[half][3][c]));
          float f = 0.f, shift = 0.f;
          if (!unset(old)) {
            m = fmaxf(m, -old);
            f = ex2(-old - m);
          }
          if (m > -INFINITY) {  // a row that has seen nothing stays unset
            const float neg = 0.f - m;
            shift = neg - old;
            sm.neg[half][c] = neg;
          }
          sm.alpha[half][c] = f;
          sm.shift[half][c] = shift;
        }
        bar_sync(id, 128);
        if (done > 0) {  // O so far, once the last product is in; eight columns at a time (sixteen spilled: 209 -> 207 us)
          const float2* al = reinterpret_cast<const float2*>(sm.alpha[half] + cb);
          wait_pv(n - 1);
          tc_after();
#pragma unroll 1
          for (int c0 = 0; c0 < C; c0 += 8) {
            uint32_t o[8];
            tc_ld(o, to + c0);
#pragma unroll
            for (int i = 0; i < 8; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * sm.alpha[half][cb + c0 + i]);
            tc_st(to + c0, o);
          }
#pragma unroll
          for (int i = 0; i < C / 2; i++) l2[i] = mul2(l2[i], al[i]);
          tc_wait_st();
        }
        const float2* sh = reinterpret_cast<const float2*>(sm.shift[half] + cb);
#pragma unroll
        for (int i = 0; i < C / 2; i++) x[i] = add2(x[i], sh[i]);
      }
      if (done > 0) wait_pv(n - 1);  // P is free again
      uint8_t* p_at = p_smem + tl * 128;
#pragma unroll
      for (int q = 0; q < C / 8; q++) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int i = 4 * q + e;
          const float2 pr = make_float2(ex2(x[i].x), ex2(x[i].y));
          l2[i] = add2(l2[i], pr);
          h[e] = pack_h2(pr.x, pr.y);
        }
        *reinterpret_cast<uint4*>(p_at + (((cb / 8 + q) ^ (tl & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_async_smem();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(KVQ_BAR(p_full, half));
      n++;
      done++;
    }
    // ---- the segment's results ----
    {
      float v[C];
#pragma unroll
      for (int i = 0; i < C / 2; i++) { v[2 * i] = l2[i].x; v[2 * i + 1] = l2[i].y; }
      warp_columns<C, false>(v, lane);
      sm.red[half][w][cb + (C == 32 ? lane : lane >> 1)] = v[0];
    }
    bar_sync(id, 128);
    if (tl < C) {
      const float* r = &sm.red[half][0][cb + tl];
      const float l = (r[0] + r[kHalfRows]) + (r[2 * kHalfRows] + r[3 * kHalfRows]);
      const float neg = sm.neg[half][cb + tl];
      const bool any = mine > 0 && (!unset(neg) || isnan(l));  // a row of NaN has no maximum
      sm.ml[half][cb + tl] = make_float2(any ? -neg : -INFINITY, any ? l : 0.f);
    }
    if (mine > 0) {
      wait_pv(n - 1);
      tc_after();
    }
    const bool whole = wk.t0 == 0 && wk.t1 == p.tiles;
    // this CTA's records: 0 for the segment its share begins in, else 1
    const int xi = wk.s * p.blocks + wk.block, begin = cta_begin(p, blockIdx.x);
    float* rec = p.parts + ((size_t)blockIdx.x * 2 + (xi * p.tiles + wk.t0 == begin ? 0 : 1)) * p.rec;
    const int rr = (DUAL ? half * kHalfRows : 0) + cb;  // first row within the block
    // C rows of bf16 leave from shared memory, 16 bytes a thread
    auto flush = [&](const uint8_t* sh) {
      for (int i = tl; i < C * 16; i += 128) {
        const int r = i >> 4, q = i & 15;
        if (r < nr) {
          const int row = r0 + r, node = row / a.group, g = row - node * a.group;
          reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                   (((long long)b * a.n + node) * a.q_heads + j * a.group + g) * kHeadDim)[q] =
              *reinterpret_cast<const uint4*>(sh + r * 256 + 16 * q);
        }
      }
    };
    const int ch = channel_of(tl);
    if constexpr (DUAL) {
      bar_sync(id, 128);  // ml
      uint32_t o[C];
      tc_ld(o, to);
      tc_before();
      if (whole) {
        uint8_t* sh = p_smem + (wg % S::kSubs) * (C * 256);
#pragma unroll
        for (int i = 0; i < C; i++) {
          const float l = sm.ml[half][cb + i].y;
          reinterpret_cast<__nv_bfloat16*>(sh)[i * kHeadDim + ch] =
              __float2bfloat16_rn(l != 0.f ? __uint_as_float(o[i]) * out_scale / l : 0.f);
        }
        bar_sync(id, 128);
        flush(sh);
        bar_sync(6 + half, kSoftThreads / 2);  // P is written again
      } else {
#pragma unroll
        for (int i = 0; i < C; i++)
          if (i < nr) rec[2 * p.block_rows + (rr + i) * kHeadDim + tl] = __uint_as_float(o[i]);
        if (tl < nr) {
          rec[rr + tl] = sm.ml[half][cb + tl].x;
          rec[p.block_rows + rr + tl] = sm.ml[half][cb + tl].y;
        }
      }
    } else {
      // join the halves: half 1 hands its O over in shared memory (both P areas: [COLS][128] fp32)
      bar_sync(5, kSoftThreads);  // ml of both; every product of both halves is in
      float* other_o = reinterpret_cast<float*>(p_all) + cb * kTile;
      if (half == 1 && mine > 0) {
        uint32_t o[C];
        tc_ld(o, to);
#pragma unroll
        for (int i = 0; i < C; i++) other_o[i * kTile + tl] = __uint_as_float(o[i]);
      }
      tc_before();
      bar_sync(5, kSoftThreads);
      if (half == 0) {
        const int other = wk.t1 - wk.t0 - mine;
        uint32_t o[C];
        if (mine > 0) {
          tc_ld(o, to);
          tc_before();
        }
#pragma unroll
        for (int i = 0; i < C; i++) {
          const float2 m0 = sm.ml[0][cb + i], m1 = sm.ml[1][cb + i];
          const float m = fmaxf(m0.x, m1.x);
          const float f0 = m0.y != 0.f ? ex2(m0.x - m) : 0.f, f1 = m1.y != 0.f ? ex2(m1.x - m) : 0.f;
          float v = mine > 0 ? __uint_as_float(o[i]) * f0 : 0.f;
          if (other > 0) v = fmaf(other_o[i * kTile + tl], f1, v);
          const float l = m0.y * f0 + m1.y * f1;
          if (whole) {
            o[i] = __float_as_uint(l != 0.f ? v * out_scale / l : 0.f);
          } else if (i < nr) {
            rec[2 * p.block_rows + (rr + i) * kHeadDim + tl] = v;
            if (tl == i) {
              rec[rr + i] = m;
              rec[p.block_rows + rr + i] = l;
            }
          }
        }
        if (whole) {
          bar_sync(id, 128);  // other_o is read
          uint8_t* sh = reinterpret_cast<uint8_t*>(other_o);
#pragma unroll
          for (int i = 0; i < C; i++)
            reinterpret_cast<__nv_bfloat16*>(sh)[i * kHeadDim + ch] = __float2bfloat16_rn(__uint_as_float(o[i]));
          bar_sync(id, 128);
          flush(sh);
        }
      }
      bar_sync(5, kSoftThreads);  // P and ml are written again
    }
  }
}

template <int REGS>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

template <int BITS, int COLS, bool DUAL>
__global__ void __launch_bounds__(Split<COLS>::kThreads, 1) tree_kernel(const __grid_constant__ TreePlan p) {
  using S = Split<COLS>;
  using Lay = Layout<BITS>;
  constexpr int kWiden0 = S::kSoft, kCtl0 = kWiden0 + S::kWiden;
  extern __shared__ uint8_t raw[];
  const uint32_t raw_at = smem_u32(raw), smem_at = (raw_at + 1023u) & ~1023u;
  const uint32_t sb = smem_at + Lay::kSmall, ring_at = smem_at + Lay::kRing;
  uint8_t* base = raw + (smem_at - raw_at);
  Small& sm = *reinterpret_cast<Small*>(base + Lay::kSmall);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (warp == kCtl0 + 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int i = 0; i < kMaxStages; i++) {
      mbar_init(KVQ_BAR(ring_full, i), 1);
      mbar_init(KVQ_BAR(ring_free, i), 4 * S::kShare);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(KVQ_BAR(k_full, i), 4 * S::kShare);
      mbar_init(KVQ_BAR(k_free, i), DUAL ? 2 : 1);
      mbar_init(KVQ_BAR(v_full, i), 4 * S::kShare);
      mbar_init(KVQ_BAR(v_free, i), DUAL ? 2 : 1);
      mbar_init(KVQ_BAR(q_full, i), S::kSoft / 2);
      mbar_init(KVQ_BAR(s_full, i), 1);
      mbar_init(KVQ_BAR(s_free, i), S::kSoft / 2);
      mbar_init(KVQ_BAR(p_full, i), S::kSoft / 2);
      mbar_init(KVQ_BAR(pv_done, i), 1);
      mbar_init(KVQ_BAR(drain, i), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < 2 * kTile) {  // the widening warps write the first 8 bytes of a token's row
    uint8_t* centre = base + Lay::kCentre + (threadIdx.x / kTile) * kCentreBytes + narrow_at(threadIdx.x % kTile);
    *reinterpret_cast<uint4*>(centre) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(centre + 128) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
  }
  tc_before();
  __syncthreads();
  tc_after();
  pdl_wait();  // the cache, q, k, v and the mask may be written by earlier kernels
  const Walk wk{cta_begin(p, blockIdx.x), cta_begin(p, blockIdx.x + 1), 0, 0, 0, 0};
  if (warp < kWiden0) {
    regs_up<S::kSoftRegs>();
    softmax_role<BITS, COLS, DUAL>(p, sm, sb, base, wk, warp >> 2, threadIdx.x & 127);
  } else if (warp < kCtl0) {
    if constexpr (S::kWidenRegs > S::kRegs) regs_up<S::kWidenRegs>();
    if constexpr (S::kWidenRegs < S::kRegs) regs_down<S::kWidenRegs>();
    const int group = (warp - kWiden0) >> 2, buf = group & 1, part = group >> 1, w = warp & 3;
    // One loop for both kinds of Key groups, or one each: 28 rows over 4 bits and
    // per-channel groups 237 us and 213, 63 x 8 rows over 8 bits 491 and 503.
    if constexpr (COLS == 64)
      widen_role<BITS, COLS, kAnyKeys>(p, sm, sb, ring_at, wk, buf, part, w, lane);
    else if (p.a.c.kmc)
      widen_role<BITS, COLS, kChannelKeys>(p, sm, sb, ring_at, wk, buf, part, w, lane);
    else
      widen_role<BITS, COLS, kTokenKeys>(p, sm, sb, ring_at, wk, buf, part, w, lane);
  } else {
    regs_down<S::kCtlRegs>();
    if (warp == kCtl0)
      produce<BITS>(p, sm, sb, ring_at, wk);
    else if (warp < kCtl0 + 3)
      mma_role<BITS, COLS, DUAL>(p, sm, sb, smem_at, wk, warp - kCtl0 - 1);
    __syncwarp();
  }
  tc_before();
  __syncthreads();
  pdl_launch_dependents();
  tc_after();
  if (warp == kCtl0 + 3) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sm.tmem) : "memory");
}

template <int BITS, int COLS, bool DUAL>
cudaError_t launch_cols(const TreePlan& p, cudaStream_t s) {
  static DeviceOnce once;
  if (cudaError_t e = once([] {
        return cudaFuncSetAttribute(tree_kernel<BITS, COLS, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<BITS>::kBytes);
      }))
    return e;
  return launch_pdl(tree_kernel<BITS, COLS, DUAL>, dim3(p.grid), dim3(Split<COLS>::kThreads), Layout<BITS>::kBytes, s, p);
}

}  // namespace

template <int BITS>
cudaError_t launch_tree_bits(const TreePlan& p, cudaStream_t s) {
  switch (p.block_rows) {
    case 16: return launch_cols<BITS, 16, false>(p, s);
    case 32: return launch_cols<BITS, 32, false>(p, s);
    case 64: return launch_cols<BITS, 64, false>(p, s);
    default: return launch_cols<BITS, 64, true>(p, s);
  }
}

}  // namespace kvq
