// Losses over the vocabulary with their gradients (pg_vocab_ce, pg_vocab_distill and their _grad calls).
//
// With z = scale h W^T (h [N, d], W [V, d]; for the distillation scale / T in scale's place), p = softmax(z) and
// targets w_ij (cross entropy: 1 at t_i; distillation: the teacher's softmax over its list),
//   lse_i = log sum_j exp z_ij        loss_i = sum_j w_ij log w_ij - sum_j w_ij z_ij + lse_i (+ zl lse_i^2)
//   dz_ij = g_i (beta_i p_ij - w_ij)  beta_i = 1 + 2 zl lse_i,  g_i = grad_scale row_weight_i
//   dh = scale dz W,  dW = scale dz^T h
// Three products of 2 N V d operations; the first alone without gradients.
//
// The logits exist only tile by tile in TMEM. A row has a reference c_i <= lse_i that the epilogue of the first
// product knows beforehand: the logit of its target, or of the heaviest token of its list, a dot product of its own
// (vocab_prepare_kernel). The epilogue stores u_ij = exp(z_ij - c_i), adds up each tile's rows and keeps the listed
// tokens' logits. One small kernel a chunk (vocab_rows_kernel) then has lse_i, the loss and
// f_i = g_i scale beta_i exp(c_i - lse_i), puts
//   u_ij - w_ij exp(lse_i - c_i) / beta_i
// at the targets (from fp32 logits; cross entropy keeps its sums without the target's term, so that 1 - p and a small loss are the
// others' sum and no difference of numbers near 1), and
//   dh_i = f_i (U W)_i,   dW = U^T (f h)
// are two more products. So the logits are made once, nothing normalises U, and a gradient costs 6 N V d
// operations; making the logits again in place of keeping U would cost 8. U is kept in bf16, whose exponent takes
// exp(+-87); u's rounding (2^-8 at most) is a rounding of p, and that of f h another of dW's. It is kept for a chunk of
// the rows, 2 GiB or 256 rows where those take more. A tile's row whose sum passes 2^57 (logits 40 above the targets') takes the row's largest logit
// of that tile as its reference instead, and vocab_rows_kernel brings the whole row to the largest of its references: a pass over
// the rows that need it and no others. (Only where a row's weight is next to nothing is lse the reference.)
//
// Precision. bf16 operands and bf16 gradients take one product of bf16 operands each. fp32 values are sums of bf16
// "pieces" (value = p0 + p1 + p2, 8 bits each), and their products the sum of the pieces' products down to 2^-24 (six of
// nine): fp32 operands are split beforehand, and U and f h have three pieces for an fp32 gradient. (An fp32 dW of bf16
// operands has f in U, which takes the logits a second time, and h as it is.) All sums are fp32 in TMEM, and long ones that an
// fp32 result comes of are made in groups.
//
// The products: 256 x 256 tiles on CTA pairs (tcgen05, cta_group::2), 128-deep k-blocks of both operands by
// TMA into a ring of three, two accumulators in TMEM, eight epilogue warps. Up to 128 rows, where reading W is all that
// counts, the first product and dh have kernels of their own in which W's rows and columns are the tile's rows; up to 8
// rows of an fp32 W, kernels of fp32 FMAs.
//
// Bound by the tensor cores, and in long calls by the power limit (the measured bf16 rate: 1914 TFLOP/s for a short
// product, 1721 for seconds of them). 16,384 x 50,304 x 768: 762-779 us, 1.63-1.66 PFLOP/s. With gradients, 65,536 x 50,304 x 768:
// 10.1-10.5 ms, 1.45-1.50; 8192 x 128,000 x 2560: 10.1-10.6 ms, 1.52-1.60. Of 2.33 ms a chunk of 16,384 rows by 768 (at full
// clocks) the first product is 0.77 (0.62 without U: its stores go through L2 beside 16 TB/s of operand loads), the other two 1.41.
#include <cuda_bf16.h>

#include <limits.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "pg_conv_math.cuh"
#include "pg_umma.cuh"
#include "pg_vec.h"

namespace pg {
namespace {

constexpr int kErrVocab = 524288;        // device error bit: a wait of these products gave up
constexpr int kMaxVocabWidth = 16384;    // d
constexpr int64_t kMaxVocab = (1 << 24) - 1;
constexpr int kMaxList = 256;            // teacher tokens a row
constexpr int kAtOnce = 1024;            // segments whose beginnings a block collects
constexpr int kPlanUnits = 76;           // CTA pairs that the plan counts on (any number gives the same results)
constexpr int64_t kKeepBytes = 2ll << 30;  // of U, f h, the pieces of h and the lists
constexpr int64_t kSumBytes = 256 << 20;   // of the tiles' sums
constexpr int kMaxParts = 32;              // of a gradient, and
constexpr int kPartTiles = 640;            // tiles that they come to, at most
constexpr int kMaxForwardRows = 16384;   // h of that many rows stays in L2 while W passes by

constexpr int kPrepThreads = 256;
constexpr int kFewTable = 1024;           // above it dh of few rows is made by itself
constexpr int kSmallRows = 8;             // up to here an fp32 W takes FMAs in place of products of pieces
constexpr int kSmallThreads = 256;
constexpr int kFewRows = 128;             // up to here the first product has W's rows for its tiles' rows
constexpr int kTile = 256;
constexpr int kThreads = 384;            // warps 0 and 1 issue copies and products, 4 to 11 are the epilogue's
constexpr int kEpiFirst = 4;
constexpr int kEpiWarps = 8;
constexpr int kStages = 3;
constexpr int kOperandBytes = 128 * kBK * 2;
constexpr int kStageBytes = 4096;        // an epilogue warp's: 32 rows of 128 bytes, or two buffers of 32 rows of 64
constexpr size_t kRing = static_cast<size_t>(kStages) * 2 * kOperandBytes;
constexpr size_t kSmem = 1024 + kRing + kEpiWarps * kStageBytes;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) |  // kind::f16: fp32 sums, bf16 operands
                            (static_cast<uint32_t>(kTile >> 4) << 24);  // M; N and the layouts go with the job

// A tensor core cuts what falls below its sum where an fp32 addition rounds, so a sum's error grows with its length, to
// one side: 1.4e-6 of the logits at d = 2560, 4e-6 with the six products of fp32 operands. Where an fp32 result comes
// of it, sums longer than kGroup k-blocks are made in groups, which the epilogue adds up in registers. Products of pieces
// run from the smallest to the largest, k-block by k-block, and of the largest every few instructions (of 16 k) make a sum of
// their own, so that next to nothing is cut. With 2, 4 and 8 of them everywhere: 512 x 1024 x 96 in fp32 42, 39 and 38.5 us, its
// gradients 1.3e-7, 1.7e-7 and 2.7e-7 off; 3001 x 32,003 x 515 with an fp32 dW 876, 787 and 745 us. The logits' errors count most,
// as exp makes them relative ones: 2 for them and where the six products of a gradient hide it, 4 where there are three (821 us).
// What is cut leans to one side in every row, so a table's gradient over many rows gathers it: fp32 dW of bf16 operands, 11,708
// x 604 x 1200, is 3.3e-7 off with logits in sums of ten k-blocks, 1.5e-7 of two and 1.4e-7 of one (8192 x 50,304 x 768 3.11, 3.38
// and 3.58 ms).
constexpr int kGroup = 10;               // bf16 operands and gradients (80 additions: 7e-7 of a logit)
constexpr int kGroupPieces = 1;          // fp32 operands or gradients
__host__ __device__ __forceinline__ int cut_of(bool logits, int passes) { return logits || passes >= 6 ? 2 : 4; }

// How many sums a tile's product along k-blocks [kb0, kb1) of `depth` is made of. Of pieces: one of the small products a group, and
// of the largest one every `cut` instructions, of which the last k-block has as many as there is depth for.
__host__ __device__ constexpr int sums_of(int kb0, int kb1, int group, int passes, int64_t depth, int cut) {
  const int groups = group < kb1 - kb0 ? (kb1 - kb0 + group - 1) / group : 1;
  if (passes == 1) return groups;
  const int64_t left = (depth - static_cast<int64_t>(kb1 - 1) * kBK + 15) / 16;
  const int steps = left < kBK / 16 ? static_cast<int>(left) : kBK / 16;
  return groups + (kb1 - kb0 - 1) * (kBK / 16 / cut) + (steps + cut - 1) / cut;
}

// The same as the issuing threads make them (vocab_product_kernel, few_products), counted: an epilogue that waited for another
// number would wait in vain.
constexpr int sums_issued(int kb0, int kb1, int group, int passes, int64_t depth, int cut) {
  int n = 0;
  for (int k0 = kb0; k0 < kb1; k0 += group < kb1 - k0 ? group : kb1 - k0) {
    const int len = group < kb1 - k0 ? group : kb1 - k0;
    ++n;
    for (int kb = 0, at = k0; kb < len * passes; ++kb) {
      const int64_t left = depth - static_cast<int64_t>(at) * kBK;
      if (++at == k0 + len) at = k0;
      for (int k = 0; k < kBK / 16 && k * 16 < left; ++k)
        if (passes > 1 && kb >= len * (passes - 1) && k % cut == 0) ++n;
    }
  }
  return n;
}

constexpr bool sums_agree() {
  const int all[] = {1, 2, 3, 10, 1 << 30}, pieces[] = {1, 3, 6};
  for (int group : all)
    for (int passes : pieces)
      for (int cut = 2; cut <= 8; cut *= 2)
        for (int kb0 = 0; kb0 < 3; ++kb0)
          for (int64_t depth = kb0 * kBK + 1; depth <= (kb0 + 7) * kBK; depth += 61)
            for (int kb1 = static_cast<int>((depth + kBK - 1) / kBK); kb1 > kb0; kb1 -= 2)
              if (sums_of(kb0, kb1, group, passes, depth, cut) != sums_issued(kb0, kb1, group, passes, depth, cut)) return false;
  return true;
}
static_assert(sums_agree(), "the epilogue waits for other sums than are made");

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Sums in groups take 128 registers a thread in the epilogue: its two warpgroups take over what the first does not need.
constexpr int kLaunchRegs = 168, kIssueRegs = 72, kEpiRegs = 216;
static_assert(kIssueRegs * 128 + kEpiRegs * 256 <= kLaunchRegs * kThreads, "a warpgroup would wait for registers that nobody gives up");

constexpr float kSumLimit = 0x1p57f;     // of a tile's row; above it the row changes its reference
// A row's factor weight / sum below this takes lse for the row's reference, so that its sum is 1: f h has pieces 2^-16 of it, and
// h may be small, where numbers end at 2^-126. (With weights of 1 no sum comes near.)
constexpr float kLeastFactor = 0x1p-90f;

// The kernels of a call but its first are scheduled while the one before still runs. Each waits for that one's end
// before it reads or writes memory, and reads what earlier kernels wrote by coherent loads.
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct VocabMaps {
  CUtensorMap h, W, U, Ust, F;           // U for loads and (boxes of 32 rows and columns) for stores; F: f h
  CUtensorMap Ufew;                      // U in boxes of as many rows as `few` has columns
  CUtensorMap Gh, Gw;                    // the gradients, for stores
};

struct VocabArgs {
  const void *h, *W;                     // as given
  const int32_t *targets, *ids;          // [N] or [N, K]
  const void* tlogits;                   // [N, K]
  const float* row_weight;
  float *loss, *lse;
  int32_t* err;
  __nv_bfloat16 *hp, *Wp;                // pieces [pieces][rows][dp], or null
  __nv_bfloat16 *U, *F;                  // [pieces][Nc][Vp], [pieces][Nc][dp]
  float2* sums;                          // [segments: halves of the first product's tiles][Nc]: reference (log2), sum
  float *zk, *wk;                        // [Nc][K] targets' logits <h, W_j>, weights (-1: none, or a later place of the same)
  int32_t* sorted;                       // [Nc][K] listed tokens, ascending (zk and wk in their order), then INT_MAX
  const int32_t* listed;                 // sorted, or the chunk's targets
  uint16_t* at;                          // [segments + 1][Nc] where in it each segment's tokens begin
  float *c, *a;                          // [Nc] reference (log2; +inf: no target), the sum of w log w
  float* f;                              // [Nc]
  float* acc;                            // [V][d] dW over chunks, or null
  float *parts, *parts_w;                // [q][Nc][d] of dh, [q_w][V][d] of dW, or null
  void *gh, *gw;
  int* err_word;
  int64_t row0;                          // of the chunk
  int64_t V, Vp;
  int N, Nc, d, dp, K, rows;             // rows: of this chunk
  int h_dtype, w_dtype, t_dtype, gh_dtype, gw_dtype;
  int np_h, np_w, np_u, np_f;            // pieces
  int accumulate, first, last;           // first, last chunk
  float k2;                              // scale log2(e)
  float scale, inv_t, zl, grad_scale;
  // schedule of the gradients' products
  int q, q_w, tiles2, tiles3, nd, light, delta, heavy;  // parts of dh and dW; tiles of each; tiles a row of them
  int passes_h, passes_w;                // piece products of dh, dW
  int group, group_h, group_w;           // k-blocks that one sum in TMEM takes: logits, dh, dW
  int wide, seg, seg_log;                // columns of a logits tile, and of a segment of it (its half), and that's log2
  int twice;                             // U is made once the rows' sums are there, by the logits again
  int tma_h, tma_w;                      // tiles of dh, dW go out by TMA
  int few_h;                             // dh is made for few rows
  int small;                             // few rows and an fp32 W: FMAs
  int at_log;                            // log2 of the tokens that a place of `at` stands for
  int segs;                              // sums a row
};

// ------------------------------------------------------------------- fp32 values as bf16 pieces

__device__ __forceinline__ uint16_t bf16_bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// x becomes what rounding it to bf16 left; returns the rounded value's bits. (Infinities and NaN leave 0.) FULL: x may be any
// number, also one next to fp32's largest, which rounding would make infinite: at most bf16's largest is taken. (Infinities and
// NaN are the next piece's then. For all three pieces, with comparisons of the bits: 16 x 128,000 x 2560 1204 us, 1130 like this.)
template <bool FULL = false>
__device__ __forceinline__ uint16_t take_piece(float& x) {
  constexpr float kMost = 0x1.FEp127f;
  const uint16_t b = bf16_bits(FULL ? fminf(fmaxf(x, -kMost), kMost) : x);
  const float r = __uint_as_float(static_cast<uint32_t>(b) << 16);
  x = FULL || fabsf(r) <= 3.4e38f ? x - r : 0.f;
  return b;
}

template <bool FULL = false>
__device__ __forceinline__ uint4 take_pieces(float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = take_piece<FULL>(x[2 * k]), hi = take_piece<FULL>(x[2 * k + 1]);
    w[k] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Products of pieces (i, j) with i + j below the larger count, the smallest first: what is left out is below 2^-8 of
// the smallest kept.
__host__ __device__ __forceinline__ int passes_of(int a, int b) {
  const int m = a > b ? a : b;
  int n = 0;
  for (int i = 0; i < a; ++i)
    for (int j = 0; j < b; ++j) n += i + j < m;
  return n;
}

__device__ __forceinline__ void piece_of(int a, int b, int pass, int* i, int* j) {
  int n = 0;
  for (int both = (a > b ? a : b) - 1; both >= 0; --both)
    for (*i = 0; *i <= both; ++*i) {
      *j = both - *i;
      if (*i < a && *j < b && n++ == pass) return;
    }
}

// dst [pieces][rows][dp] from src [rows][d], zeros behind a row's end, 8 columns a thread. Also the copy of bf16 rows
// that TMA cannot take as they are (d % 8 != 0). Bound by memory.
template <int DT, bool VEC>
__device__ void split_rows(const void* src, int64_t rows, int d, int dp, int pieces, __nv_bfloat16* dst, int64_t block) {
  const int per_row = dp / 8;
  const int64_t at = block * kPrepThreads + threadIdx.x, r = at / per_row;
  if (r >= rows) return;
  const int c = static_cast<int>(at - r * per_row) * 8;
  float x[8] = {};
  if (VEC) {
    if (c < d) load_cols<DT, 8>(src, r * d + c, x);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float y[1] = {0.f};
      if (c + k < d) load_cols<DT, 1>(src, r * d + c + k, y);
      x[k] = y[0];
    }
  }
  *reinterpret_cast<uint4*>(dst + r * dp + c) = take_pieces<DT == PG_F32>(x);
  for (int p = 1; p < pieces; ++p) *reinterpret_cast<uint4*>(dst + (p * rows + r) * dp + c) = take_pieces(x);
}

// --------------------------------------------------------------------------- the targets' logits

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// <h_i, W_j> of up to E rows j by one warp, fp32 in a fixed order.
template <int HT, int WT, bool VEC, int E>
__device__ __forceinline__ void warp_dots(const VocabArgs& g, int64_t i, const int64_t (&j)[E], float (&sum)[E]) {
  constexpr int kStep = VEC ? 8 : 1;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.f;
#pragma unroll 8
  for (int c = lane * kStep; c < g.d; c += 32 * kStep) {
    float x[kStep], y[E][kStep];
    load_cols<HT, kStep>(g.h, i * g.d + c, x);
#pragma unroll
    for (int e = 0; e < E; ++e) load_cols<WT, kStep>(g.W, j[e] * g.d + c, y[e]);
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < kStep; ++k) sum[e] = fmaf(x[k], y[e][k], sum[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = warp_sum(sum[e]);
}

// A logit as a reference: +infinity stands for a row without a target, and what is relative to -infinity is NaN.
__device__ __forceinline__ float as_reference(float z) {
  return z == INFINITY ? __int_as_float(0x7fffffff) : z == -INFINITY ? -0x1.FFFFFEp127f : z;
}

// Cross entropy: one warp a row, a row of h and one of W.
template <int HT, int WT, bool VEC>
__device__ void target_rows(const VocabArgs& g, int block) {
  const int r = block * (kPrepThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= g.rows) return;
  const int64_t i = g.row0 + r, t = __ldg(g.targets + i);
  const bool valid = t >= 0 && t < g.V;
  float z[1] = {0.f};
  if (valid) {
    const int64_t j[1] = {t};
    warp_dots<HT, WT, VEC, 1>(g, i, j, z);
  }
  if (lane != 0) return;
  if (!valid && g.err) atomicMin(reinterpret_cast<unsigned int*>(g.err), static_cast<unsigned int>(i));
  g.zk[r] = z[0];
  g.wk[r] = valid ? 1.f : -1.f;
  g.c[r] = valid ? as_reference(z[0] * g.k2) : INFINITY;
}

// 32 R keys, key m * 32 + lane in x[m] of a lane, in ascending order (bitonic).
template <int R>
__device__ __forceinline__ void sort_keys(uint32_t (&x)[R]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32 * R; k *= 2)
#pragma unroll
    for (int j = k / 2; j; j /= 2)
#pragma unroll
      for (int m = 0; m < R; ++m) {
        if (j >= 32) {
          if (m & (j / 32)) continue;
          const bool up = !(m * 32 & k);
          const uint32_t a = x[m], b = x[m | j / 32];
          x[m] = up ? min(a, b) : max(a, b);
          x[m | j / 32] = up ? max(a, b) : min(a, b);
        } else {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, x[m], j);
          const bool up = !((m * 32 + lane) & k);
          x[m] = up == !(lane & j) ? min(x[m], other) : max(x[m], other);
        }
      }
}

// (u - top) / T of a finite u. The difference first: u / T may be infinite where the list's differences are ordinary, and is
// rounded at u's size. Where the difference passes fp32's range (signs differ), T is divided by first.
__device__ __forceinline__ float over_temperature(float u, float top, float inv_t) {
  const float d = u - top;
  return d > -INFINITY ? d * inv_t : u * inv_t - top * inv_t;
}

// Distillation: one warp a row, 8 rows a block. The teacher's softmax; the list sorted by token (R registers of a lane), so
// that the tiles of the first product find what is theirs (`at`, where each segment's tokens begin) and keep those logits;
// and the dot product of the heaviest token, for a reference. (Dot products of all listed tokens took 101 of 1346 us at
// 8192 x 50,304 x 768 with lists of 32.) Bound by its instructions: 4096 lists of 64 12 us.
template <int HT, int WT, bool VEC, int R>
__device__ void list_rows(const VocabArgs& g, int block, uint32_t (*s_key)[kMaxList], float (*s_w)[kMaxList], uint16_t (*s_at)[8]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = block * (kPrepThreads / 32) + warp;
  const bool there = r < g.rows;
  const int64_t i = g.row0 + (there ? r : 0);
  constexpr uint32_t kNone = 0xFFFFFFFFu;  // (tokens are below 2^24 - 1)
  float u[R];
  uint32_t key[R];                         // token and place
  float top = -INFINITY;
  bool outside = false, poison = false;
#pragma unroll
  for (int m = 0; m < R; ++m) {
    const int k = m * 32 + lane;
    u[m] = -INFINITY;
    key[m] = kNone;
    if (k >= g.K || !there) continue;
    const int32_t token = __ldg(g.ids + i * g.K + k);
    if (token >= 0 && token < g.V) {
      key[m] = static_cast<uint32_t>(token) << 8 | static_cast<uint32_t>(k);
      float y[1];
      if (g.t_dtype == PG_F32) load_cols<PG_F32, 1>(g.tlogits, i * g.K + k, y);
      else load_cols<PG_BF16, 1>(g.tlogits, i * g.K + k, y);
      u[m] = y[0];
      poison |= !(u[m] < INFINITY);  // (also NaN, which fmaxf passes over)
      top = fmaxf(top, u[m]);
    } else {
      outside = true;
    }
  }
  top = warp_max(top);
  poison = __any_sync(0xffffffffu, poison);
  if (__any_sync(0xffffffffu, outside) && lane == 0 && g.err)
    atomicMin(reinterpret_cast<unsigned int*>(g.err), static_cast<unsigned int>(i));
  const bool some = poison || top > -INFINITY;
  uint32_t heaviest = kNone;
  float total = 0.f;
#pragma unroll
  for (int m = 0; m < R; ++m) {
    if (u[m] == top) heaviest = min(heaviest, key[m]);
    if (!some) key[m] = kNone;
    u[m] = u[m] == -INFINITY ? -INFINITY : over_temperature(u[m], top, g.inv_t);
    total += expf(u[m]);
  }
  total = warp_sum(total);
  const float log_total = logf(total);
  float a = 0.f;
#pragma unroll
  for (int m = 0; m < R; ++m) {
    const float logp = poison ? __int_as_float(0x7fffffff) : u[m] - log_total, w = !some ? 0.f : expf(logp);
    s_w[warp][m * 32 + lane] = w;
    if (key[m] != kNone && !(w == 0.f)) a += w * logp;
  }
  a = warp_sum(a);
  heaviest = __reduce_min_sync(0xffffffffu, heaviest);
  float z[1] = {0.f};
  if (some && there) {
    const int64_t j[1] = {heaviest == kNone ? 0 : heaviest >> 8};
    warp_dots<HT, WT, VEC, 1>(g, i, j, z);
  }
  sort_keys<R>(key);
#pragma unroll
  for (int m = 0; m < R; ++m) s_key[warp][m * 32 + lane] = key[m];
  __syncwarp();
#pragma unroll
  for (int m = 0; m < R; ++m) {
    const int k = m * 32 + lane;
    if (k >= g.K || !there) continue;
    const uint32_t token = key[m] >> 8;
    float w = -1.f;  // what the gradient puts at the token: its later places count with its first
    if (key[m] != kNone && (k == 0 || s_key[warp][k - 1] >> 8 != token)) {
      w = s_w[warp][key[m] & 255];
      for (int e = k + 1; e < g.K && s_key[warp][e] >> 8 == token; ++e) w += s_w[warp][s_key[warp][e] & 255];
    }
    const int64_t to = static_cast<int64_t>(r) * g.K + k;
    g.sorted[to] = key[m] == kNone ? INT_MAX : static_cast<int32_t>(token);
    g.wk[to] = w;
  }
  if (lane == 0 && there) {
    g.c[r] = some ? as_reference(poison ? __int_as_float(0x7fffffff) : z[0] * g.k2) : INFINITY;
    g.a[r] = some ? a : 0.f;
  }
  // where each segment's tokens begin: a lane walks a run of segments, the block stores its 8 rows' together
  const int segs = static_cast<int>((g.V + (1 << g.at_log) - 1) >> g.at_log);
  for (int q0 = 0; q0 <= segs; q0 += kAtOnce) {
    const int n = min(kAtOnce, segs + 1 - q0), run = (n + 31) / 32;
    int pos = 0;
    const uint32_t start = min(static_cast<uint32_t>(q0 + lane * run) << g.at_log, kNone >> 8);
#pragma unroll
    for (int step = 16 * R; step; step >>= 1)
      if ((s_key[warp][pos + step - 1] >> 8) < start) pos += step;
    if (s_key[warp][pos] >> 8 < start) ++pos;  // (32 R - 1 of them at most so far)
    for (int q = lane * run; q < min(n, (lane + 1) * run); ++q) {
      const uint32_t from = min(static_cast<uint32_t>(q0 + q) << g.at_log, kNone >> 8);
      while (pos < 32 * R && s_key[warp][pos] >> 8 < from) ++pos;
      s_at[q][warp] = static_cast<uint16_t>(pos);
    }
    __syncthreads();
    for (int q = threadIdx.x; q < n; q += kPrepThreads)
      *reinterpret_cast<uint4*>(g.at + static_cast<int64_t>(q0 + q) * g.Nc + block * 8) = *reinterpret_cast<const uint4*>(s_at[q]);
    __syncthreads();
  }
}

// What the products need beforehand: the pieces of W (first chunk) and of the chunk's h, and the rows' targets.
template <int HT, int WT, bool VEC, bool LIST>
__global__ void __launch_bounds__(kPrepThreads) vocab_prepare_kernel(const __grid_constant__ VocabArgs g, int blocks_w, int blocks_h) {
  grid_dep_wait();
  grid_dep_launch();
  int block = blockIdx.x;
  if (block < blocks_w) {
    split_rows<WT, VEC>(g.W, g.V, g.d, g.dp, g.np_w, g.Wp, block);
  } else if ((block -= blocks_w) < blocks_h) {
    const uint8_t* h = static_cast<const uint8_t*>(g.h) + g.row0 * g.d * (HT == PG_F32 ? 4 : 2);
    split_rows<HT, VEC>(h, g.rows, g.d, g.dp, g.np_h, g.hp, block);
  } else if constexpr (LIST) {
    __shared__ uint32_t s_key[LIST ? 8 : 1][kMaxList];
    __shared__ float s_w[LIST ? 8 : 1][kMaxList];
    __shared__ __align__(16) uint16_t s_at[LIST ? kAtOnce : 1][8];
    block -= blocks_h;
    if (g.K <= 32) list_rows<HT, WT, VEC, 1>(g, block, s_key, s_w, s_at);
    else if (g.K <= 64) list_rows<HT, WT, VEC, 2>(g, block, s_key, s_w, s_at);
    else if (g.K <= 128) list_rows<HT, WT, VEC, 4>(g, block, s_key, s_w, s_at);
    else list_rows<HT, WT, VEC, 8>(g, block, s_key, s_w, s_at);
  } else {
    target_rows<HT, WT, VEC>(g, block - blocks_h);
  }
}

// --------------------------------------------------------------------------------- products

enum VocabKind { kSums, kKeep, kGrads, kAgain };  // logits without and with U; the gradients; the logits again, for U alone

// One tile of a product D = P Q^T: the k-blocks [kb0, kb1) of each piece product.
struct VocabJob {
  const CUtensorMap *P, *Q;
  bool p_mn, q_mn;
  int np_p, np_q, passes;
  int i;                                 // tile's row, in tiles
  int64_t col0;                          // its first column
  int n;                                 // its columns: as many as there are left, to 32
  int kb0, kb1;
  int64_t depth;                         // of the whole product
  int group;                             // k-blocks of one sum in TMEM
  int product, part;                     // 0: logits, 1: dh, 2: dW
};

__device__ __forceinline__ int columns(int64_t left, int wide) {
  return left < wide ? (static_cast<int>(left) + 31) / 32 * 32 : wide;
}

// The r-th job of this unit; false behind the last.
// The gradients: first the units of dh (its tiles in q parts along V, part by part so that the units at work read the
// same rows of W), then the tiles of dW. Where the units of dh do not come out even, those that have one fewer take
// `delta` tiles of dW more.
template <int KIND>
__device__ __forceinline__ bool job_at(const VocabArgs& g, const VocabMaps& maps, int unit, int units, int r, VocabJob* w) {
  if constexpr (KIND != kGrads) {
    // tiles that are at work together share their rows of W, and h stays in L2
    const int nm = (g.rows + kTile - 1) / kTile;
    const uint32_t t = static_cast<uint32_t>(r) * units + unit;
    if (t >= static_cast<uint32_t>(nm) * static_cast<uint32_t>((g.V + g.wide - 1) / g.wide)) return false;
    w->P = &maps.h;
    w->Q = &maps.W;
    w->p_mn = w->q_mn = false;
    w->np_p = g.np_h;
    w->np_q = g.np_w;
    w->passes = passes_of(g.np_h, g.np_w);
    w->i = static_cast<int>(t % static_cast<uint32_t>(nm));
    w->col0 = static_cast<int64_t>(t / static_cast<uint32_t>(nm)) * g.wide;
    w->n = columns(g.V - w->col0, g.wide);
    w->kb0 = 0;
    w->kb1 = (g.d + kBK - 1) / kBK;
    w->depth = g.d;
    w->group = g.group;
    w->product = w->part = 0;
    return true;
  } else {
    const int n2 = g.tiles2 * g.q, mine = n2 / units + (unit < g.heavy);
    if (r < mine) {
      const int u = r * units + unit, t = u % g.tiles2;
      const int64_t all = (g.V + kBK - 1) / kBK;
      w->part = u / g.tiles2;
      w->P = &maps.U;
      w->Q = &maps.W;
      w->p_mn = false;
      w->q_mn = true;
      w->np_p = g.gh_dtype == PG_F32 ? g.np_u : 1;
      w->np_q = g.gh_dtype == PG_F32 ? g.np_w : 1;
      w->passes = g.passes_h;
      w->i = t / g.nd;
      w->col0 = t % g.nd * kTile;
      w->n = columns(g.d - w->col0, kTile);
      w->depth = g.V;
      w->kb0 = static_cast<int>(all * w->part / g.q);
      w->kb1 = static_cast<int>(all * (w->part + 1) / g.q);
      w->group = g.group_h;
      w->product = 1;
      return true;
    }
    r -= mine;
    int t;
    if (unit >= g.heavy && r < g.delta) {
      t = r * g.light + (unit - g.heavy);
    } else {
      if (unit >= g.heavy) r -= g.delta;
      t = g.delta * g.light + r * units + unit;
    }
    if (t >= g.tiles3 * g.q_w) return false;
    w->part = t / g.tiles3;
    t -= w->part * g.tiles3;
    const int all = (g.rows + kBK - 1) / kBK;
    w->P = &maps.U;
    w->Q = &maps.F;
    w->p_mn = w->q_mn = true;
    w->np_p = g.gw_dtype == PG_F32 ? g.np_u : 1;
    w->np_q = g.gw_dtype == PG_F32 ? g.np_f : 1;
    w->passes = g.passes_w;
    w->i = t / g.nd;
    w->col0 = t % g.nd * kTile;
    w->n = columns(g.d - w->col0, kTile);
    w->depth = g.rows;
    w->kb0 = static_cast<int>(static_cast<int64_t>(all) * w->part / g.q_w);
    w->kb1 = static_cast<int>(static_cast<int64_t>(all) * (w->part + 1) / g.q_w);
    w->group = g.group_w;
    w->product = 2;
    return true;
  }
}

struct VocabBars {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// `wait` without a call, across which the sums that the epilogue holds in registers would have to be saved.
template <bool PAIR>
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (poll<PAIR>(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  while (!poll<PAIR>(bar, parity))
    if (*abort || now_ns() - t0 > kAsyncWaitNs) return false;
  return true;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// All but the latest of this thread's stores have read their shared memory.
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Logits of a tile: a warp has 32 rows (a lane each) and 128 columns, 32 at a time. u = 2^(k2 z - c) in fp32 for the row's sum,
// and to U through the warp's shared memory (32 rows of 64 bytes, swizzled as the TMA store reads them; two such buffers in turn, so
// that a store reads one while the other fills). skip: the column of the row's target, which its sum leaves out, or -1.
template <int KIND>
__device__ __forceinline__ float logits_half(const VocabArgs& g, const VocabMaps& maps, uint32_t from, uint8_t* s_row, int row0, int64_t col0,
                                             float c, bool dead, float f, int skip) {
  constexpr bool KEEP = KIND != kSums;
  const int lane = threadIdx.x & 31;
  const int64_t end = min(col0 + g.seg, g.V);
  const uint64_t k2 = pk(g.k2, g.k2), c2 = pk(-c, -c);
  const bool some_dead = KEEP && __any_sync(0xffffffffu, dead), some_skip = KIND != kAgain && __any_sync(0xffffffffu, skip >= 0);
  uint64_t sum[2] = {0, 0};
  if (KEEP && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // of an earlier tile
  __syncwarp();
  uint32_t r[2][32];
  tmem_load(from, r[0]);
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const int64_t c0 = col0 + ch * 32;
    if (c0 >= end) break;
    tmem_wait(r[ch & 1]);
    if (ch < 3) tmem_load(from + (ch + 1) * 32, r[(ch + 1) & 1]);
    float x[32];
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      upk(fma2(pk(__uint_as_float(r[ch & 1][k]), __uint_as_float(r[ch & 1][k + 1])), k2, c2), x[k], x[k + 1]);
      x[k] = exp2_fast(x[k]);
      x[k + 1] = exp2_fast(x[k + 1]);
    }
    if (c0 + 32 > end) {
      const int left = static_cast<int>(end - c0);
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = k < left ? x[k] : 0.f;
    }
    const uint32_t out = skip >> 5 == ch ? 1u << (skip & 31) : 0u;
    if (some_skip && __any_sync(0xffffffffu, out)) {
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = out >> k & 1 ? 0.f : x[k];
    }
    if constexpr (KIND == kAgain) {
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] *= f;
    } else {
#pragma unroll
      for (int k = 0; k < 32; k += 2) sum[k / 2 & 1] = add2(sum[k / 2 & 1], pk(x[k], x[k + 1]));
    }
    if constexpr (KEEP) {
      for (int p = 0; p < g.np_u; ++p) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = two_bf16(x[2 * k], x[2 * k + 1]);
        if (p + 1 < g.np_u) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            x[2 * k] -= __uint_as_float(w[k] << 16);
            x[2 * k + 1] -= __uint_as_float(w[k] & 0xFFFF0000u);
          }
        }
        if (some_dead) {  // (a row without a target may hold anything)
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = dead ? 0u : w[k];
        }
        uint8_t* buf = s_row + ((ch * g.np_u + p) & 1) * (kStageBytes / 2);
        if (lane == 0) stores_read();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(buf + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)) =
              make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) store_box(&maps.Ust, smem_addr(buf), static_cast<int>(c0), row0, p);
        __syncwarp();  // (TMEM's loads and waits want all lanes at once)
      }
    }
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  float lo, hi;
  upk(add2(sum[0], sum[1]), lo, hi);
  return lo + hi;
}

// Token t's place among `wide` tokens from col0 on, or -1. (One past V is in no sum.)
__device__ __forceinline__ int place_in(int32_t t, int64_t col0, int wide) {
  const uint32_t at = static_cast<uint32_t>(t) - static_cast<uint32_t>(col0);
  return at < static_cast<uint32_t>(wide) ? static_cast<int>(at) : -1;
}

// The listed tokens of this lane's row that fall into a segment: places [e, end) of the sorted list, the first's token. Cross
// entropy: its target, wherever that is. (Read a tile ahead: nothing is done with it before.)
struct Listed {
  int e, end;
  int32_t token;
};

__device__ __forceinline__ Listed listed_in(const VocabArgs& g, int row, int64_t col0) {
  Listed l = {0, 0, -1};
  if (row >= g.rows || col0 >= g.V) return l;
  if (g.ids) {
    const int64_t seg = static_cast<uint32_t>(col0) >> g.at_log;
    l.e = g.at[seg * g.Nc + row];
    l.end = g.at[(seg + 1) * g.Nc + row];
  } else {
    l.token = g.listed[row];
  }
  return l;
}

__device__ __forceinline__ void first_listed(const VocabArgs& g, int row, Listed* l) {
  if (l->e < l->end) l->token = g.sorted[static_cast<int64_t>(row) * g.K + l->e];
}

// The listed tokens' logits of a warp's rows and segment. TMEM gives all lanes one column at a time, so a few of them are
// loaded one by one; from kDense on the columns pass through shared memory, where a lane reads its own.
constexpr int kDense = 48;

template <bool KEEP>
__device__ __noinline__ void keep_listed(const VocabArgs& g, uint8_t* s_row, uint32_t from, int row0, int64_t col0, Listed listed) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(row0 + lane) * g.K;
  if (__reduce_add_sync(0xffffffffu, listed.end - listed.e) >= kDense) {
    if (KEEP && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // (of U's tile before)
    __syncwarp();
#pragma unroll 1
    for (int c0 = 0; c0 < g.seg && col0 + c0 < g.V; c0 += 32) {
      uint32_t r[32];
      tmem_load(from + c0, r);
      tmem_wait(r);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4*>(s_row + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
      for (; listed.e < listed.end; ++listed.e) {
        const int at = static_cast<int>(g.sorted[row + listed.e] - col0) - c0;  // ascending
        if (at >= 32) break;
        g.zk[row + listed.e] = *reinterpret_cast<const float*>(s_row + lane * 128 + ((at >> 2 ^ (lane & 7)) << 4) + (at & 3) * 4);
      }
      __syncwarp();
    }
    return;
  }
  while (__any_sync(0xffffffffu, listed.e < listed.end)) {  // one a row at a time
    const bool mine = listed.e < listed.end;
    const int at = mine ? static_cast<int>(listed.token - col0) : -1;
    float y = 0.f;
    for (uint32_t left = __ballot_sync(0xffffffffu, mine); left;) {  // four in flight
      uint32_t v[4];
      int l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        l[k] = left ? __ffs(left) - 1 : 32;
        left &= left - 1;
        const int column = __shfl_sync(0xffffffffu, at, l[k] & 31);
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v[k]) : "r"(from + max(column, 0)));
      }
      tmem_wait(v);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane == l[k]) y = __uint_as_float(v[k]);
    }
    if (mine) {
      g.zk[row + listed.e] = y;
      if (++listed.e < listed.end) listed.token = g.sorted[row + listed.e];
    }
  }
}

template <int KIND>
__device__ __forceinline__ void logits_epilogue(const VocabArgs& g, const VocabMaps& maps, const VocabJob& w, uint8_t* s_row,
                                                uint32_t from, int row0, int half, float c, Listed listed) {
  constexpr bool KEEP = KIND != kSums;
  const int lane = threadIdx.x & 31;
  const int64_t col0 = w.col0 + half * g.seg;
  if (row0 >= g.rows || col0 >= g.V) return;
  if constexpr (KIND == kAgain) {  // f is the row's part of the gradient over its sum
    const float f = row0 + lane < g.rows ? g.f[row0 + lane] : 0.f;
    logits_half<KIND>(g, maps, from, s_row, row0, col0, c, f == 0.f, f, -1);
    return;
  }
  // A target's own term is not in its row's sum: vocab_rows_kernel adds it, and has what p leaves over without a difference of
  // numbers near one
  const int skip = g.ids ? -1 : place_in(listed.token, col0, g.seg);
  if (g.ids) keep_listed<KEEP>(g, s_row, from, row0, col0, listed);
  const bool dead = row0 + lane >= g.rows || c == INFINITY;
  float sum = logits_half<KIND>(g, maps, from, s_row, row0, col0, c, dead, 1.f, skip);
  float ref = c;
  const bool over = !dead && !(sum <= kSumLimit);
  if (__any_sync(0xffffffffu, over)) {  // logits far above the targets': the tile's largest for a reference
    float top = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      uint32_t r[32];
      tmem_load(from + h * 32, r);
      tmem_wait(r);
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (h * 32 + k < g.seg && col0 + h * 32 + k < g.V) top = fmaxf(top, __uint_as_float(r[k]) * g.k2);
    }
    if (over) ref = top == -INFINITY ? 0.f : top;
    if (KEEP && lane == 0) stores_done();  // the same places are written again
    __syncwarp();
    sum = logits_half<KIND>(g, maps, from, s_row, row0, col0, ref, dead, 1.f, skip);
  }
  if (row0 + lane < g.rows) g.sums[static_cast<int64_t>(static_cast<uint32_t>(col0) >> g.seg_log) * g.Nc + row0 + lane] = make_float2(ref, sum);
}

// Where this chunk's dW goes, and what is added to it.
__device__ __forceinline__ void table_target(const VocabArgs& g, void** dst, int* dtype, const float** add32, const __nv_bfloat16** add16) {
  const bool through = g.acc && !g.last;
  *dtype = through ? PG_F32 : g.gw_dtype;
  *dst = through ? g.acc : g.gw;
  if (g.gw_dtype == PG_F32) {
    if (!g.first || g.accumulate) *add32 = static_cast<const float*>(g.gw);
  } else {
    if (!g.first) *add32 = g.acc;
    if (g.last && g.accumulate) *add16 = static_cast<const __nv_bfloat16*>(g.gw);
  }
}

// A gradient's tile. TMEM gives a lane one row; global memory wants neighbouring lanes on one row, so 32 columns
// at a time pass through the warp's shared memory.
__device__ __forceinline__ void grad_epilogue(const VocabArgs& g, const VocabMaps& maps, const VocabJob& w, uint8_t* s_row,
                                              uint32_t from, int row0, int half) {
  const int lane = threadIdx.x & 31;
  const bool dh = w.product == 1, part = dh ? g.parts != nullptr : g.parts_w != nullptr;
  const int64_t rows = dh ? g.rows : g.V;
  if (row0 >= rows) return;
  float f = 1.f;
  if (dh && !part && !g.twice) f = row0 + lane < rows ? g.f[row0 + lane] : 0.f;
  void* dst;
  int dtype = PG_F32;
  const float* add32 = nullptr;
  const __nv_bfloat16* add16 = nullptr;
  if (part) {
    dst = dh ? g.parts + static_cast<int64_t>(w.part) * g.Nc * g.d : g.parts_w + static_cast<int64_t>(w.part) * g.V * g.d;
  } else if (dh) {
    dtype = g.gh_dtype;
    dst = static_cast<uint8_t*>(g.gh) + g.row0 * g.d * (dtype == PG_F32 ? 4 : 2);
  } else {
    table_target(g, &dst, &dtype, &add32, &add16);
  }
  const bool vec = g.d % 4 == 0 && reinterpret_cast<uintptr_t>(dst) % (dtype == PG_F32 ? 16 : 8) == 0 &&
                   (!add32 || reinterpret_cast<uintptr_t>(add32) % 16 == 0);
  uint32_t r2[2][32];
  __syncwarp();  // (of the last rows' tile some lanes have read f)
  tmem_load(from, r2[0]);
  if (dh ? g.tma_h : g.tma_w) {  // rows past the last and columns past d are cut off
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // of an earlier tile
    __syncwarp();
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      const int c0 = static_cast<int>(w.col0) + half * (kTile / 2) + ch * 32;
      if (c0 >= g.d) break;
      uint32_t(&r)[32] = r2[ch & 1];
      tmem_wait(r);
      if (ch < 3) tmem_load(from + (ch + 1) * 32, r2[(ch + 1) & 1]);
      float x[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] = f == 0.f ? 0.f : f * __uint_as_float(r[k]);
      uint8_t* buf = s_row;
      if (dtype == PG_F32) {  // one buffer of 32 rows of 128 bytes
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4*>(buf + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
      } else {                // two of 64, in turn
        buf += (ch & 1) * (kStageBytes / 2);
        if (lane == 0) stores_read();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(buf + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)) =
              make_uint4(two_bf16(x[8 * k], x[8 * k + 1]), two_bf16(x[8 * k + 2], x[8 * k + 3]), two_bf16(x[8 * k + 4], x[8 * k + 5]),
                         two_bf16(x[8 * k + 6], x[8 * k + 7]));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) store_box(dh ? &maps.Gh : &maps.Gw, smem_addr(buf), c0, row0, 0);
      __syncwarp();
    }
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    return;
  }
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const int c0 = static_cast<int>(w.col0) + half * (kTile / 2) + ch * 32;
    if (c0 >= g.d) break;
    uint32_t(&r)[32] = r2[ch & 1];
    tmem_wait(r);
    if (ch < 3) tmem_load(from + (ch + 1) * 32, r2[(ch + 1) & 1]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float4 v;
      float* x = &v.x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = f == 0.f ? 0.f : f * __uint_as_float(r[4 * k + e]);
      *reinterpret_cast<float4*>(s_row + lane * 128 + ((k ^ (lane & 7)) << 4)) = v;
    }
    __syncwarp();
    if (vec) {  // (d % 4 == 0: four columns are inside or outside together)
      const int lc = lane & 7, col = c0 + lc * 4;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int lr = 4 * k + (lane >> 3);
        if (row0 + lr >= rows || col >= g.d) continue;
        float4 v = *reinterpret_cast<const float4*>(s_row + lr * 128 + ((lc ^ (lr & 7)) << 4));
        const int64_t at = static_cast<int64_t>(row0 + lr) * g.d + col;
        if (add32) {
          const float4 o = *reinterpret_cast<const float4*>(add32 + at);
          v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
        }
        if (add16) {
          const uint2 o = *reinterpret_cast<const uint2*>(add16 + at);
          v.x += __uint_as_float(o.x << 16); v.y += __uint_as_float(o.x & 0xFFFF0000u);
          v.z += __uint_as_float(o.y << 16); v.w += __uint_as_float(o.y & 0xFFFF0000u);
        }
        if (dtype == PG_F32) *reinterpret_cast<float4*>(static_cast<float*>(dst) + at) = v;
        else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dst) + at) = make_uint2(two_bf16(v.x, v.y), two_bf16(v.z, v.w));
      }
    } else {
      const int col = c0 + lane;
#pragma unroll 4
      for (int lr = 0; lr < 32; ++lr) {
        if (row0 + lr >= rows || col >= g.d) break;
        float v = *reinterpret_cast<const float*>(s_row + lr * 128 + (((lane >> 2) ^ (lr & 7)) << 4) + (lane & 3) * 4);
        const int64_t at = static_cast<int64_t>(row0 + lr) * g.d + col;
        if (add32) v += add32[at];
        if (add16) v += __bfloat162float(add16[at]);
        if (dtype == PG_F32) static_cast<float*>(dst)[at] = v;
        else static_cast<__nv_bfloat16*>(dst)[at] = __float2bfloat16_rn(v);
      }
    }
    __syncwarp();
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

template <int KIND, bool GROUPS>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_product_kernel(const __grid_constant__ VocabMaps maps, const __grid_constant__ VocabArgs g) {
  extern __shared__ uint8_t s_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  __shared__ VocabBars bars_s;
  VocabBars* bars = &bars_s;
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(smem_addr(&bars->full[s]), 1);
      bar_init(smem_addr(&bars->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(smem_addr(&bars->acc_full[s]), 1);
      bar_init(smem_addr(&bars->acc_empty[s]), 2 * kEpiWarps);
    }
    bar_init(smem_addr(&bars->done), 1);
    bars->abort = 0;
    bar_init_fence();
    fence_async_smem();
  }
  if (warp == 1) tmem_alloc<true>(smem_addr(&bars->tmem), kTmemCols);
  fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers and TMEM exist before any remote use
  fence_after();
  const uint32_t tmem = bars->tmem;
  grid_dep_wait();
  grid_dep_launch();

  int stage = 0, acc = 0;
  uint32_t ring_phase = 0, acc_phase = 0;
  bool fine = true;
  VocabJob w;
  if (warp < kEpiFirst) {
    if constexpr (GROUPS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0 && lane == 0) {
      for (int r = 0; fine && job_at<KIND>(g, maps, unit, units, r, &w); ++r) {
        const int p0 = w.i * kTile + static_cast<int>(rank) * 128, q0 = static_cast<int>(w.col0) + static_cast<int>(rank) * (w.n / 2);
        for (int k0 = w.kb0; k0 < w.kb1; k0 += w.group) {
          const int k1 = min(k0 + w.group, w.kb1);
          for (int pass = 0; fine && pass < w.passes; ++pass) {
            int zp = 0, zq = 0;
            if (w.passes > 1) piece_of(w.np_p, w.np_q, pass, &zp, &zq);
            for (int kb = k0; kb < k1; ++kb) {
              if (!wait<true>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u, abort)) {
                fine = false;
                break;
              }
              const uint32_t full = smem_addr(&bars->full[stage]);
              const uint32_t dp = smem_addr(ring + stage * (2 * kOperandBytes)), dq = dp + kOperandBytes;
              const uint32_t bar = in_cta(full, 0);
              if (rank == 0) bar_expect(full, 2 * 2 * kOperandBytes);
              load_operand<true, 128>(dp, w.P, w.P, w.p_mn, p0, kb * kBK, zp, bar);
              load_operand<true, 128>(dq, w.Q, w.Q, w.q_mn, q0, kb * kBK, zq, bar);
              if (++stage == kStages) {
                stage = 0;
                ring_phase ^= 1u;
              }
            }
          }
          if (!fine) break;
        }
      }
    }
    if (warp == 1 && lane == 0 && rank == 0) {
      for (int r = 0; fine && job_at<KIND>(g, maps, unit, units, r, &w); ++r) {
        const uint32_t idesc = kIdesc | (static_cast<uint32_t>(w.n >> 3) << 17) | (w.p_mn ? 1u << 15 : 0u) | (w.q_mn ? 1u << 16 : 0u);
        // 16 k further: 32 bytes along a K-major line (after four, the deeper half), two 8-k
        // groups of an MN-major tile
        const uint32_t step_p = w.p_mn ? 2048 >> 4 : 32 >> 4, step_q = w.q_mn ? 2048 >> 4 : 32 >> 4;
        const uint32_t half_p = w.p_mn ? 4 * step_p : kOperandBytes / 2 >> 4, half_q = w.q_mn ? 4 * step_q : kOperandBytes / 2 >> 4;
        uint32_t d = 0, more_of_it = 0;
        auto begin = [&]() {
          fine = fine && wait<true>(smem_addr(&bars->acc_empty[acc]), acc_phase ^ 1u, abort);
          fence_after();
          d = tmem + static_cast<uint32_t>(acc * kTile);
          more_of_it = 0;
        };
        auto finish = [&]() {
          commit<true>(smem_addr(&bars->acc_full[acc]));
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        };
        for (int k0 = w.kb0; fine && k0 < w.kb1; k0 += w.group) {
          const int len = min(k0 + w.group, w.kb1) - k0, blocks = len * w.passes;
          begin();
          for (int kb = 0, at = k0; fine && kb < blocks; ++kb) {
            if (!wait<true>(smem_addr(&bars->full[stage]), ring_phase, abort)) {
              fine = false;
              break;
            }
            fence_after();
            const uint32_t sp = smem_addr(ring + stage * (2 * kOperandBytes));
            const uint64_t dp = operand_desc(sp, w.p_mn), dq = operand_desc(sp + kOperandBytes, w.q_mn);
            const int64_t left = w.depth - static_cast<int64_t>(at) * kBK;  // (what is behind it is zero)
            const int cut = GROUPS && w.passes > 1 && kb >= blocks - len ? cut_of(KIND != kGrads, w.passes) : 0;
            if (++at == k0 + len) at = k0;
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              if (k * 16 >= left) break;
              if (cut && (k & (cut - 1)) == 0) {
                finish();
                begin();
              }
              if (!fine) break;
              mma_f16<true>(d, dp + (k / 4) * half_p + (k % 4) * step_p, dq + (k / 4) * half_q + (k % 4) * step_q, idesc, more_of_it);
              more_of_it = 1;
            }
            if (!fine) break;
            commit<true>(smem_addr(&bars->empty[stage]));
            if (++stage == kStages) {
              stage = 0;
              ring_phase ^= 1u;
            }
          }
          if (fine) finish();
        }
      }
    }
  } else {
    if constexpr (GROUPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quarter = warp & 3, half = (warp - kEpiFirst) >> 2;
    uint8_t* s_row = ring + kRing + (warp - kEpiFirst) * kStageBytes;
    // What a tile needs of its rows is read while the tile before is worked on.
    bool more = job_at<KIND>(g, maps, unit, units, 0, &w);
    float c = INFINITY, next_c = INFINITY;
    Listed listed = {0, 0, -1}, next_listed = {0, 0, -1};
    auto row_of = [&](const VocabJob& job) { return job.i * kTile + static_cast<int>(rank) * 128 + quarter * 32; };
    auto read_rows = [&](const VocabJob& job) {
      const int row = row_of(job) + lane;
      next_c = INFINITY;
      if (row < g.rows) next_c = g.c[row];
      if (KIND != kAgain) next_listed = listed_in(g, row, job.col0 + half * g.seg);
    };
    if (KIND != kGrads && more) {
      read_rows(w);
      if (KIND != kAgain && g.ids) first_listed(g, row_of(w) + lane, &next_listed);
    }
    for (int r = 0; fine && more; ++r) {
      const int row0 = row_of(w);
      VocabJob next;
      if (KIND != kGrads) {
        c = next_c;
        listed = next_listed;
      }
      more = job_at<KIND>(g, maps, unit, units, r + 1, &next);
      if (KIND != kGrads && more) read_rows(next);
      const uint32_t warp_from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                 static_cast<uint32_t>(half * (KIND == kGrads ? kTile / 2 : g.seg));
      auto acquire = [&]() {
        fine = __all_sync(0xffffffffu, wait_inline<true>(smem_addr(&bars->acc_full[acc]), acc_phase, abort));
        fence_after();
        return fine;
      };
      auto release = [&]() {
        fence_before();
        __syncwarp();
        // (Released to the CTA alone: what the issuing thread waits for are this warp's TMEM loads, which are done. A release
        // to the cluster waits until the epilogue's global stores are.)
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_cta(smem_addr(&bars->acc_empty[acc]), 0))
                       : "memory");
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      };
      const int sums = GROUPS ? sums_of(w.kb0, w.kb1, w.group, w.passes, w.depth, cut_of(KIND != kGrads, w.passes)) : 1;
      if (GROUPS && sums > 1) {
        // all but the last in registers; the last goes back to TMEM with the others added
        float z[128];
#pragma unroll
        for (int k = 0; k < 128; ++k) z[k] = 0.f;
        for (int k = 1; k < sums; ++k) {
          if (!acquire()) break;
          const uint32_t from = warp_from + static_cast<uint32_t>(acc * kTile);
          uint32_t r[2][16];  // 16 columns come while the 16 before are added
          tmem_load16(from, r[0]);
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            tmem_wait(r[ch & 1]);
            if (ch < 7) tmem_load16(from + (ch + 1) * 16, r[(ch + 1) & 1]);
#pragma unroll
            for (int k = 0; k < 16; ++k) z[ch * 16 + k] += __uint_as_float(r[ch & 1][k]);
          }
          release();
        }
        if (!fine || !acquire()) break;
        const uint32_t from = warp_from + static_cast<uint32_t>(acc * kTile);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          if (KIND != kGrads && ch * 32 >= g.seg) break;  // (the columns behind are the other half's)
          uint32_t r[32];
          tmem_load(from + ch * 32, r);
          tmem_wait(r);
#pragma unroll
          for (int k = 0; k < 32; ++k) z[ch * 32 + k] += __uint_as_float(r[k]);
          tmem_store(from + ch * 32, z + ch * 32);
        }
        tmem_stored();
      } else if (!acquire()) {
        break;
      }
      const uint32_t from = warp_from + static_cast<uint32_t>(acc * kTile);
      if constexpr (KIND == kGrads) grad_epilogue(g, maps, w, s_row, from, row0, half);
      else logits_epilogue<KIND>(g, maps, w, s_row, from, row0, half, c, listed);
      release();
      w = next;
      if (KIND != kGrads && KIND != kAgain && more && g.ids) first_listed(g, row_of(w) + lane, &next_listed);
    }
    if (KIND != kSums && lane == 0) stores_done();
  }
  if (!fine) {
    atomicOr(g.err_word, kErrVocab);
    *abort = 1;
  }
  __syncwarp();

  // every copy has landed and every MMA and commit has finished before the CTA (or its peer) may exit and its
  // TMEM is given back
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      const uint64_t t0 = now_ns();
      while (!poll<true>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u) && now_ns() - t0 < kAsyncWaitNs / 8) {
      }
      if (++stage == kStages) {
        stage = 0;
        ring_phase ^= 1u;
      }
    }
  }
  if (warp == 1 && lane == 0 && rank == 0) {
    commit_here<true>(smem_addr(&bars->done));
    const uint64_t t0 = now_ns();
    while (!poll<true>(smem_addr(&bars->done), 0) && now_ns() - t0 < kAsyncWaitNs) {
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  pair_sync();
  if (warp == 1) tmem_free<true>(tmem, kTmemCols);
}

// ------------------------------------------------------------------------------- few rows

// The first product for up to 128 rows, where reading W is all that counts: W's rows are the tile's rows (128 a CTA), the
// rows of h its columns (NT of them), so that a stage of the ring holds little beside W and the tensor core waits for
// it alone. A lane has one row of W and all rows of h; sums over a warp's 32 rows of W (a segment) by halving.
// 8 x 128,000 x 2560: 100 us, 6.55 TB/s, against 152 us on 256 x 256 tiles of pairs, whose ring holds 96 KB of W an SM.
template <int NT>
struct Few {
  static constexpr int kWBytes = 128 * kBK * 2, kHBytes = NT * kBK * 2;
  static constexpr int kStages = NT == 32 ? 5 : NT == 64 ? 4 : 3;
  static constexpr int kThreads = 192;
  static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(NT >> 3) << 17) | (8u << 24);
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * (kWBytes + kHBytes);
};

template <int NT>
struct FewBars {
  uint64_t full[Few<NT>::kStages], empty[Few<NT>::kStages], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// Lane t of a warp gets op over all lanes of x[t].
template <typename Op>
__device__ __forceinline__ float reduce_columns(float (&x)[32], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const bool up = lane & o;
      const float give = up ? x[k] : x[k + o], keep = up ? x[k + o] : x[k];
      x[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  return x[0];
}

// Sums (reference, sum) as one, at the larger reference.
__device__ __forceinline__ float2 joined(float2 a, float2 b) {
  if (b.x == a.x) return make_float2(a.x, a.y + b.y);
  if (b.x > a.x) return make_float2(b.x, a.y * exp2f(a.x - b.x) + b.y);
  return make_float2(a.x, a.y + b.y * exp2f(b.x - a.x));
}

// The issuing thread's part of a group: k-blocks [k0, k0 + len) of each product of pieces, W K-major or MN-major.
template <int NT, bool MN>
__device__ __forceinline__ void few_products(FewBars<NT>* bars, volatile int* abort, uint32_t tmem, uint32_t ring, int k0, int len, int passes,
                                             int64_t depth, int* stage, uint32_t* ring_phase, int* acc, uint32_t* acc_phase, bool* fine) {
  using T = Few<NT>;
  uint32_t d = 0, more = 0;
  auto begin = [&]() {
    *fine = *fine && wait<false>(smem_addr(&bars->acc_empty[*acc]), *acc_phase ^ 1u, abort);
    fence_after();
    d = tmem + static_cast<uint32_t>(*acc * NT);
    more = 0;
  };
  auto finish = [&]() {
    commit<false>(smem_addr(&bars->acc_full[*acc]));
    *acc ^= 1;
    if (*acc == 0) *acc_phase ^= 1u;
  };
  begin();
  for (int kb = 0, at = k0; *fine && kb < len * passes; ++kb) {
    if (!wait<false>(smem_addr(&bars->full[*stage]), *ring_phase, abort)) {
      *fine = false;
      break;
    }
    fence_after();
    const uint32_t sw = ring + *stage * (T::kWBytes + T::kHBytes);
    const uint64_t dw = operand_desc(sw, MN), dh = operand_desc(sw + T::kWBytes, false);
    const int64_t left = depth - static_cast<int64_t>(at) * kBK;
    const int cut = passes > 1 && kb >= len * (passes - 1) ? cut_of(!MN, passes) : 0;
    if (++at == k0 + len) at = k0;
#pragma unroll
    for (int k = 0; k < kBK / 16; ++k) {
      if (k * 16 >= left) break;
      if (cut && (k & (cut - 1)) == 0) {
        finish();
        begin();
      }
      if (!*fine) break;
      mma_f16<false>(d, MN ? dw + k * (2048 >> 4) : dw + (k / 4) * (T::kWBytes / 2 >> 4) + (k % 4) * 2,
                     dh + (k / 4) * (T::kHBytes / 2 >> 4) + (k % 4) * 2, T::kIdesc | (MN ? 1u << 15 : 0u), more);
      more = 1;
    }
    if (!*fine) break;
    commit<false>(smem_addr(&bars->empty[*stage]));
    if (++*stage == T::kStages) {
      *stage = 0;
      *ring_phase ^= 1u;
    }
  }
  if (*fine) finish();
}

// A warp's segment of 32 rows of W (a lane each) and 32 rows of h from c0 on, with the logits in r: keeps listed tokens' logits
// and (keep) the segment's part of U, and gives lane k the reference and sum of row c0 + k (without its target, which lane
// `skip` of the warp has, if any). z is the warp's shared memory.
__device__ __forceinline__ float2 segment_sum(const VocabArgs& g, bool keep, const uint32_t (&r)[32], float (*z)[33], const float* s_c, int c0,
                                              int64_t v0, int e, int end, int skip) {
  const int lane = threadIdx.x & 31, row = c0 + lane;
  const bool in = v0 + lane < g.V;
  auto s_u = reinterpret_cast<uint16_t(*)[40]>(&z[0][0]);  // rows of 80 bytes
  const float c = s_c[row];
  const bool alive = c != INFINITY;
  if (__any_sync(0xffffffffu, e < end)) {  // each lane looks its row's tokens up in what the others have
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 32; ++k) z[k][lane] = __uint_as_float(r[k]);
    __syncwarp();
    for (const int64_t row_at = static_cast<int64_t>(row) * g.K; e < end; ++e) {
      const int64_t from_v0 = g.sorted[row_at + e] - v0;
      if (from_v0 >= 0 && from_v0 < 32) g.zk[row_at + e] = z[lane][from_v0];
    }
    __syncwarp();
  }
  uint32_t terms = in ? 0xffffffffu : 0;   // rows of h in whose sums this lane's row of W is
  if (__any_sync(0xffffffffu, skip >= 0)) {
#pragma unroll
    for (int k = 0; k < 32; ++k) terms &= __shfl_sync(0xffffffffu, skip, k) == lane ? ~(1u << k) : 0xffffffffu;
  }
  float ref = c, sum;
#pragma unroll 1
  for (int again = 0; again < 2; ++again) {
    float x[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float to = again ? __shfl_sync(0xffffffffu, ref, k) : s_c[c0 + k];
      x[k] = terms >> k & 1 ? exp2_fast(fmaf(__uint_as_float(r[k]), g.k2, -to)) : 0.f;
    }
    if (keep) {
      for (int p = 0; p < g.np_u; ++p) {
        float y[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = x[k];
        for (int q = 0; q < p; ++q)
#pragma unroll
          for (int k = 0; k < 32; ++k) take_piece(y[k]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 32; ++k) s_u[k][lane] = s_c[c0 + k] == INFINITY ? 0 : take_piece(y[k]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int to = k * 8 + lane / 4;
          if (c0 + to < g.rows)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(g.U) + (static_cast<int64_t>(p) * g.Nc + c0 + to) * g.Vp + v0 +
                                      lane % 4 * 8) = *reinterpret_cast<const uint4*>(&s_u[to][lane % 4 * 8]);
        }
      }
    }
    sum = reduce_columns(x, [](float a, float b) { return a + b; });
    const bool over = !again && alive && !(sum <= kSumLimit);
    if (!__any_sync(0xffffffffu, over)) break;  // else: logits far above the targets', the segment's largest for a reference
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = in ? __uint_as_float(r[k]) * g.k2 : -INFINITY;
    const float top = reduce_columns(x, [](float a, float b) { return fmaxf(a, b); });
    if (over) ref = top == -INFINITY ? 0.f : top;
  }
  return make_float2(ref, sum);
}

template <int NT, bool KEEP>
__global__ void __launch_bounds__(Few<NT>::kThreads, 1)
    vocab_few_kernel(const __grid_constant__ VocabMaps maps, const __grid_constant__ VocabArgs g) {
  using T = Few<NT>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t s_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  __shared__ FewBars<NT> bars_s;
  __shared__ float s_c[NT];
  __shared__ float2 s_all[4][KEEP ? 1 : NT];
  __shared__ __align__(16) float s_z[4][32][33];
  FewBars<NT>* bars = &bars_s;
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      bar_init(smem_addr(&bars->full[s]), 1);
      bar_init(smem_addr(&bars->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(smem_addr(&bars->acc_full[s]), 1);
      bar_init(smem_addr(&bars->acc_empty[s]), 4);
    }
    bar_init(smem_addr(&bars->done), 1);
    bars->abort = 0;
    bar_init_fence();
    fence_async_smem();
  }
  if (warp == 1) tmem_alloc<false>(smem_addr(&bars->tmem), 2 * NT);
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x < NT) s_c[threadIdx.x] = threadIdx.x < g.rows ? g.c[threadIdx.x] : INFINITY;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars->tmem;

  const int tiles = static_cast<int>((g.V + 127) / 128), blocks = (g.d + kBK - 1) / kBK, passes = passes_of(g.np_w, g.np_h);
  int stage = 0, acc = 0;
  uint32_t ring_phase = 0, acc_phase = 0;
  bool fine = true;
  if (warp == 0) {
    if (lane == 0) {
      for (int t = blockIdx.x; fine && t < tiles; t += gridDim.x)
        for (int k0 = 0; fine && k0 < blocks; k0 += g.group)
          for (int pass = 0; fine && pass < passes; ++pass) {
            int zw = 0, zh = 0;
            if (passes > 1) piece_of(g.np_w, g.np_h, pass, &zw, &zh);
            for (int kb = k0; kb < min(k0 + g.group, blocks); ++kb) {
              if (!wait<false>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u, abort)) {
                fine = false;
                break;
              }
              const uint32_t full = smem_addr(&bars->full[stage]), dw = smem_addr(ring + stage * (T::kWBytes + T::kHBytes));
              bar_expect(full, T::kWBytes + T::kHBytes);
              load_operand<false, 128>(dw, &maps.W, &maps.W, false, t * 128, kb * kBK, zw, full);
              load_operand<false, NT>(dw + T::kWBytes, &maps.h, &maps.h, false, 0, kb * kBK, zh, full);
              if (++stage == S) {
                stage = 0;
                ring_phase ^= 1u;
              }
            }
          }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      for (int t = blockIdx.x; fine && t < tiles; t += gridDim.x)
        for (int k0 = 0; fine && k0 < blocks; k0 += g.group) {
          const int len = min(g.group, blocks - k0);
          few_products<NT, false>(bars, abort, tmem, smem_addr(ring), k0, len, passes, g.d, &stage, &ring_phase, &acc, &acc_phase, &fine);
        }
    }
  } else {
    const int quarter = warp & 3;
    if (!KEEP) {  // one sum a warp, in a segment of its own
      for (int k = lane; k < NT; k += 32) s_all[warp - 2][k] = make_float2(s_c[k], 0.f);
      __syncwarp();
    }
    for (int t = blockIdx.x; fine && t < tiles; t += gridDim.x) {
      const int64_t v0 = t * 128ll + quarter * 32;
      const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      auto acquire = [&]() {
        fine = __all_sync(0xffffffffu, wait_inline<false>(smem_addr(&bars->acc_full[acc]), acc_phase, abort));
        fence_after();
        return fine;
      };
      auto release = [&]() {
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars->acc_empty[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      };
      const int sums = sums_of(0, blocks, g.group, passes, g.d, cut_of(true, passes));
      if (sums > 1) {  // as in the other products: in registers, and back to TMEM with the last
        float z[NT];
#pragma unroll
        for (int k = 0; k < NT; ++k) z[k] = 0.f;
        for (int n = 1; n <= sums; ++n) {
          if (!acquire()) break;
          const bool last = n == sums;
#pragma unroll
          for (int c = 0; c < NT; c += 32) {
            uint32_t r[32];
            tmem_load(from + static_cast<uint32_t>(acc * NT + c), r);
            tmem_wait(r);
#pragma unroll
            for (int k = 0; k < 32; ++k) z[c + k] += __uint_as_float(r[k]);
            if (last) tmem_store(from + static_cast<uint32_t>(acc * NT + c), z + c);
          }
          if (last) tmem_stored();
          else release();
        }
        if (!fine) break;
      } else if (!acquire()) {
        break;
      }
      const int64_t seg = v0 >> 5;
      // 32 rows of h at a time. (Unrolled over all of them the code ran out of the instruction cache: 64 x 50,304 x 768 with
      // U 92 us.)
#pragma unroll 1
      for (int c0 = 0; c0 < g.rows && v0 < g.V; c0 += 32) {
        uint32_t r[32];
        tmem_load(from + static_cast<uint32_t>(acc * NT + c0), r);
        const int row = c0 + lane;  // the row of h whose sum this lane gets
        int e = 0, end = 0, skip = -1;
        if (g.ids && row < g.rows) {
          e = g.at[static_cast<int64_t>(t) * g.Nc + row];  // (the four warps' tokens)
          end = g.at[(t + 1ll) * g.Nc + row];
        }
        if (!g.ids && row < g.rows) skip = place_in(g.listed[row], v0, 32);
        __syncwarp();  // (TMEM's loads and waits want all lanes at once)
        tmem_wait(r);
        const float2 got = segment_sum(g, KEEP, r, s_z[warp - 2], s_c, c0, v0, e, end, skip);
        if (KEEP) {
          if (row < g.rows) g.sums[seg * g.Nc + row] = got;
        } else {
          s_all[warp - 2][row] = joined(s_all[warp - 2][row], got);
        }
        __syncwarp();
      }
      release();
    }
    if (!KEEP)
      for (int k = lane; k < g.rows; k += 32) g.sums[(blockIdx.x * 4ll + quarter) * g.Nc + k] = s_all[warp - 2][k];
  }
  if (!fine) {
    atomicOr(g.err_word, kErrVocab);
    *abort = 1;
  }
  __syncwarp();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      const uint64_t t0 = now_ns();
      while (!poll<false>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u) && now_ns() - t0 < kAsyncWaitNs / 8) {
      }
      if (++stage == S) {
        stage = 0;
        ring_phase ^= 1u;
      }
    }
  }
  if (warp == 1 && lane == 0) {
    commit_here<false>(smem_addr(&bars->done));
    const uint64_t t0 = now_ns();
    while (!poll<false>(smem_addr(&bars->done), 0) && now_ns() - t0 < kAsyncWaitNs) {
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 1) tmem_free<false>(tmem, 2 * NT);
}

// dh's parts for few rows, where reading W is all that counts again: the columns of W are the tile's rows (128 a CTA), the
// rows of U its columns, and the products run along a part of V; the parts are joined as the others are.
template <int NT>
__global__ void __launch_bounds__(Few<NT>::kThreads, 1)
    vocab_few_grad_kernel(const __grid_constant__ VocabMaps maps, const __grid_constant__ VocabArgs g) {
  using T = Few<NT>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t s_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  __shared__ FewBars<NT> bars_s;
  FewBars<NT>* bars = &bars_s;
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      bar_init(smem_addr(&bars->full[s]), 1);
      bar_init(smem_addr(&bars->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(smem_addr(&bars->acc_full[s]), 1);
      bar_init(smem_addr(&bars->acc_empty[s]), 4);
    }
    bar_init(smem_addr(&bars->done), 1);
    bars->abort = 0;
    bar_init_fence();
    fence_async_smem();
  }
  if (warp == 1) tmem_alloc<false>(smem_addr(&bars->tmem), 2 * NT);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars->tmem;
  grid_dep_wait();
  grid_dep_launch();

  const int tiles = (g.d + 127) / 128, all = static_cast<int>((g.V + kBK - 1) / kBK), units = tiles * g.q;
  const int np_u = g.gh_dtype == PG_F32 ? g.np_u : 1, np_w = g.gh_dtype == PG_F32 ? g.np_w : 1;
  auto first_block = [&](int part) { return static_cast<int>(static_cast<int64_t>(all) * part / g.q); };
  int stage = 0, acc = 0;
  uint32_t ring_phase = 0, acc_phase = 0;
  bool fine = true;
  if (warp == 0) {
    if (lane == 0) {
      for (int u = blockIdx.x; fine && u < units; u += gridDim.x) {
        const int part = u / tiles, col0 = (u - part * tiles) * 128, kb1 = first_block(part + 1);
        for (int k0 = first_block(part); fine && k0 < kb1;) {
          const int k1 = kb1 - k0 > g.group_h ? k0 + g.group_h : kb1;
          for (int pass = 0; fine && pass < g.passes_h; ++pass) {
            int zw = 0, zu = 0;
            if (g.passes_h > 1) piece_of(np_w, np_u, pass, &zw, &zu);
            for (int kb = k0; kb < k1; ++kb) {
              if (!wait<false>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u, abort)) {
                fine = false;
                break;
              }
              const uint32_t full = smem_addr(&bars->full[stage]), dw = smem_addr(ring + stage * (T::kWBytes + T::kHBytes));
              bar_expect(full, T::kWBytes + T::kHBytes);
              load_operand<false, 128>(dw, &maps.W, &maps.W, true, col0, kb * kBK, zw, full);
              load_operand<false, NT>(dw + T::kWBytes, &maps.Ufew, &maps.Ufew, false, 0, kb * kBK, zu, full);
              if (++stage == S) {
                stage = 0;
                ring_phase ^= 1u;
              }
            }
          }
          k0 = k1;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      for (int u = blockIdx.x; fine && u < units; u += gridDim.x) {
        const int part = u / tiles, kb1 = first_block(part + 1);
        for (int k0 = first_block(part); fine && k0 < kb1;) {
          const int k1 = kb1 - k0 > g.group_h ? k0 + g.group_h : kb1;
          few_products<NT, true>(bars, abort, tmem, smem_addr(ring), k0, k1 - k0, g.passes_h, g.V, &stage, &ring_phase, &acc, &acc_phase, &fine);
          k0 = k1;
        }
      }
    }
  } else {
    const int quarter = warp & 3;
    for (int u = blockIdx.x; fine && u < units; u += gridDim.x) {
      const int part = u / tiles, col = (u - part * tiles) * 128 + quarter * 32 + lane, kb1 = first_block(part + 1);
      float z[NT];
#pragma unroll
      for (int k = 0; k < NT; ++k) z[k] = 0.f;
      for (int n = sums_of(first_block(part), kb1, g.group_h, g.passes_h, g.V, cut_of(false, g.passes_h)); n; --n) {
        if (!__all_sync(0xffffffffu, wait_inline<false>(smem_addr(&bars->acc_full[acc]), acc_phase, abort))) {
          fine = false;
          break;
        }
        fence_after();
#pragma unroll
        for (int c = 0; c < NT; c += 32) {
          uint32_t r[32];
          tmem_load(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * NT + c), r);
          tmem_wait(r);
#pragma unroll
          for (int k = 0; k < 32; ++k) z[c + k] += __uint_as_float(r[k]);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&bars->acc_empty[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!fine) break;
      float* to = g.parts + static_cast<int64_t>(part) * g.Nc * g.d + col;
#pragma unroll
      for (int k = 0; k < NT; ++k)
        if (k < g.rows && col < g.d) to[static_cast<int64_t>(k) * g.d] = z[k];
    }
  }
  if (!fine) {
    atomicOr(g.err_word, kErrVocab);
    *abort = 1;
  }
  __syncwarp();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      const uint64_t t0 = now_ns();
      while (!poll<false>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u) && now_ns() - t0 < kAsyncWaitNs / 8) {
      }
      if (++stage == S) {
        stage = 0;
        ring_phase ^= 1u;
      }
    }
  }
  if (warp == 1 && lane == 0) {
    commit_here<false>(smem_addr(&bars->done));
    const uint64_t t0 = now_ns();
    while (!poll<false>(smem_addr(&bars->done), 0) && now_ns() - t0 < kAsyncWaitNs) {
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 1) tmem_free<false>(tmem, 2 * NT);
}

// ------------------------------------------------------------- rows so few that fp32 additions keep up with W

// A lane's four of 128 columns of a row from c0 on, zeros behind its end: neighbours, or (not VEC) 32 apart, so that a warp's
// loads are lines either way. W's do not stay in the L1 cache, which h has to itself.
template <bool VEC>
__device__ __forceinline__ int column_of(int k) {
  const int lane = threadIdx.x & 31;
  return VEC ? lane * 4 + k : lane + 32 * k;
}

template <bool VEC>
__device__ __forceinline__ float4 four_of(const float* row, int c0, int d) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const int c = c0 + column_of<VEC>(0);
  if (VEC) {
    if (c < d)
      asm("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(row + c));
  } else {
    if (c < d) v.x = __ldg(row + c);
    if (c + 32 < d) v.y = __ldg(row + c + 32);
    if (c + 64 < d) v.z = __ldg(row + c + 64);
    if (c + 96 < d) v.w = __ldg(row + c + 96);
  }
  return v;
}

template <int HT, bool VEC>
__device__ __forceinline__ float4 four_of_h(const VocabArgs& g, int row, int c0) {
  const int c = c0 + column_of<VEC>(0);
  const int64_t at = static_cast<int64_t>(row) * g.d + c;
  if (VEC && c >= g.d) return make_float4(0.f, 0.f, 0.f, 0.f);
  if (VEC && HT == PG_F32) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(g.h) + at));
  float x[4] = {};
  if (VEC) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(g.h) + at));
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y[1] = {0.f};
      if (c + 32 * k < g.d) load_cols<HT, 1>(g.h, at + 32 * k, y);
      x[k] = y[0];
    }
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}

// The first product of an fp32 W with up to 8 rows of h, in fp32 FMAs: W is read once, as it is, and no pieces of it are made.
// A warp has a segment of 32 rows of W, four of them at a time, its lanes along d (both halves of a packed FMA along d, too);
// h comes from the L1 cache. Bound by the loads under way (two blocks an SM leave 128 registers a thread, of which the fp32 kernel
// spills 368 bytes): 8 x 128,000 x 2560 347 us, 3.8 TB/s, the call 355-362 (in pieces 1130, of which 477 make them and 640 the six
// products, whose sums in TMEM follow one another), 8 x 10,000 x 768 39 us (49). Sixteen rows, two of
// W at a time, take longer than pieces unless W is far larger than L2 (16 x 10,000 x 768 76 us and 49).
template <int HT, bool VEC>
__global__ void __launch_bounds__(kSmallThreads, 2) vocab_small_kernel(const __grid_constant__ VocabArgs g, int keep) {
  constexpr int NB = kSmallRows, R = 32 / NB, kWarps = kSmallThreads / 32;
  __shared__ float s_c[32];
  __shared__ __align__(16) float s_z[kWarps][32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x < 32) s_c[threadIdx.x] = threadIdx.x < g.rows ? g.c[threadIdx.x] : INFINITY;
  __syncthreads();
  const int segs = static_cast<int>((g.V + 31) / 32);
  const float* W = static_cast<const float*>(g.W);
  float(*z)[33] = s_z[warp];
  for (int seg = warp * gridDim.x + blockIdx.x; seg < segs; seg += gridDim.x * kWarps) {
    const int64_t v0 = seg * 32ll;
#pragma unroll 1
    for (int i = 0; i < NB; ++i) {  // (rows past V are read as the last one, and left out by the sums)
      const float* rows[R];
#pragma unroll
      for (int k = 0; k < R; ++k) rows[k] = W + min(v0 + i * R + k, g.V - 1) * g.d;
      uint64_t sum[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) sum[k] = 0;
      float4 w[R], next[R];
#pragma unroll
      for (int k = 0; k < R; ++k) w[k] = four_of<VEC>(rows[k], 0, g.d);
#pragma unroll 2
      for (int c = 0; c < g.d; c += 128) {
#pragma unroll
        for (int k = 0; k < R; ++k) next[k] = four_of<VEC>(rows[k], c + 128, g.d);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const float4 x = four_of_h<HT, VEC>(g, min(n, g.rows - 1), c);
#pragma unroll
          for (int k = 0; k < R; ++k) {
            sum[k * NB + n] = fma2(pk(w[k].x, w[k].y), pk(x.x, x.y), sum[k * NB + n]);
            sum[k * NB + n] = fma2(pk(w[k].z, w[k].w), pk(x.z, x.w), sum[k * NB + n]);
          }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) w[k] = next[k];
      }
      float x[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        float lo, hi;
        upk(sum[k], lo, hi);
        x[k] = lo + hi;
      }
      __syncwarp();
      z[lane % NB][i * R + lane / NB] = reduce_columns(x, [](float a, float b) { return a + b; });
    }
    __syncwarp();
    uint32_t r[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = k < NB ? __float_as_uint(z[k][lane]) : 0u;
    __syncwarp();
    int e = 0, end = 0, skip = -1;
    if (g.ids && lane < g.rows) {
      e = g.at[(v0 >> g.at_log) * g.Nc + lane];
      end = g.at[((v0 >> g.at_log) + 1) * g.Nc + lane];
    }
    if (!g.ids && lane < g.rows) skip = place_in(g.listed[lane], v0, 32);
    const float2 got = segment_sum(g, keep, r, z, s_c, 0, v0, e, end, skip);
    if (lane < g.rows) g.sums[static_cast<int64_t>(seg) * g.Nc + lane] = got;
    __syncwarp();
  }
}

// dh's parts likewise: a warp has 128 columns of W (four a lane) and every eighth 32 rows of the part, with their U in its shared
// memory; the block's warps add up in turn. 8 x 128,000 x 2560 347 us (pieces 620).
template <bool VEC>
__global__ void __launch_bounds__(kSmallThreads, 2) vocab_small_grad_kernel(const __grid_constant__ VocabArgs g) {
  constexpr int NB = kSmallRows, kWarps = kSmallThreads / 32, kFly = 8;
  __shared__ __align__(16) float s_u[kWarps][32][NB];
  __shared__ __align__(16) float s_sum[NB][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  const int tiles = (g.d + 127) / 128, part = blockIdx.x / tiles, first = (blockIdx.x - part * tiles) * 128;
  const int64_t all = (g.V + kBK - 1) / kBK, begin = all * part / g.q * kBK, end = min(all * (part + 1) / g.q * kBK, g.V);
  const int np_u = g.gh_dtype == PG_F32 ? g.np_u : 1;
  const float* W = static_cast<const float*>(g.W);
  uint64_t sum[NB][2];
#pragma unroll
  for (int n = 0; n < NB; ++n) sum[n][0] = sum[n][1] = 0;
  for (int64_t v0 = begin + warp * 32; v0 < end; v0 += kWarps * 32) {
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float u = 0.f;
      if (n < g.rows && v0 + lane < end)
        for (int p = 0; p < np_u; ++p) u += __bfloat162float(g.U[(static_cast<int64_t>(p) * g.Nc + n) * g.Vp + v0 + lane]);
      s_u[warp][lane][n] = u;
    }
    __syncwarp();
#pragma unroll 1
    for (int k0 = 0; k0 < 32 && v0 + k0 < end; k0 += kFly) {
      float4 w[kFly];
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        w[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (v0 + k0 + k < end) w[k] = four_of<VEC>(W + (v0 + k0 + k) * g.d, first, g.d);
      }
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
#pragma unroll
        for (int n = 0; n < NB; n += 4) {
          const float4 u = *reinterpret_cast<const float4*>(&s_u[warp][k0 + k][n]);
          const float* each = &u.x;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            sum[n + m][0] = fma2(pk(w[k].x, w[k].y), pk(each[m], each[m]), sum[n + m][0]);
            sum[n + m][1] = fma2(pk(w[k].z, w[k].w), pk(each[m], each[m]), sum[n + m][1]);
          }
        }
      }
    }
  }
  for (int turn = 0; turn < kWarps; ++turn) {
    if (turn == warp) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float v[4];
        upk(sum[n][0], v[0], v[1]);
        upk(sum[n][1], v[2], v[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) s_sum[n][column_of<VEC>(k)] = turn ? s_sum[n][column_of<VEC>(k)] + v[k] : v[k];
      }
    }
    __syncthreads();
  }
  float* to = g.parts + static_cast<int64_t>(part) * g.Nc * g.d;
  for (int k = threadIdx.x; k < g.rows * 128; k += kSmallThreads)
    if (first + k % 128 < g.d) to[static_cast<int64_t>(k / 128) * g.d + first + k % 128] = s_sum[k / 128][k % 128];
}

// ------------------------------------------------------------------- rows, once their sums are there

constexpr int kRowWarps = 16, kRowsPer = 8;

// 8 rows a block: their sums over all tiles (four lanes of each of 16 warps share a row's; joined in a fixed order), lse
// and loss; for the gradients f, the targets' places of U, and f h (two warps a row).
template <bool GRAD, int HT, bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps) vocab_rows_kernel(const __grid_constant__ VocabArgs g) {
  __shared__ float2 s_all[kRowWarps][kRowsPer];
  __shared__ int s_moved[kRowWarps][kRowsPer], s_fix[kRowsPer];
  __shared__ float s_ref[kRowsPer], s_f[kRowsPer], s_peak[kRowsPer], s_place[kRowsPer], s_a[kRowsPer];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = lane & (kRowsPer - 1);
  const int r0 = blockIdx.x * kRowsPer, r = r0 + k;
  const bool in = r < g.rows;
  grid_dep_wait();
  grid_dep_launch();
  const float c = in ? g.c[r] : INFINITY, target_z = in && !g.ids ? g.zk[r] : 0.f;
  float2 all = make_float2(c, 0.f);
  int moved = 0;
  if (in && c != INFINITY) {
    const float2* at = g.sums + r;
    constexpr int kFly = 8, kStep = 4 * kRowWarps;
    for (int s = warp * 4 + lane / kRowsPer; s < g.segs; s += kFly * kStep) {
      float2 v[kFly];
#pragma unroll
      for (int j = 0; j < kFly; ++j) v[j] = at[static_cast<int64_t>(min(s + j * kStep, g.segs - 1)) * g.Nc];
#pragma unroll
      for (int j = 0; j < kFly; ++j) {
        if (s + j * kStep >= g.segs) break;
        moved |= v[j].x != c;
        all = joined(all, v[j]);
      }
    }
  }
#pragma unroll
  for (int o = kRowsPer; o < 32; o *= 2) {
    const float2 other = make_float2(__shfl_down_sync(0xffffffffu, all.x, o), __shfl_down_sync(0xffffffffu, all.y, o));
    moved |= __shfl_down_sync(0xffffffffu, moved, o);
    all = joined(all, other);
  }
  if (g.ids && warp < kRowsPer && r0 + warp < g.rows) {  // sum of w (log w - z + c) of row r0 + warp
    const int row = r0 + warp;
    const float c1 = __shfl_sync(0xffffffffu, c, warp);
    float a = 0.f;
    for (int e = lane; c1 != INFINITY && e < g.K; e += 32) {
      const float w = g.wk[static_cast<int64_t>(row) * g.K + e];
      if (w != -1.f && w != 0.f) a += w * fmaf(g.zk[static_cast<int64_t>(row) * g.K + e], g.k2, -c1);
    }
    a = g.a[row] - warp_sum(a) * kLn2;
    if (lane == 0) s_a[warp] = a;
  }
  if (lane < kRowsPer) {
    s_all[warp][k] = all;
    s_moved[warp][k] = moved;
  }
  __syncthreads();
  if (threadIdx.x < kRowsPer && in) {
    for (int w = 1; w < kRowWarps; ++w) {
      all = joined(all, s_all[w][k]);
      moved |= s_moved[w][k];
    }
    const bool alive = c != INFINITY, target = alive && !g.ids;
    // What follows is relative to the row's reference: of lse itself only 2^-24 is known, of exp(lse - reference) 2^-24 too.
    // Cross entropy: the target's own term, beside the sum of the others
    const float d = target ? fmaf(target_z, g.k2, -all.x) : 0.f;
    float own = target ? exp2f(d) : 0.f, sum = all.y + own;
    const float lse = (all.x + log2f(sum)) * kLn2;
    const int64_t i = g.row0 + r;
    if (g.lse) g.lse[i] = alive ? lse : 0.f;
    if (g.loss) {
      const float loss = g.ids ? s_a[k] + (all.x - c + log2f(sum)) * kLn2 : all.y <= own ? log1pf(all.y / own) : (log2f(sum) - d) * kLn2;
      g.loss[i] = alive ? loss + g.zl * lse * lse : 0.f;
    }
    if (GRAD) {
      float weight = alive ? g.grad_scale * g.scale : 0.f;
      if (alive && g.row_weight) weight *= __ldg(g.row_weight + i);
      float more = 2.f * g.zl * lse, beta = 1.f + more;
      if (fabsf(beta) < 1e-6f) {  // (its part of U is divided by it)
        beta = copysignf(1e-6f, beta);
        more = beta - 1.f;
      }
      float to = all.x;
      if (weight != 0.f && fabsf(weight * beta) < sum * kLeastFactor) {  // (rounded or not, to is what U is brought to)
        to += log2f(sum);
        const float by = exp2f(all.x - to);
        own *= by, all.y *= by, sum *= by;
        moved |= to != all.x;
      }
      const float f = weight == 0.f ? 0.f : weight * beta / sum;
      g.f[r] = f;
      s_f[k] = f;
      s_ref[k] = to;
      s_peak[k] = sum / beta;                       // what a weight of 1 takes off U
      s_place[k] = fmaf(own, more, -all.y) / beta;  // own - sum / beta, of what p leaves over
      // a row without weight must not bring its infinities and NaN into dW; a row without a target is zero already
      s_fix[k] = !alive ? 3 : weight == 0.f && !(fabsf(lse) < INFINITY) ? 2 : moved;
    }
  }
  if (!GRAD) return;
  if (g.twice && threadIdx.x < kRowsPer && in && c != INFINITY) g.c[r] = s_ref[k];
  __syncthreads();
  const int mine = warp % kRowsPer, part = warp / kRowsPer, row = r0 + mine;
  constexpr int kLanes = 32 * (kRowWarps / kRowsPer);
  const bool some = row < g.rows;
  const int fix = some && !g.twice ? s_fix[mine] : 3;
  float f = some ? s_f[mine] : 0.f;
  if (g.twice && f != 0.f) f = 1.f;  // (U has it; rows without a gradient may still hold anything)
  const float to = some ? s_ref[mine] : 0.f;
  if (fix == 1 || fix == 2) {
    for (int64_t at = (part * 32 + lane) * 8; at < g.Vp; at += kLanes * 8) {
      const float by = fix == 2 ? 0.f : exp2f(0.5f * (g.sums[(at >> g.seg_log) * g.Nc + row].x - to));  // (its square may underflow)
      float x[8] = {};
      for (int p = 0; p < g.np_u; ++p) {
        float y[8];
        read_cols<PG_BF16, 8>(g.U, (static_cast<int64_t>(p) * g.Nc + row) * g.Vp + at, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += y[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fix == 2 || at + e >= g.V ? 0.f : x[e] * by * by;
      for (int p = 0; p < g.np_u; ++p)
        *reinterpret_cast<uint4*>(g.U + (static_cast<int64_t>(p) * g.Nc + row) * g.Vp + at) = take_pieces(x);
    }
  }
  __syncthreads();
  if (!some) return;
  if (s_fix[mine] < 2) {  // (a U that is made later gets these by vocab_targets_kernel)
    for (int e = part * 32 + lane; e < g.K; e += kLanes) {
      const int64_t at = static_cast<int64_t>(row) * g.K + e;
      const float w = g.wk[at];
      if (w == -1.f || w == 0.f) continue;
      float x = g.ids ? exp2_fast(fmaf(g.zk[at], g.k2, -to)) - w * s_peak[mine] : s_place[mine];
      if (g.twice) {
        g.zk[at] = s_f[mine] * x;
        continue;
      }
      for (int p = 0; p < g.np_u; ++p)
        reinterpret_cast<uint16_t*>(g.U)[(static_cast<int64_t>(p) * g.Nc + row) * g.Vp + g.listed[at]] = take_piece(x);
    }
  }
  if (!g.F) return;
  for (int col = (part * 32 + lane) * 8; col < g.dp; col += kLanes * 8) {
    float x[8] = {};
    if (VEC) {
      if (col < g.d) load_cols<HT, VEC ? 8 : 1>(g.h, (g.row0 + row) * g.d + col, reinterpret_cast<float(&)[VEC ? 8 : 1]>(x));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float y[1] = {0.f};
        if (col + e < g.d) load_cols<HT, 1>(g.h, (g.row0 + row) * g.d + col + e, y);
        x[e] = y[0];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f == 0.f ? 0.f : f * x[e];
    for (int p = 0; p < g.np_f; ++p)
      *reinterpret_cast<uint4*>(g.F + (static_cast<int64_t>(p) * g.Nc + row) * g.dp + col) = take_pieces(x);
  }
}

// The targets' places of a U that was made with f (vocab_rows_kernel has left them in zk): one warp a row.
__global__ void __launch_bounds__(256) vocab_targets_kernel(const __grid_constant__ VocabArgs g) {
  grid_dep_wait();
  grid_dep_launch();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= g.rows || g.f[r] == 0.f) return;
  for (int e = lane; e < g.K; e += 32) {
    const int64_t at = static_cast<int64_t>(r) * g.K + e;
    const float w = g.wk[at];
    if (w == -1.f || w == 0.f) continue;
    float x = g.zk[at];
    for (int p = 0; p < g.np_u; ++p)
      reinterpret_cast<uint16_t*>(g.U)[(static_cast<int64_t>(p) * g.Nc + r) * g.Vp + g.listed[at]] = take_piece(x);
  }
}

// A gradient from its parts, COLS columns a thread: dh (blocks below blocks_h), dW.
template <int COLS>
__global__ void __launch_bounds__(256) vocab_join_kernel(const __grid_constant__ VocabArgs g, int blocks_h) {
  grid_dep_wait();
  grid_dep_launch();
  const bool dh = static_cast<int>(blockIdx.x) < blocks_h;
  const int64_t rows = dh ? g.rows : g.V, part = (dh ? g.Nc : g.V) * g.d;
  const int64_t at = (static_cast<int64_t>(blockIdx.x - (dh ? 0 : blocks_h)) * 256 + threadIdx.x) * COLS;
  if (at >= rows * g.d) return;
  const float* from = (dh ? g.parts : g.parts_w) + at;
  const int q = dh ? g.q : g.q_w;
  float x[COLS] = {};
#pragma unroll 4
  for (int p = 0; p < q; ++p, from += part) {
    if constexpr (COLS == 4) {
      const float4 v = *reinterpret_cast<const float4*>(from);
      x[0] += v.x; x[1] += v.y; x[2] += v.z; x[3] += v.w;
    } else {
      x[0] += *from;
    }
  }
  void* dst = g.gh;
  int dtype = g.gh_dtype;
  int64_t to = at;
  if (dh) {
    const float f = g.twice ? 1.f : g.f[at / g.d];
#pragma unroll
    for (int e = 0; e < COLS; ++e) x[e] = f == 0.f ? 0.f : f * x[e];
    to += g.row0 * g.d;
  } else {
    const float* add32 = nullptr;
    const __nv_bfloat16* add16 = nullptr;
    table_target(g, &dst, &dtype, &add32, &add16);
#pragma unroll
    for (int e = 0; e < COLS; ++e) {
      if (add32) x[e] += add32[at + e];
      if (add16) x[e] += __bfloat162float(add16[at + e]);
    }
  }
  if constexpr (COLS == 4) {
    if (dtype == PG_F32) *reinterpret_cast<float4*>(static_cast<float*>(dst) + to) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dst) + to) = make_uint2(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]));
  } else {
    if (dtype == PG_F32) static_cast<float*>(dst)[to] = x[0];
    else static_cast<__nv_bfloat16*>(dst)[to] = __float2bfloat16_rn(x[0]);
  }
}

// ------------------------------------------------------------------------------ host side

struct Sizes {
  int64_t N, V;
  int d, K;
  int h_dtype, w_dtype, gh_dtype, gw_dtype;  // gradients: -1 where there is none
  bool grad, list;
};

// Whether an operand needs its own copy: pieces of fp32, or rows that TMA cannot step over.
bool needs_copy(int dtype, int d) { return dtype == PG_F32 || d % 8 != 0; }

// How units of the gradients' products fall on `units` pairs: those of dh first, `heavy` pairs with one more, then those of
// dW, of which the others take `delta` more.
void spread(VocabArgs* g, int units, double cost2, double cost3) {
  const int64_t n2 = static_cast<int64_t>(g->tiles2) * g->q, n3 = static_cast<int64_t>(g->tiles3) * g->q_w;
  g->heavy = static_cast<int>(n2 % units);
  g->light = units - g->heavy;
  g->delta = g->heavy ? static_cast<int>(std::min<int64_t>(static_cast<int64_t>(cost2 / cost3 + 0.5), n3 / g->light)) : 0;
}

// Parts of dh along V and of dW along the rows: as few as leave the pairs evenly busy. In the time of a k-block (0.65 us), a
// tile takes 4 more (its first loads, its last sums and stores), a part's sums a store and a load of its tile (4 MB a
// k-block), and their own launch 8. (Tiles of 128 or 64 columns of d for small problems: a k-block takes as long, 4096 x
// 50,304 x 768 604, 828 and 1367 us with 256, 128 and 64, and 512 x 1024 x 96 in fp32 76, 81 and 74.)
void plan_schedule(VocabArgs* g, int units, bool has_h, bool has_w) {
  const int nm = (g->Nc + kTile - 1) / kTile;
  const int64_t nv = (g->V + kTile - 1) / kTile, kv = (g->V + kBK - 1) / kBK, kn = (std::min(g->N, g->Nc) + kBK - 1) / kBK;
  g->nd = (g->d + kTile - 1) / kTile;
  g->tiles2 = has_h ? nm * g->nd : 0;
  g->tiles3 = has_w ? static_cast<int>(nv * g->nd) : 0;
  g->passes_h = g->gh_dtype == PG_F32 ? passes_of(g->np_u, g->np_w) : 1;
  g->passes_w = g->gw_dtype == PG_F32 ? passes_of(g->np_u, g->np_f) : 1;
  g->group_h = g->gh_dtype == PG_F32 ? kGroupPieces : 1 << 30;  // (a bf16 gradient's own rounding is far above)
  g->group_w = g->gw_dtype == PG_F32 ? kGroupPieces : 1 << 30;
  if (has_h && g->N <= kFewRows && g->V > kFewTable) {
    // few rows: dh by itself, in as many parts as fill the SMs once or twice (a table of a few k-blocks: with dW)
    const int tiles = (g->d + 127) / 128;
    double best = -1;
    for (int waves = 1; waves <= 2; ++waves) {
      const int q = static_cast<int>(std::min<int64_t>(std::max(1, 2 * units * waves / tiles), kv));
      const double full = static_cast<double>(q) * tiles / (2 * units * ((q * tiles + 2 * units - 1) / (2 * units)));
      if (full <= best + 0.04) continue;
      best = full;
      g->few_h = q;
    }
    g->tiles2 = 0;
    has_h = false;
  }
  double best = -1;
  int best_q = 1, best_qw = 1;
  for (int q = 1; q <= (has_h ? kMaxParts : 1) && (q == 1 || (kv >= 2 * q && static_cast<int64_t>(q) * g->tiles2 <= kPartTiles)); ++q)
    for (int qw = 1; qw <= (has_w ? kMaxParts : 1) && (qw == 1 || (kn >= 2 * qw && static_cast<int64_t>(qw) * g->tiles3 <= kPartTiles)); qw *= 2) {
      g->q = q;
      g->q_w = qw;
      const double cost2 = static_cast<double>((kv + q - 1) / q) * g->passes_h + 4, cost3 = static_cast<double>((kn + qw - 1) / qw) * g->passes_w + 4;
      spread(g, units, cost2, cost3);
      const int a = static_cast<int>(static_cast<int64_t>(g->tiles2) * q / units);
      const int64_t rest = static_cast<int64_t>(g->tiles3) * qw - static_cast<int64_t>(g->delta) * g->light;
      double t = std::max((a + (g->heavy ? 1 : 0)) * cost2, a * cost2 + g->delta * cost3) + static_cast<double>((rest + units - 1) / units) * cost3;
      if (q > 1) t += static_cast<double>(q) * nm * kTile * g->d * 8 / 4e6;
      if (qw > 1) t += static_cast<double>(qw) * g->V * g->d * 8 / 4e6;
      if (q > 1 || qw > 1) t += 8;
      if (best >= 0 && t >= best) continue;
      best = t;
      best_q = q;
      best_qw = qw;
    }
  g->q = g->few_h ? g->few_h : best_q;
  g->q_w = best_qw;
}

// Sizes of everything, and its place in the workspace (base null: the size alone). What is reserved never falls as the
// rows become more, though tiles and parts are then cut in other ways: a workspace for N rows serves any call of fewer.
size_t carve_vocab(uint8_t* base, const Sizes& s, VocabArgs* g) {
  uint8_t* first = base ? reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(base) + 127) & ~uintptr_t(127)) : nullptr;
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* ptr = first ? first + at : nullptr;
    at += static_cast<size_t>((bytes + 127) / 128 * 128);
    return ptr;
  };
  const bool has_h = s.gh_dtype >= 0, has_w = s.gw_dtype >= 0, is_few = s.N <= kFewRows;
  g->V = s.V;
  g->Vp = (s.V + 63) / 64 * 64;
  g->N = static_cast<int>(s.N);
  g->d = s.d;
  g->dp = (s.d + 63) / 64 * 64;
  g->K = s.K;
  g->h_dtype = s.h_dtype;
  g->w_dtype = s.w_dtype;
  g->gh_dtype = s.gh_dtype;
  g->gw_dtype = s.gw_dtype;
  g->np_h = s.h_dtype == PG_F32 ? 3 : 1;
  g->np_w = s.w_dtype == PG_F32 ? 3 : 1;
  g->np_u = s.gh_dtype == PG_F32 || s.gw_dtype == PG_F32 ? 3 : 1;
  // An fp32 dW of bf16 operands: f h has 24 bits, so U and f h take six products. With f in U, made from the logits a second
  // time, what is left of f h is h (without the rows that have no gradient): three products and one more of the logits
  // (3001 x 32,003 x 515 1025 -> 820 us, 8192 x 50,304 x 768 4.36 -> 3.58 ms).
  g->twice = s.grad && s.gw_dtype == PG_F32 && s.h_dtype == PG_BF16 && s.w_dtype == PG_BF16 && !is_few;
  const int np_f = s.gw_dtype == PG_F32 ? 3 : 1;
  g->np_f = g->twice ? 1 : np_f;
  g->small = s.N <= kSmallRows && s.w_dtype == PG_F32 && (!has_h || s.V > kFewTable);
  const int blocks = (s.d + kBK - 1) / kBK, longest = g->np_h * g->np_w > 1 || g->np_u > 1 ? kGroupPieces : kGroup;
  const int groups = (blocks + longest - 1) / longest;
  g->group = (blocks + groups - 1) / groups;
  // narrower tiles of the logits where the widest leave pairs idle
  g->wide = kTile;
  while (g->wide > 64 && (s.N + kTile - 1) / kTile * ((s.V + g->wide - 1) / g->wide) <= kPlanUnits / 2) g->wide /= 2;
  if (is_few) g->wide = 64;
  g->seg = g->wide / 2;
  g->seg_log = g->seg == 128 ? 7 : g->seg == 64 ? 6 : 5;
  g->at_log = is_few ? 7 : g->seg_log;
  const int64_t widest = (s.V + kTile - 1) / kTile;  // tiles a row of them
  const int64_t row_bytes = 2 * (g->np_u * g->Vp + (has_w ? np_f * g->dp : 0) + (needs_copy(s.h_dtype, s.d) ? g->np_h * g->dp : 0)) +
                            (s.list ? 12ll * s.K + 2 * (2 * widest + 1) : 0);  // lists: zk, wk, sorted, at
  int64_t most = std::min(s.grad ? kKeepBytes / row_bytes : kMaxForwardRows, kSumBytes / (16 * widest));
  most = std::max<int64_t>(kTile, most / kTile * kTile);
  const int64_t chunks = (s.N + most - 1) / most;
  const int unit = is_few ? kRowsPer : kTile;  // (few rows: those that are there, to the lists' blocks)
  g->Nc = static_cast<int>(((s.N + chunks - 1) / chunks + unit - 1) / unit * unit);
  const int64_t rows = std::min(most, (s.N + unit - 1) / unit * unit);  // room for these (Nc of them or more)
  g->Wp = needs_copy(s.w_dtype, s.d) && !g->small ? reinterpret_cast<__nv_bfloat16*>(take(2ll * g->np_w * s.V * g->dp)) : nullptr;
  g->hp = needs_copy(s.h_dtype, s.d) && !g->small ? reinterpret_cast<__nv_bfloat16*>(take(2ll * g->np_h * rows * g->dp)) : nullptr;
  // (narrower tiles are kPlanUnits at most, for a chunk of kTile rows; few rows have a sum for 32 columns, or four a CTA of 128)
  const int64_t sums_few = 2 * ((s.V + 127) / 128);
  g->sums = reinterpret_cast<float2*>(take(16 * (is_few ? std::max(sums_few * rows, int64_t{kTile})
                                                        : std::max({widest * rows, static_cast<int64_t>(kPlanUnits) * kTile, sums_few * kTile}))));
  g->zk = reinterpret_cast<float*>(take(4ll * rows * s.K));
  g->wk = reinterpret_cast<float*>(take(4ll * rows * s.K));
  g->sorted = s.list ? reinterpret_cast<int32_t*>(take(4ll * rows * s.K)) : nullptr;
  const int64_t places = (2 * widest + 1) * rows;
  g->at = s.list ? reinterpret_cast<uint16_t*>(take(2 * (is_few ? places : std::max(places, int64_t{3} * kPlanUnits * kTile)))) : nullptr;
  g->c = reinterpret_cast<float*>(take(4 * rows));
  g->a = reinterpret_cast<float*>(take(4 * rows));
  g->U = nullptr;
  g->F = nullptr;
  g->f = g->acc = g->parts = g->parts_w = nullptr;
  if (s.grad) {
    g->f = reinterpret_cast<float*>(take(4 * rows));
    g->U = reinterpret_cast<__nv_bfloat16*>(take(2ll * g->np_u * rows * g->Vp));
    if (has_w) {
      g->F = reinterpret_cast<__nv_bfloat16*>(take(2ll * np_f * rows * g->dp));
      if (chunks > 1 && s.gw_dtype == PG_BF16) g->acc = reinterpret_cast<float*>(take(4ll * s.V * s.d));
    }
    plan_schedule(g, kPlanUnits, has_h, has_w);
    const int64_t kv = (s.V + kBK - 1) / kBK, kn = (std::min(s.N, rows) + kBK - 1) / kBK;
    if (has_h) {  // parts of a chunk's rows, or as many as few rows have
      const int64_t some = std::min<int64_t>(kMaxParts * (is_few ? 1 : rows / kTile), kPartTiles / g->nd);
      const int64_t few = std::min<int64_t>(kv, std::max(1, 4 * kPlanUnits / ((s.d + 127) / 128)));
      float* to = reinterpret_cast<float*>(take(4ll * (is_few ? rows : kTile) * s.d * std::max({some, few, int64_t{1}})));
      if (g->q > 1 || g->few_h) g->parts = to;
    }
    const int64_t parts_w = std::min({int64_t{kMaxParts}, kn / 2, kPartTiles / (widest * g->nd)});
    if (has_w && parts_w > 1) {  // (one part goes where the gradient goes)
      float* to = reinterpret_cast<float*>(take(4ll * s.V * s.d * parts_w));
      if (g->q_w > 1) g->parts_w = to;
    }
  }
  return at + 128;
}

// [pieces, rows, cols] bf16 (or fp32) with row stride ld, in boxes of box_cols columns (as wide as the swizzle) and box_rows rows.
bool vocab_map(CUtensorMap* map, const void* ptr, int pieces, int64_t rows, int64_t cols, int64_t ld, int64_t piece_rows,
               int box_cols, int box_rows, CUtensorMapSwizzle swizzle, bool f32 = false) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(pieces)};
  const cuuint64_t size = f32 ? 4 : 2;
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * size, static_cast<cuuint64_t>(piece_rows) * ld * size};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// CTA pairs of the kernel that are resident at once on the current device.
template <int KIND, bool GROUPS>
pg_status vocab_units(int* units) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return PG_ERR_DEVICE;
  *units = known[dev].load(std::memory_order_relaxed);
  if (*units) return PG_OK;
  auto kern = vocab_product_kernel<KIND, GROUPS>;
  cudaFuncAttributes attrs;
  e = cudaFuncGetAttributes(&attrs, kern);
  if (e != cudaSuccess) return cuda_fail(e);
  if (GROUPS && attrs.numRegs < kLaunchRegs) return PG_ERR_UNSUPPORTED;  // its warpgroups share out this many
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return cuda_fail(e);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * static_cast<unsigned>(sm_count()));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
  if (e != cudaSuccess) return cuda_fail(e);
  if (n < 1) return PG_ERR_DEVICE;
  known[dev].store(n, std::memory_order_relaxed);
  *units = n;
  return PG_OK;
}

// A kernel that is scheduled while the one before it in the call still runs (early), of one CTA or pairs.
template <typename... Params, typename... Args>
pg_status launch_next(void (*kern)(Params...), int64_t blocks, int threads, size_t smem, bool pair, bool early, cudaStream_t stream,
                      const Args&... args) {
  if (blocks >= (1ll << 31)) return PG_ERR_SHAPE;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (early) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e == cudaSuccess ? after_launch(1) : cuda_fail(e);
}

template <int KIND, bool GROUPS>
pg_status launch_product(const VocabMaps& maps, const VocabArgs& g, int64_t jobs, cudaStream_t stream) {
  int units;
  pg_status st = vocab_units<KIND, GROUPS>(&units);
  if (st != PG_OK) return st;
  units = static_cast<int>(std::min<int64_t>(units, jobs));
  VocabArgs a = g;
  if (KIND == kGrads)  // the same parts on however many pairs there are
    spread(&a, units, static_cast<double>((a.V + kBK - 1) / kBK) / a.q * a.passes_h + 4,
           static_cast<double>((a.rows + kBK - 1) / kBK) / a.q_w * a.passes_w + 4);
  return launch_next(vocab_product_kernel<KIND, GROUPS>, 2ll * units, kThreads, kSmem, true, true, stream, maps, a);
}

// CTAs of the first product for few rows. (No more than its tiles: 4 sums a CTA fit in place of 4 a tile.)
int64_t few_blocks(int64_t V) { return std::min<int64_t>(sm_count(), (V + 127) / 128); }

template <int NT>
pg_status launch_few(const VocabMaps& maps, const VocabArgs& g, bool keep, cudaStream_t stream) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return PG_ERR_DEVICE;
  if (!known[dev].load(std::memory_order_relaxed)) {
    const int bytes = static_cast<int>(Few<NT>::kSmem);
    if ((e = cudaFuncSetAttribute(vocab_few_kernel<NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(vocab_few_kernel<NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess)
      return cuda_fail(e);
    known[dev].store(1, std::memory_order_relaxed);
  }
  return launch_next(keep ? vocab_few_kernel<NT, true> : vocab_few_kernel<NT, false>, few_blocks(g.V), Few<NT>::kThreads, Few<NT>::kSmem, false, true,
                     stream, maps, g);
}

template <int NT>
pg_status launch_few_grad(const VocabMaps& maps, const VocabArgs& g, cudaStream_t stream) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return PG_ERR_DEVICE;
  if (!known[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(vocab_few_grad_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Few<NT>::kSmem));
    if (e != cudaSuccess) return cuda_fail(e);
    known[dev].store(1, std::memory_order_relaxed);
  }
  const int64_t blocks = std::min<int64_t>(sm_count(), static_cast<int64_t>((g.d + 127) / 128) * g.q);
  return launch_next(vocab_few_grad_kernel<NT>, blocks, Few<NT>::kThreads, Few<NT>::kSmem, false, true, stream, maps, g);
}

// Two blocks an SM, as the kernel's registers allow, or as many as there are segments for.
template <int HT, bool VEC>
pg_status launch_small_of(const VocabArgs& g, bool keep, cudaStream_t stream) {
  const int64_t blocks = std::min<int64_t>(2 * sm_count(), (g.V + 31) / 32);
  return launch_next(vocab_small_kernel<HT, VEC>, blocks, kSmallThreads, 0, false, true, stream, g, static_cast<int>(keep));
}

pg_status launch_small(const VocabArgs& g, bool keep, bool vec, cudaStream_t stream) {
  if (g.h_dtype == PG_F32) return vec ? launch_small_of<PG_F32, true>(g, keep, stream) : launch_small_of<PG_F32, false>(g, keep, stream);
  return vec ? launch_small_of<PG_BF16, true>(g, keep, stream) : launch_small_of<PG_BF16, false>(g, keep, stream);
}

pg_status launch_small_grad(const VocabArgs& g, bool vec, cudaStream_t stream) {
  return launch_next(vec ? vocab_small_grad_kernel<true> : vocab_small_grad_kernel<false>, static_cast<int64_t>((g.d + 127) / 128) * g.q,
                     kSmallThreads, 0, false, true, stream, g);
}

using PrepareFn = void (*)(const VocabArgs, int, int);
using ArgsFn = void (*)(const VocabArgs);

template <int HT, int WT>
PrepareFn prepare_fn(bool list, bool vec) {
  if (list) return vec ? vocab_prepare_kernel<HT, WT, true, true> : vocab_prepare_kernel<HT, WT, false, true>;
  return vec ? vocab_prepare_kernel<HT, WT, true, false> : vocab_prepare_kernel<HT, WT, false, false>;
}

ArgsFn rows_fn(bool grad, int ht, bool vec) {
  if (!grad) return vocab_rows_kernel<false, PG_F32, false>;
  if (ht == PG_F32) return vec ? vocab_rows_kernel<true, PG_F32, true> : vocab_rows_kernel<true, PG_F32, false>;
  return vec ? vocab_rows_kernel<true, PG_BF16, true> : vocab_rows_kernel<true, PG_BF16, false>;
}

pg_status run_vocab(VocabArgs g, const Sizes& s, cudaStream_t stream) {
  pg_status st;
  const bool list = g.ids != nullptr;
  const bool vec_h = s.d % 8 == 0 && aligned(g.h, vec_bytes(s.h_dtype)), vec = vec_h && aligned(g.W, vec_bytes(s.w_dtype));
  const bool vec_four = s.d % 4 == 0 && aligned(g.W, 16) && aligned(g.h, 4 * dtype_bytes(s.h_dtype));
  const PrepareFn prepare = s.h_dtype == PG_F32
      ? (s.w_dtype == PG_F32 ? prepare_fn<PG_F32, PG_F32>(list, vec) : prepare_fn<PG_F32, PG_BF16>(list, vec))
      : (s.w_dtype == PG_F32 ? prepare_fn<PG_BF16, PG_F32>(list, vec) : prepare_fn<PG_BF16, PG_BF16>(list, vec));
  VocabMaps maps;
  const int64_t ldw = g.Wp ? g.dp : s.d, ldh = g.hp ? g.dp : s.d;
  if (!g.small && !vocab_map(&maps.W, g.Wp ? g.Wp : g.W, g.np_w, s.V, s.d, ldw, s.V, kLine, 128, CU_TENSOR_MAP_SWIZZLE_128B)) return PG_ERR_CUDA;
  const bool groups = sums_of(0, (s.d + kBK - 1) / kBK, g.group, passes_of(g.np_h, g.np_w), s.d, 2) > 1;
  auto split_blocks = [&](int64_t rows) { return (rows * (g.dp / 8) + kPrepThreads - 1) / kPrepThreads; };
  for (int64_t row0 = 0; row0 < s.N; row0 += g.Nc) {
    g.row0 = row0;
    g.rows = static_cast<int>(std::min<int64_t>(g.Nc, s.N - row0));
    g.listed = list ? g.sorted : g.targets + row0;
    g.first = row0 == 0;
    g.last = row0 + g.Nc >= s.N;
    const int64_t blocks_w = g.Wp && g.first ? split_blocks(s.V) : 0, blocks_h = g.hp ? split_blocks(g.rows) : 0;
    const int64_t blocks = blocks_w + blocks_h + (g.rows + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
    if (blocks >= (1ll << 31)) return PG_ERR_SHAPE;
    st = launch_next(prepare, blocks, kPrepThreads, 0, false, !g.first, stream, g, static_cast<int>(blocks_w), static_cast<int>(blocks_h));
    if (st != PG_OK) return st;
    const uint8_t* h = static_cast<const uint8_t*>(g.h) + row0 * s.d * static_cast<int64_t>(dtype_bytes(s.h_dtype));
    const int few = s.N > kFewRows ? 0 : s.N > 64 ? 128 : s.N > 32 ? 64 : 32;
    if (!g.small && !vocab_map(&maps.h, g.hp ? static_cast<const void*>(g.hp) : h, g.np_h, g.rows, s.d, ldh, g.rows, kLine, few ? few : 128,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return PG_ERR_CUDA;
    const int64_t jobs = static_cast<int64_t>((g.rows + kTile - 1) / kTile) * ((s.V + g.wide - 1) / g.wide);
    if (s.grad) {
      if (!vocab_map(&maps.U, g.U, g.np_u, g.rows, s.V, g.Vp, g.Nc, kLine, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
          !vocab_map(&maps.Ust, g.U, g.np_u, g.rows, s.V, g.Vp, g.Nc, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B) ||
          (g.F && !vocab_map(&maps.F, g.F, g.np_f, g.rows, s.d, g.dp, g.Nc, kLine, 128, CU_TENSOR_MAP_SWIZZLE_128B)))
        return PG_ERR_CUDA;
      if (!g.F) maps.F = maps.U;
      maps.Ufew = maps.Gh = maps.Gw = maps.U;
      if (g.small) maps.h = maps.W = maps.U;
      if (g.few_h && !g.small && !vocab_map(&maps.Ufew, g.U, g.np_u, g.rows, s.V, g.Vp, g.Nc, kLine, few, CU_TENSOR_MAP_SWIZZLE_128B)) return PG_ERR_CUDA;
      // tiles that nothing is added to, of matrices that TMA can step over
      auto out_map = [&](CUtensorMap* map, void* dst, int dtype, int64_t rows) {
        const bool f32 = dtype == PG_F32;
        if (s.d % (f32 ? 4 : 8) || !aligned(dst, 16)) return 0;
        return vocab_map(map, dst, 1, rows, s.d, s.d, rows, 32, 32, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, f32) ? 1 : -1;
      };
      const bool through = g.acc && !g.last;
      g.tma_w = s.gw_dtype >= 0 && !g.parts_w && g.first && !g.accumulate
                    ? out_map(&maps.Gw, through ? static_cast<void*>(g.acc) : g.gw, through ? PG_F32 : s.gw_dtype, s.V) : 0;
      g.tma_h = s.gh_dtype >= 0 && !g.parts
                    ? out_map(&maps.Gh, static_cast<uint8_t*>(g.gh) + row0 * s.d * static_cast<int64_t>(dtype_bytes(s.gh_dtype)), s.gh_dtype, g.rows) : 0;
      if (g.tma_w < 0 || g.tma_h < 0) return PG_ERR_CUDA;
    } else {
      maps.U = maps.Ust = maps.F = maps.Ufew = maps.Gh = maps.Gw = maps.h;  // (small: no map is looked at)
    }
    if (g.small)
      st = launch_small(g, s.grad, vec_four, stream);
    else if (few)
      st = few == 32 ? launch_few<32>(maps, g, s.grad, stream) : few == 64 ? launch_few<64>(maps, g, s.grad, stream)
                                                                             : launch_few<128>(maps, g, s.grad, stream);
    else if (s.grad && !g.twice)
      st = groups ? launch_product<kKeep, true>(maps, g, jobs, stream) : launch_product<kKeep, false>(maps, g, jobs, stream);
    else
      st = groups ? launch_product<kSums, true>(maps, g, jobs, stream) : launch_product<kSums, false>(maps, g, jobs, stream);
    if (st != PG_OK) return st;
    g.segs = few && !s.grad && !g.small ? static_cast<int>(4 * few_blocks(g.V)) : static_cast<int>((g.V + g.seg - 1) / g.seg);
    st = launch_next(rows_fn(s.grad, s.h_dtype, vec_h), (g.rows + kRowsPer - 1) / kRowsPer, 32 * kRowWarps, 0, false, true, stream, g);
    if (st != PG_OK) return st;
    if (g.twice) {
      st = groups ? launch_product<kAgain, true>(maps, g, jobs, stream) : launch_product<kAgain, false>(maps, g, jobs, stream);
      if (st != PG_OK) return st;
      if ((st = launch_next(vocab_targets_kernel, (g.rows + 7) / 8, 256, 0, false, true, stream, g)) != PG_OK) return st;
    }
    VocabArgs b = g;
    if (g.tiles2) b.tiles2 = (g.rows + kTile - 1) / kTile * g.nd;  // a last chunk has fewer rows
    b.q_w = std::min(g.q_w, (g.rows + kBK - 1) / kBK);             // (no part without a k-block)
    if (g.few_h && g.small) {
      if ((st = launch_small_grad(g, vec_four, stream)) != PG_OK) return st;
    } else if (g.few_h) {
      st = few == 32 ? launch_few_grad<32>(maps, g, stream) : few == 64 ? launch_few_grad<64>(maps, g, stream) : launch_few_grad<128>(maps, g, stream);
      if (st != PG_OK) return st;
    }
    const int64_t units = s.grad ? static_cast<int64_t>(b.tiles2) * b.q + static_cast<int64_t>(b.tiles3) * b.q_w : 0;
    if (!s.grad) continue;
    const bool pieces = s.gh_dtype == PG_F32 || s.gw_dtype == PG_F32;
    if (units && (st = pieces ? launch_product<kGrads, true>(maps, b, units, stream) : launch_product<kGrads, false>(maps, b, units, stream)) != PG_OK)
      return st;
    if (g.parts || g.parts_w) {
      const bool four = s.d % 4 == 0 && (!g.parts || aligned(g.gh, 4 * dtype_bytes(s.gh_dtype))) &&
                        (!g.parts_w || aligned(g.gw, 4 * dtype_bytes(s.gw_dtype)));
      auto join_blocks = [&](int64_t rows) { return (rows * s.d / (four ? 4 : 1) + 255) / 256; };
      const int64_t join_h = g.parts ? join_blocks(g.rows) : 0, join_w = g.parts_w ? join_blocks(s.V) : 0;
      if (join_h + join_w >= (1ll << 31)) return PG_ERR_SHAPE;
      st = launch_next(four ? vocab_join_kernel<4> : vocab_join_kernel<1>, join_h + join_w, 256, 0, false, true, stream, b, static_cast<int>(join_h));
      if (st != PG_OK) return st;
    }
  }
  return PG_OK;
}

pg_status check_sizes(const Sizes& s) {
  if (s.N < 0 || s.N >= (1ll << 31) || s.V < 1 || s.V > kMaxVocab || s.d < 1 || s.d > kMaxVocabWidth || s.K < 1 || s.K > kMaxList)
    return PG_ERR_SHAPE;
  if (!real_dtype(s.h_dtype) || !real_dtype(s.w_dtype)) return PG_ERR_DTYPE;
  if (s.grad && ((s.gh_dtype != -1 && !real_dtype(s.gh_dtype)) || (s.gw_dtype != -1 && !real_dtype(s.gw_dtype)))) return PG_ERR_DTYPE;
  return PG_OK;
}

pg_status vocab_workspace(const Sizes& s, size_t* bytes) {
  if (!bytes) return PG_ERR_NULL;
  pg_status st = check_sizes(s);
  if (st != PG_OK) return st;
  VocabArgs g = {};
  *bytes = s.N == 0 ? 0 : carve_vocab(nullptr, s, &g);
  return PG_OK;
}

// What the four calls share, behind their own checks.
struct Call {
  Sizes s;
  const void *h, *W;
  const int32_t* targets;
  const int32_t* ids;
  const void* tlogits;
  int t_dtype;
  const float* row_weight;
  float scale, inv_t, zl, grad_scale;
  int accumulate;
  float *loss, *lse;
  void *gh, *gw;
  void* workspace;
  size_t workspace_bytes;
  int32_t* err;
  cudaStream_t stream;
};

// An operand that TMA reads in place has to start on 16 bytes.
bool operand_aligned(const void* p, int dtype, int d) { return aligned(p, needs_copy(dtype, d) ? dtype_bytes(dtype) : 16); }

pg_status call_vocab(const Call& c) {
  size_t need;
  pg_status st = vocab_workspace(c.s, &need);
  if (st != PG_OK) return st;
  const bool list = c.s.list;
  if (list && !real_dtype(c.t_dtype)) return PG_ERR_DTYPE;
  if (!std::isfinite(c.scale) || !std::isfinite(c.zl) || !std::isfinite(c.grad_scale) || !std::isfinite(c.inv_t) || !(c.inv_t > 0.f) ||
      !std::isfinite(c.scale * c.inv_t * kLog2e))
    return PG_ERR_UNSUPPORTED;
  const bool has_w = c.s.grad && c.s.gw_dtype >= 0, has_h = c.s.grad && c.s.gh_dtype >= 0;
  if (c.s.N == 0 && !(has_w && !c.accumulate)) return PG_OK;
  if (has_w && !c.gw) return PG_ERR_NULL;
  if (has_w && !aligned(c.gw, dtype_bytes(c.s.gw_dtype))) return PG_ERR_ALIGN;
  if (c.s.N == 0) {
    if (device_cc() != 103) return PG_ERR_DEVICE;
    cudaError_t e = cudaMemsetAsync(c.gw, 0, static_cast<size_t>(c.s.V) * c.s.d * dtype_bytes(c.s.gw_dtype), c.stream);
    return e == cudaSuccess ? PG_OK : cuda_fail(e);
  }
  if (!c.h || !c.W || (list ? !c.ids || !c.tlogits : !c.targets) || (has_h && !c.gh) || (!c.s.grad && !c.loss)) return PG_ERR_NULL;
  if (!operand_aligned(c.h, c.s.h_dtype, c.s.d) || !operand_aligned(c.W, c.s.w_dtype, c.s.d) || !aligned(c.targets, 4) ||
      !aligned(c.ids, 4) || (list && !aligned(c.tlogits, dtype_bytes(c.t_dtype))) || !aligned(c.row_weight, 4) || !aligned(c.loss, 4) ||
      !aligned(c.lse, 4) || !aligned(c.err, 4) || (has_h && !aligned(c.gh, dtype_bytes(c.s.gh_dtype))) || !aligned(c.workspace, 16))
    return PG_ERR_ALIGN;
  if (!c.workspace || c.workspace_bytes < need) return PG_ERR_WORKSPACE;
  if (device_cc() != 103) return PG_ERR_DEVICE;
  if ((st = prepare_err(c.err, c.stream)) != PG_OK) return st;

  VocabArgs g = {};
  carve_vocab(static_cast<uint8_t*>(c.workspace), c.s, &g);
  g.h = c.h;
  g.W = c.W;
  g.targets = list ? nullptr : c.targets;
  g.ids = list ? c.ids : nullptr;
  g.tlogits = c.tlogits;
  g.t_dtype = c.t_dtype;
  g.row_weight = c.row_weight;
  g.loss = c.loss;
  g.lse = c.lse;
  g.err = c.err;
  g.gh = c.gh;
  g.gw = c.gw;
  g.err_word = device_error_word();
  g.accumulate = c.accumulate;
  g.scale = c.scale * c.inv_t;
  g.inv_t = c.inv_t;
  g.k2 = c.scale * c.inv_t * kLog2e;
  g.zl = c.zl;
  g.grad_scale = c.grad_scale;
  return run_vocab(g, c.s, c.stream);
}

}  // namespace
}  // namespace pg

using namespace pg;

extern "C" pg_status pg_vocab_ce_workspace_size(int64_t N, int64_t V, int32_t d, int32_t h_dtype, int32_t w_dtype, size_t* bytes) {
  return vocab_workspace({N, V, d, 1, h_dtype, w_dtype, -1, -1, false, false}, bytes);
}

extern "C" pg_status pg_vocab_ce_grad_workspace_size(int64_t N, int64_t V, int32_t d, int32_t h_dtype, int32_t w_dtype,
                                                     int32_t gh_dtype, int32_t gw_dtype, size_t* bytes) {
  return vocab_workspace({N, V, d, 1, h_dtype, w_dtype, gh_dtype, gw_dtype, true, false}, bytes);
}

extern "C" pg_status pg_vocab_distill_workspace_size(int64_t N, int64_t V, int32_t d, int32_t K, int32_t h_dtype, int32_t w_dtype,
                                                     size_t* bytes) {
  return vocab_workspace({N, V, d, K, h_dtype, w_dtype, -1, -1, false, true}, bytes);
}

extern "C" pg_status pg_vocab_distill_grad_workspace_size(int64_t N, int64_t V, int32_t d, int32_t K, int32_t h_dtype,
                                                          int32_t w_dtype, int32_t gh_dtype, int32_t gw_dtype, size_t* bytes) {
  return vocab_workspace({N, V, d, K, h_dtype, w_dtype, gh_dtype, gw_dtype, true, true}, bytes);
}

extern "C" pg_status pg_vocab_ce(const void* h, int32_t h_dtype, int64_t N, const void* W, int32_t w_dtype, int64_t V, int32_t d,
                                 const int32_t* targets, float scale, float z_loss, float* loss, float* lse, void* workspace,
                                 size_t workspace_bytes, int32_t* err_index, pg_stream_t stream) {
  Call c = {};
  c.s = {N, V, d, 1, h_dtype, w_dtype, -1, -1, false, false};
  c.h = h; c.W = W; c.targets = targets; c.t_dtype = -1;
  c.scale = scale; c.inv_t = 1.f; c.zl = z_loss;
  c.loss = loss; c.lse = lse;
  c.workspace = workspace; c.workspace_bytes = workspace_bytes; c.err = err_index; c.stream = stream;
  return call_vocab(c);
}

extern "C" pg_status pg_vocab_ce_grad(const void* h, int32_t h_dtype, int64_t N, const void* W, int32_t w_dtype, int64_t V, int32_t d,
                                      const int32_t* targets, float scale, float z_loss, const float* row_weight, float grad_scale,
                                      float* loss, float* lse, void* grad_h, int32_t gh_dtype, void* grad_w, int32_t gw_dtype,
                                      int32_t accumulate, void* workspace, size_t workspace_bytes, int32_t* err_index,
                                      pg_stream_t stream) {
  Call c = {};
  c.s = {N, V, d, 1, h_dtype, w_dtype, gh_dtype, gw_dtype, true, false};
  c.h = h; c.W = W; c.targets = targets; c.t_dtype = -1;
  c.row_weight = row_weight;
  c.scale = scale; c.inv_t = 1.f; c.zl = z_loss; c.grad_scale = grad_scale;
  c.accumulate = accumulate;
  c.loss = loss; c.lse = lse; c.gh = grad_h; c.gw = grad_w;
  c.workspace = workspace; c.workspace_bytes = workspace_bytes; c.err = err_index; c.stream = stream;
  return call_vocab(c);
}

extern "C" pg_status pg_vocab_distill(const void* h, int32_t h_dtype, int64_t N, const void* W, int32_t w_dtype, int64_t V, int32_t d,
                                      const int32_t* ids, const void* logits, int32_t logits_dtype, int32_t K, float scale,
                                      float temperature, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                      int32_t* err_index, pg_stream_t stream) {
  Call c = {};
  c.s = {N, V, d, K, h_dtype, w_dtype, -1, -1, false, true};
  if (!real_dtype(logits_dtype)) return PG_ERR_DTYPE;
  c.h = h; c.W = W; c.ids = ids; c.tlogits = logits; c.t_dtype = logits_dtype;
  c.scale = scale; c.inv_t = 1.f / temperature;
  c.loss = loss; c.lse = lse;
  c.workspace = workspace; c.workspace_bytes = workspace_bytes; c.err = err_index; c.stream = stream;
  return call_vocab(c);
}

extern "C" pg_status pg_vocab_distill_grad(const void* h, int32_t h_dtype, int64_t N, const void* W, int32_t w_dtype, int64_t V, int32_t d,
                                           const int32_t* ids, const void* logits, int32_t logits_dtype, int32_t K, float scale,
                                           float temperature, const float* row_weight, float grad_scale, float* loss, float* lse,
                                           void* grad_h, int32_t gh_dtype, void* grad_w, int32_t gw_dtype, int32_t accumulate,
                                           void* workspace, size_t workspace_bytes, int32_t* err_index, pg_stream_t stream) {
  Call c = {};
  c.s = {N, V, d, K, h_dtype, w_dtype, gh_dtype, gw_dtype, true, true};
  if (!real_dtype(logits_dtype)) return PG_ERR_DTYPE;
  c.h = h; c.W = W; c.ids = ids; c.tlogits = logits; c.t_dtype = logits_dtype;
  c.row_weight = row_weight;
  c.scale = scale; c.inv_t = 1.f / temperature; c.grad_scale = grad_scale;
  c.accumulate = accumulate;
  c.loss = loss; c.lse = lse; c.gh = grad_h; c.gw = grad_w;
  c.workspace = workspace; c.workspace_bytes = workspace_bytes; c.err = err_index; c.stream = stream;
  return call_vocab(c);
}
