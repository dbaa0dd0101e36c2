// Orthogonalised updates by Newton-Schulz steps (pg_orthogonalize), for a batch of matrices.
//
// X [m, n] is G divided by its Frobenius norm; p = min(m, n), q = max(m, n). A step is
//   A  = X X^T (m <= n) or X^T X     [p, p], symmetric
//   Bm = a I + b A + c A A           [p, p], symmetric
//   X  <- Bm X (m <= n) or X Bm      [m, n]
// three products of 2 p p q, 2 p p p and 2 p p q operations, the symmetric ones half of that.
// X stays in G's orientation: where a product needs its columns as the long rows of an
// operand, the tensor core reads the tile "MN-major" (the descriptor's transpose), and since
// Bm holds a I the last product has only what rounding left (below) to add. The tiles of A and
// Bm below the diagonal are neither computed nor stored: an operand that needs one reads its
// mirror image MN-major.
//
// Between the products X, A and Bm are held as fp16 scaled by 2^10 (pg.h): 11 significant
// bits, against the 8 of the bf16 result. That is enough for A and Bm: they multiply X, so their
// roundings stay small relative to the directions that X has. It is not for X itself: its rounding
// spreads over all singular directions, and each later step multiplies by a = 3.44 what lies in those
// that G does not have, 485-fold from X0 on (256 x 1024 of rank 1: 15 % of the result, of rank 4: 7 %).
// So X is held as a sum hi + lo of two fp16 numbers, 22 bits. A is made of hi alone (its error is
// one of A's own size), and the last step takes hi alone (its rounding grows a-fold at most).
// The other steps' X <- Bm (hi + lo) is Bm hi + a lo, the addend in the epilogue: Bm differs from a I
// where X has directions, and there lo is a rounding that does not grow. Where Bm is one k-block
// deep (p <= 128), Bm lo is one more k-block and is taken whole, as fast (128 x 1024: 79 us both ways).
// The diagonals of A and Bm keep fp32: where X's singular values are near one another (a side many times
// the other) A and Bm are nearly multiples of I, their diagonals' roundings do not average out, and a step
// stretches them up to fivefold (0.0029 off at 32 x 984 without, 0.0018 with). Their products' epilogues
// store what rounding left of A's diagonal and the ratio that rounding Bm's changed; Bm's diagonal gets the
// former's share, b + 2 c A_ii of it, and X's rows (X Bm: columns) are scaled by the ratio.
// Relative to the formulas the results are 0.0017-0.0028 off, of which 0.0017 are the bf16 result's own
// rounding, over ranks from 1 to full, spectra over up to six decades and sides from 24 to 2560. The low
// part and the diagonals cost 3 % of a small call and 13 % of the largest (256 x 1024: 80 -> 82 us, five
// 2560 x 1280: 316 -> 358); Bm lo at every size would add half to the products instead.
//
// One cooperative launch does the whole update (large batches: norm and scaling before it): norm,
// scaling, and 3 * steps products on the tensor cores. The tiles of all products stand in one list,
// product by product and matrix by matrix; unit u takes tiles u, u + units, .. of it, and a tile's
// loads wait until all tiles of the product before it of the same matrix are stored (a counter a
// matrix). So no unit waits for matrices that it does not touch, and the last round of one product
// is filled up with the next one's tiles. Every wait is for tiles earlier in the list, which every
// unit walks in order: all waits end. The held matrices stay in L2 where they fit.
//   warp 0      TMA producer: 128-deep k-blocks of both operands, 128-byte swizzle, into a ring
//   warp 1      tcgen05.mma issuer, two accumulators in TMEM
//   warps 2..9  epilogue: tcgen05.ld, the sum of the three terms, fp16 (or the bf16 result)
//
// Bound by the tensor cores where the tiles fill them: five 2560 x 1280 matrices need 367 GFLOP
// (189 us at the measured bf16 rate) and take 350-366 us, 0.53 of that rate: one step 104 us (of them
// norm 14, scaling 14), the second 58 more, each further one 68. A k-block takes 0.65 us (the rate of a
// large library product), 41 us of a step; 9 are the low part of X in the epilogue (57 us a step
// without reading and writing it); the rest is the chain: 75 tiles of A, 75 of Bm and 250 of X on 76
// CTA pairs, each product's first loads behind the last stores of the one before. One 768 x 1024 matrix
// (11 GFLOP) takes 108 us for 15 products, 31 the first step and 19.4 each further one: 7 us a product of
// loads from L2 (48 KB a k-block and SM at some 90 GB/s), the first copy, the last epilogue and the
// counter.
#include <cuda.h>
#include <cuda_fp16.h>

#include <stddef.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "pg_umma.cuh"
#include "pg_vec.h"

namespace pg {
namespace {

constexpr int kErrOrtho = 262144;       // device error bit: a wait of this kernel gave up
constexpr int kMaxSide = 16384;
constexpr int kMaxBatch = 4096;
constexpr float kHold = 1024.f;         // X, A and Bm are stored times 2^10
constexpr float kUnhold = 1.f / 1024.f;
constexpr float kUp = 0x1p90f, kDown = 0x1p-90f;
constexpr int kNormParts = 128;         // partial sums of squares per matrix, at most
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kRowsP = 128;             // rows of P that a CTA stages
static_assert(kRowsP == kBK, "one box shape serves both layouts");

// Tiles: a CTA pair computes 256 x 256 (each CTA stages 128 rows of P and 128 of Q and
// accumulates 128 rows), a single CTA 128 x 64.
template <bool PAIR>
struct Tile {
  static constexpr int kM = PAIR ? 256 : 128;
  static constexpr int kN = PAIR ? 256 : 64;
  static constexpr int kRowsQ = PAIR ? 128 : 64;
  static constexpr int kPBytes = kRowsP * kBK * 2;
  static constexpr int kQBytes = kRowsQ * kBK * 2;
  static constexpr int kStages = PAIR ? 3 : 4;
  static constexpr int kChunkN = 32;       // columns that an epilogue warp stages at a time
  static constexpr int kChunks = kN / 2 / kChunkN;     // of its half of the tile
  static constexpr int kStageBytes = 32 * kChunkN * 2;
  static constexpr int kTmemCols = 2 * kN;
  static constexpr uint32_t kIdesc =                   // kind::f16: fp32 sums, fp16 operands
      (1u << 4) | (static_cast<uint32_t>(kN >> 3) << 17) | (static_cast<uint32_t>(kM >> 4) << 24);
  static constexpr size_t kRing = static_cast<size_t>(kStages) * (kPBytes + kQBytes);
  static constexpr size_t kSmem = 1024 + kRing + kEpiWarps * (kStageBytes + kChunkN * sizeof(float));
};

struct OrthoCtrl {
  uint32_t barrier;
  uint32_t pad[31];
  uint32_t stored[kMaxBatch];  // per matrix: epilogue warps that have stored their part of a tile
};

struct OrthoArgs {
  const void* G;
  __nv_bfloat16* out;
  OrthoCtrl* ctrl;
  float* partial;            // [batch][parts][3]
  __half *X[2], *A, *Bm;     // [batch][m][ldx], [batch][p][ldp]
  float2* dA;                // [batch][ldp] A's diagonal as held, and what rounding left of it (times 2^10)
  float* rB;                 // [batch][ldp] Bm's diagonal over what is held of it
  __half* L[2];              // what X's rounding to fp16 left, as X; one buffer unless lo_product
  int* err_word;
  int64_t size;              // m n
  int batch, m, n, p, ldx, ldp, parts, steps, dtype;
  int g_vec, out_vec;        // accesses of 8 columns to G; to out
  int prepared;              // X0 is there already
  int lo_product;            // Bm lo is a k-block of the product; else a lo is added
  int tiles[3];              // of one matrix, of each product
  float a, b, c, eps, scale;
};

// Boxes of 64 columns and 128 rows; for the single CTA's 64 rows of Q, K-major, of 64 rows too.
struct Maps {
  CUtensorMap X[2], A, Bm, L[2];
  CUtensorMap Xq[2], Aq, Bmq;
};

// --------------------------------------------------------------------- norm and scaling

// 8 consecutive values of G as they lie in memory; the loads are volatile so that they stay
// together, ahead of their uses. They are coherent ones: the result may lie in G's place, and the
// launch that reads G may write it.
template <int DT>
struct Raw8 {
  float f[DT == PG_F32 ? 8 : 1];
  uint4 h;

  __device__ __forceinline__ void load(const void* G, int64_t at) {
    if constexpr (DT == PG_F32)
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                   : "l"(static_cast<const float*>(G) + at)
                   : "memory");
    else
      asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(h.x), "=r"(h.y), "=r"(h.z), "=r"(h.w)
                   : "l"(static_cast<const uint16_t*>(G) + at)
                   : "memory");
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (DT == PG_F32) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = f[k];
    } else {
      const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __uint_as_float((k & 1) ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    }
  }
};

// Partial sums of squares, of x, 2^90 x and 2^-90 x: whichever of the three neither overflows
// nor vanishes gives the norm, for all finite x (the least, 2^-149, squares to 2^-118; 2^28 values
// below 2^128 sum to less than 2^104). Part `part` of matrix `b` is a contiguous share of it.
template <int DT, int THREADS>
__device__ void norm_part(const OrthoArgs& g, int b, int part, float (*s_sum)[THREADS / 32]) {
  const int64_t share = ((g.size + g.parts - 1) / g.parts + 7) / 8 * 8;
  const int64_t lo = part * share, hi = min(g.size, lo + share), base = b * g.size;
  float sum[3] = {};
  auto add = [&](float x) {
    const float up = x * kUp, down = x * kDown;
    sum[0] = fmaf(x, x, sum[0]);
    sum[1] = fmaf(up, up, sum[1]);
    sum[2] = fmaf(down, down, sum[2]);
  };
  if (g.g_vec) {
    constexpr int kFly = (DT == PG_F32 ? 8 : 16) * kThreads / THREADS;  // loads in flight
    for (int64_t i = lo + threadIdx.x * 8; i < hi; i += kFly * THREADS * 8) {
      Raw8<DT> raw[kFly];
#pragma unroll
      for (int u = 0; u < kFly; ++u) raw[u].load(g.G, base + min(i + u * THREADS * 8, hi - 8));
#pragma unroll
      for (int u = 0; u < kFly; ++u) {
        if (i + u * THREADS * 8 >= hi) break;
        float x[8];
        raw[u].get(x);
#pragma unroll
        for (int k = 0; k < 8; ++k) add(x[k]);
      }
    }
  } else {
    for (int64_t i = lo + threadIdx.x; i < hi; i += THREADS) {
      float x[1];
      read_cols<DT, 1>(g.G, base + i, x);
      add(x[0]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
    if ((threadIdx.x & 31) == 0) s_sum[k][threadIdx.x >> 5] = sum[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = 0.f;
    for (int w = 0; w < THREADS / 32; ++w) t += s_sum[threadIdx.x][w];
    g.partial[(static_cast<int64_t>(b) * g.parts + part) * 3 + threadIdx.x] = t;
  }
}

// 2^10 / (|G|_F + eps) of matrix b as a product, by one warp: lane-strided sums and an xor tree, a fixed
// order. The first factor is the power of two that the norm was summed with: the quotient alone
// leaves fp32's range for norms below 2^-118, and the norm itself can.
__device__ float2 held_scale(const OrthoArgs& g, int b) {
  const int lane = threadIdx.x & 31;
  float s[3] = {};
  for (int i = lane; i < g.parts; i += 32)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += __ldcg(g.partial + (static_cast<int64_t>(b) * g.parts + i) * 3 + k);
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int o = 16; o; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  float by = 1.f, sum = s[0];
  if (s[0] <= 0x1p-60f) {
    by = kUp;
    sum = s[1];
  } else if (!(s[0] < 0x1p120f)) {  // also NaN and infinities
    by = kDown;
    sum = s[2];
  }
  return make_float2(by, kHold / (sqrtf(sum) + g.eps * by));
}

__device__ __forceinline__ uint32_t two_half(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What rounding `hi` of two values left.
__device__ __forceinline__ uint32_t two_left(uint32_t hi, float x0, float x1) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return two_half(x0 - f.x, x1 - f.y);
}

// X0: rows of G scaled and rounded into rows of stride ldx, 8 columns at a time. A block owns a
// contiguous share of the rows of all matrices.
template <int DT, int THREADS>
__device__ void scale_rows(const OrthoArgs& g, float2* s_scale) {
  const uint32_t per_row = (g.n + 7) / 8;
  const int64_t rows = static_cast<int64_t>(g.batch) * g.m;
  const int64_t lo = rows * blockIdx.x / gridDim.x, hi = rows * (blockIdx.x + 1) / gridDim.x;
  for (int64_t r0 = lo; r0 < hi;) {
    const int b = static_cast<int>(r0 / g.m);
    const int64_t r1 = min(hi, static_cast<int64_t>(b + 1) * g.m);
    __syncthreads();
    if (threadIdx.x < 32) {
      const float2 s = held_scale(g, b);
      if (threadIdx.x == 0) *s_scale = s;
    }
    __syncthreads();
    const float by = s_scale->x, scale = s_scale->y;
    const uint32_t vecs = static_cast<uint32_t>(r1 - r0) * per_row;  // < 2^31: at most m of at most 2048
    auto store = [&](uint32_t v, const float (&x)[8]) {
      const uint32_t r = v / per_row, j = (v - r * per_row) * 8;
      const int64_t at = (r0 + r) * g.ldx + j;
      uint32_t hi[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) hi[k] = two_half(x[2 * k] * by * scale, x[2 * k + 1] * by * scale);
      *reinterpret_cast<uint4*>(g.X[0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (g.steps == 1) return;
#pragma unroll
      for (int k = 0; k < 4; ++k) hi[k] = two_left(hi[k], x[2 * k] * by * scale, x[2 * k + 1] * by * scale);
      *reinterpret_cast<uint4*>(g.L[0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    };
    if (g.g_vec) {  // n % 8 == 0: a row's pieces follow the row before's
      constexpr int kFly = (DT == PG_F32 ? 8 : 12) * kThreads / THREADS;
      for (uint32_t v0 = threadIdx.x; v0 < vecs; v0 += kFly * THREADS) {
        Raw8<DT> raw[kFly];
#pragma unroll
        for (int u = 0; u < kFly; ++u)
          raw[u].load(g.G, r0 * g.n + 8ll * min(v0 + u * THREADS, vecs - 1));
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
          if (v0 + u * THREADS >= vecs) break;
          float x[8];
          raw[u].get(x);
          store(v0 + u * THREADS, x);
        }
      }
    } else {
      for (uint32_t v = threadIdx.x; v < vecs; v += THREADS) {
        const uint32_t r = v / per_row, j = (v - r * per_row) * 8;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float y[1] = {0.f};
          if (j + k < static_cast<uint32_t>(g.n)) read_cols<DT, 1>(g.G, (r0 + r) * g.n + j + k, y);
          x[k] = y[0];
        }
        store(v, x);
      }
    }
    r0 = r1;
  }
}

// The two as launches of their own, for large batches (see pg_orthogonalize).
constexpr int kPrepThreads = 640;

template <int DT>
__global__ void __launch_bounds__(kPrepThreads, 2) ortho_norm_kernel(const __grid_constant__ OrthoArgs g) {
  __shared__ float s_sum[3][kPrepThreads / 32];
  norm_part<DT, kPrepThreads>(g, blockIdx.x / g.parts, blockIdx.x % g.parts, s_sum);
}

template <int DT>
__global__ void __launch_bounds__(kPrepThreads, 2) ortho_scale_kernel(const __grid_constant__ OrthoArgs g) {
  __shared__ float2 s_scale;
  scale_rows<DT, kPrepThreads>(g, &s_scale);
}

// --------------------------------------------------------------------------- the products

// D = alpha (P Q^T + P2 Q2^T) + beta C + diag I; see the top of the file.
struct Product {
  const CUtensorMap *P, *Q, *Qrows;  // Qrows: Q in boxes of as many rows as a CTA stages of it
  const CUtensorMap *P2, *Q2;        // the low part's operands, laid out as P and Q, one k-block deep
  const __half* C;       // laid out as D, or null
  __half* D;             // [M, N]; null for the last product (out)
  __half* Dlo;           // what rounding D left, or null
  int64_t strideD;       // between matrices, elements
  int ldD, M, N, K;
  float alpha, beta, diag;
  bool symmetric, low;   // low: there are P2 and Q2
  // An operand is K-major (its rows are the matrix's), MN-major (the matrix's columns), or, A
  // and Bm, symmetric with only the tiles that reach the diagonal or lie above it stored: those
  // K-major, the others as the MN-major mirror image.
  enum Layout { kRows, kColumns, kUpper } p_in, q_in;
};

// Whether k-block k0 of the operand's rows from r0 on is read MN-major.
template <bool PAIR>
__device__ __forceinline__ bool reads_mn(Product::Layout in, int r0, int k0) {
  return in == Product::kColumns || (in == Product::kUpper && k0 / Tile<PAIR>::kM < r0 / Tile<PAIR>::kM);
}

template <bool PAIR>
__device__ __forceinline__ Product product_of(const OrthoArgs& g, const Maps& maps, int step, int kind) {
  const int cur = step & 1;
  const bool wide = g.m <= g.n;
  Product r;
  r.symmetric = kind < 2;
  r.M = r.N = r.K = g.p;
  r.P2 = r.Q2 = nullptr;
  r.low = false;
  r.C = nullptr;
  r.Dlo = nullptr;
  r.alpha = kUnhold;
  r.beta = r.diag = 0.f;
  r.ldD = g.ldp;
  if (kind == 0) {         // A
    r.P = r.Q = &maps.X[cur];
    r.Qrows = PAIR ? r.Q : &maps.Xq[cur];
    r.p_in = r.q_in = wide ? Product::kRows : Product::kColumns;
    r.D = g.A;
    r.K = wide ? g.n : g.m;
  } else if (kind == 1) {  // Bm
    r.P = r.Q = &maps.A;
    r.Qrows = PAIR ? r.Q : &maps.Aq;
    r.p_in = r.q_in = Product::kUpper;
    r.C = g.A;
    r.D = g.Bm;
    r.alpha = g.c * kUnhold;
    r.beta = g.b;
    r.diag = g.a * kHold;
  } else {                 // X
    r.P = wide ? &maps.Bm : &maps.X[cur];
    r.Q = wide ? &maps.X[cur] : &maps.Bm;
    r.Qrows = PAIR ? r.Q : wide ? &maps.Xq[cur] : &maps.Bmq;
    r.p_in = wide ? Product::kUpper : Product::kRows;
    r.q_in = wide ? Product::kColumns : Product::kUpper;
    r.D = step + 1 == g.steps ? nullptr : g.X[cur ^ 1];
    r.Dlo = step + 2 < g.steps ? g.L[cur ^ 1] : nullptr;
    if (g.lo_product) {
      r.low = step + 1 < g.steps;
      r.P2 = wide ? r.P : &maps.L[cur];
      r.Q2 = wide ? &maps.L[cur] : r.Q;
    } else {               // (a tile reads the part of lo that it writes)
      r.C = g.L[cur];
      r.beta = g.a;
    }
    r.M = g.m;
    r.N = g.n;
    r.ldD = g.ldx;
  }
  r.strideD = static_cast<int64_t>(r.M) * r.ldD;
  return r;
}

// Tiles of one matrix; symmetric: those that reach the diagonal or lie above it.
template <bool PAIR>
__host__ __device__ __forceinline__ int tiles_of(int M, int N, bool symmetric) {
  constexpr int kM = Tile<PAIR>::kM, kN = Tile<PAIR>::kN, kR = kM / kN;
  const int nm = (M + kM - 1) / kM, nn = (N + kN - 1) / kN;
  return symmetric ? nm * nn - kR * (nm * (nm - 1) / 2) : nm * nn;
}

// Tile t of the list of all products: its product, matrix and place, and how many of the matrix's
// tiles have to be stored before.
struct Work {
  int step, kind, b, i, j, before;
};

template <bool PAIR>
__device__ __forceinline__ Work work_at(const OrthoArgs& g, int t) {
  const int one = g.tiles[0] + g.tiles[1] + g.tiles[2], per_step = g.batch * one;
  Work w;
  w.step = t / per_step;
  int r = t - w.step * per_step;
  w.kind = 0;
  w.before = w.step * one;
  while (r >= g.batch * g.tiles[w.kind]) {
    r -= g.batch * g.tiles[w.kind];
    w.before += g.tiles[w.kind];
    ++w.kind;
  }
  w.b = r / g.tiles[w.kind];
  r -= w.b * g.tiles[w.kind];
  constexpr int kN = Tile<PAIR>::kN, kR = Tile<PAIR>::kM / kN;
  const int nn = ((w.kind == 2 ? g.n : g.p) + kN - 1) / kN;
  if (w.kind < 2) {
    w.i = 0;
    for (int left = nn; r >= left; left -= kR) {
      r -= left;
      ++w.i;
    }
    w.j = w.i * kR + r;
  } else {
    w.i = r / nn;
    w.j = r - w.i * nn;
  }
  return w;
}

// Waits until matrix b has `want` stored parts; false as `wait`.
__device__ __forceinline__ bool wait_stored(const OrthoArgs& g, int b, uint32_t want, volatile int* abort) {
  const uint32_t* at = &g.ctrl->stored[b];
  uint64_t t0 = 0;
  for (;;) {
    for (int k = 0; k < 64; ++k) {
      uint32_t seen;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(at) : "memory");
      if (seen >= want) return true;
    }
    if (t0 == 0) t0 = now_ns();
    if (*abort || now_ns() - t0 > kAsyncWaitNs) return false;
  }
}

// The producer tells the epilogue's warps, tile by tile, that what the tile needs is stored: they load their
// addends and factors while the tile's products run. It is at most the ring's stages and the two
// accumulators ahead of them, fewer tiles than there are barriers.
constexpr int kReady = 16;
static_assert(kReady > Tile<false>::kStages + 4 && kReady > Tile<true>::kStages + 4, "");

template <int S>
struct Bars {
  uint64_t full[S], empty[S], acc_full[2], acc_empty[2], ready[kReady], done;
  uint32_t tmem;
  int abort, ok;
};

// The grid barrier: every thread's global writes so far are visible to every block's loads
// after it; thread 0, which issues the TMA loads, orders what it has seen before them. False
// once a block gave up (about a second).
template <int S>
__device__ __forceinline__ bool grid_meet(const OrthoArgs& g, Bars<S>* bars, uint32_t* phase) {
  __syncthreads();
  *phase += 1;
  if (threadIdx.x == 0) {
    bool ok = !*static_cast<volatile int*>(&bars->abort);
    if (ok) {
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(&g.ctrl->barrier) : "memory");
      const uint32_t want = *phase * gridDim.x;
      const uint64_t t0 = now_ns();
      for (;;) {
        uint32_t seen;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(&g.ctrl->barrier) : "memory");
        if (seen >= want) break;
        if (now_ns() - t0 > kAsyncWaitNs) {
          ok = false;
          atomicOr(g.err_word, kErrOrtho);
          break;
        }
      }
      fence_async_global();
    }
    bars->ok = ok;
  }
  __syncthreads();
  return bars->ok != 0;
}

// What an epilogue writes. One instance each: its body has no branches between the columns, so
// that the arithmetic of a chunk overlaps (with them a chunk took twice as long).
enum Kind { kMakeA, kMakeB, kMakeX, kMakeXPlain, kMakeOut };  // kMakeXPlain: without an addend

// A warp takes 32 rows of a tile (its TMEM lanes) and half of its columns, in chunks. TMEM gives
// a lane one row; global memory wants neighbouring lanes on one row. So a chunk passes through
// the warp's shared memory, C the same way in: lane-per-row accesses to global memory (32 lines
// each) took half of the kernel's time. TALL: X Bm, whose columns are scaled by Bm's ratios; else its
// rows. False once a wait gave up.
template <bool PAIR, int KIND, bool TALL, int S>
__device__ __forceinline__ bool epilogue(const OrthoArgs& g, const Product& pr, const Work& w, Bars<S>* bars, uint8_t* s_epi,
                                         uint32_t tmem, uint32_t rank, int acc, uint32_t acc_phase, uint32_t nth) {
  using T = Tile<PAIR>;
  constexpr int kC = T::kChunkN, kPieces = kC / 8, kSide = 32 / kPieces;  // 16-byte pieces a row; rows an access covers
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, half = (warp - 2) >> 2;
  uint8_t* s_row = s_epi + (warp - 2) * T::kStageBytes;  // [32 rows][kC columns], pieces swizzled over the banks
  auto piece = [&](int r, int c) {
    return reinterpret_cast<uint4*>(s_row + r * (2 * kC) + ((c ^ (r * kPieces / 8 % kPieces)) << 4));
  };
  const int lr = lane / kPieces, lc = lane % kPieces;    // this lane's row (of kSide) and piece in a coalesced access
  const float alpha = KIND == kMakeOut ? pr.alpha * g.scale * kUnhold : pr.alpha;
  constexpr bool kAdds = KIND == kMakeB || KIND == kMakeX;
  constexpr bool kTimesB = KIND != kMakeA && KIND != kMakeB;
  float* s_col = reinterpret_cast<float*>(s_epi + kEpiWarps * T::kStageBytes) + (warp - 2) * kC;
  const int b = w.b, i = w.i, j = w.j;
  const int row0 = i * T::kM + static_cast<int>(rank) * kRowsP + quarter * 32;
  const int col0 = j * T::kN + half * (T::kN / 2);
  const bool some = row0 < pr.M;
  const int64_t at = b * pr.strideD + static_cast<int64_t>(row0 + lr) * pr.ldD + col0 + lc * 8;
  uint4 cw[kPieces];  // C of the next chunk, in coalesced order
  auto load_c = [&](int ch) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      cw[k] = make_uint4(0, 0, 0, 0);
      if (row0 + lr + kSide * k < pr.M && col0 + ch * kC + lc * 8 < pr.ldD)
        cw[k] = __ldcg(reinterpret_cast<const uint4*>(pr.C + at + static_cast<int64_t>(kSide * k) * pr.ldD + ch * kC));
    }
  };
  if (KIND != kMakeA &&  // (which needs nothing but its product)
      !__all_sync(0xffffffffu, wait<false>(smem_addr(&bars->ready[nth % kReady]), nth / kReady & 1u, &bars->abort)))
    return false;
  if (kAdds) load_c(0);
  const bool on_diag = row0 >= col0 && row0 < col0 + T::kN / 2;  // 32 rows and columns of it
  float2 d = make_float2(0.f, 0.f);
  if (KIND == kMakeB && on_diag && row0 + lane < pr.M) d = __ldcg(g.dA + static_cast<int64_t>(b) * g.ldp + row0 + lane);
  const float row_alpha = kTimesB && !TALL && row0 + lane < pr.M
                              ? alpha * __ldcg(g.rB + static_cast<int64_t>(b) * g.ldp + row0 + lane) : alpha;
  auto load_ratio = [&](int c) { return c + lane < pr.N ? __ldcg(g.rB + static_cast<int64_t>(b) * g.ldp + c + lane) : 0.f; };
  float ratio = kTimesB && TALL ? load_ratio(col0) : 0.f;
  if (!__all_sync(0xffffffffu, wait<PAIR>(smem_addr(&bars->acc_full[acc]), acc_phase, &bars->abort))) return false;
  fence_after();
#pragma unroll 1
  for (int ch = 0; some && ch < T::kChunks; ++ch) {
    const int c0 = col0 + ch * kC;
    if (c0 >= pr.N) break;
    uint32_t r[kC];
    const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * T::kN) +
                          static_cast<uint32_t>(half * (T::kN / 2) + ch * kC);
#pragma unroll
    for (int k = 0; k < kC; k += 32) tmem_load(from + k, r + k);
    if (kAdds) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) *piece(lr + kSide * k, lc) = cw[k];
      if (ch + 1 < T::kChunks) load_c(ch + 1);
    }
    if (kTimesB && TALL) {
      s_col[lane] = alpha * ratio;
      if (ch + 1 < T::kChunks) ratio = load_ratio(c0 + kC);
    }
    if (kAdds || (kTimesB && TALL)) __syncwarp();
    tmem_wait(r);
    float x[kC];
    if constexpr (kTimesB && TALL) {
#pragma unroll
      for (int k = 0; k < kC; k += 4) {
        const float4 f = *reinterpret_cast<const float4*>(s_col + k);
        x[k] = f.x * __uint_as_float(r[k]);
        x[k + 1] = f.y * __uint_as_float(r[k + 1]);
        x[k + 2] = f.z * __uint_as_float(r[k + 2]);
        x[k + 3] = f.w * __uint_as_float(r[k + 3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kC; ++k) x[k] = row_alpha * __uint_as_float(r[k]);
    }
    if (kAdds) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const uint4 q = *piece(lane, k);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e / 2]));
          x[8 * k + e] = fmaf(pr.beta, f.x, x[8 * k + e]);
          x[8 * k + e + 1] = fmaf(pr.beta, f.y, x[8 * k + e + 1]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {  // two columns a word: fp16, or the result in bf16
      const float* v = x + 8 * k;
      *piece(lane, k) = KIND == kMakeOut
          ? make_uint4(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]), two_bf16(v[4], v[5]), two_bf16(v[6], v[7]))
          : make_uint4(two_half(v[0], v[1]), two_half(v[2], v[3]), two_half(v[4], v[5]), two_half(v[6], v[7]));
    }
    if ((KIND == kMakeA || KIND == kMakeB) && c0 == row0) {  // the chunk's diagonal is the matrix's
      float t[kC / 2];
#pragma unroll
      for (int k = 0; k < kC / 2; ++k) t[k] = (lane & kC / 2) ? x[k + kC / 2] : x[k];
#pragma unroll
      for (int s = kC / 4; s; s >>= 1)
#pragma unroll
        for (int k = 0; k < s; ++k) t[k] = (lane & s) ? t[k + s] : t[k];
      float mine = t[0];  // of row and column `lane`
      if (KIND == kMakeB) mine += pr.diag + fmaf(2.f * g.c * kUnhold * d.x, d.y, g.b * d.y);
      const __half rounded = __float2half_rn(mine);
      const float held = __half2float(rounded);
      const int64_t to = static_cast<int64_t>(b) * g.ldp + row0 + lane;
      if (KIND == kMakeB) reinterpret_cast<__half*>(piece(lane, lane / 8))[lane % 8] = rounded;
      if (row0 + lane < pr.M) {
        if (KIND == kMakeA)
          g.dA[to] = make_float2(held, mine - held);
        else
          g.rB[to] = held != 0.f ? mine / held : 1.f;
      }
    }
    __syncwarp();
    auto store = [&](uint16_t* to, int64_t ld) {  // the staged chunk, rows of stride ld; to: this lane's first piece
      uint4 q[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) q[k] = *piece(lr + kSide * k, lc);
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        if (row0 + lr + kSide * k < pr.M) *reinterpret_cast<uint4*>(to + kSide * k * ld) = q[k];
    };
    if (KIND != kMakeOut || (g.out_vec && c0 + kC <= pr.N)) {  // (columns past N land in the padding of D's rows)
      store(KIND != kMakeOut ? reinterpret_cast<uint16_t*>(pr.D) + at + ch * kC
                             : reinterpret_cast<uint16_t*>(g.out) + b * g.size +
                                   static_cast<int64_t>(row0 + lr) * pr.N + c0 + lc * 8,
            KIND != kMakeOut ? pr.ldD : pr.N);
    } else {  // a ragged edge of the result, or one at an odd address
      uint16_t* to = reinterpret_cast<uint16_t*>(g.out) + b * g.size + static_cast<int64_t>(row0) * pr.N + c0;
      for (int e = lane; e < 32 * kC; e += 32) {
        const int rr = e / kC, cc = e % kC;
        if (row0 + rr < pr.M && c0 + cc < pr.N)
          to[static_cast<int64_t>(rr) * pr.N + cc] = reinterpret_cast<const uint16_t*>(piece(rr, cc / 8))[cc % 8];
      }
    }
    __syncwarp();
    if ((KIND == kMakeX || KIND == kMakeXPlain) && pr.Dlo) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const float* v = x + 8 * k;
        const uint4 q = *piece(lane, k);
        *piece(lane, k) = make_uint4(two_left(q.x, v[0], v[1]), two_left(q.y, v[2], v[3]), two_left(q.z, v[4], v[5]),
                                     two_left(q.w, v[6], v[7]));
      }
      __syncwarp();
      store(reinterpret_cast<uint16_t*>(pr.Dlo) + at + ch * kC, pr.ldD);
      __syncwarp();
    }
  }
  fence_before();
  __syncwarp();
  if (lane == 0) {
    const uint32_t bar = smem_addr(&bars->acc_empty[acc]);
    if constexpr (PAIR)
      asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_cta(bar, 0)) : "memory");
    else
      bar_arrive(bar);
    // this warp's part of the tile is stored (the release covers what its lanes wrote before __syncwarp)
    if (KIND != kMakeOut)
      asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(&g.ctrl->stored[b]) : "memory");
  }
  return true;
}

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_kernel(const __grid_constant__ Maps maps, const __grid_constant__ OrthoArgs g) {
  using T = Tile<PAIR>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t s_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars<S> bars_s;
  __shared__ float s_sum[3][kThreads / 32];
  __shared__ float2 s_scale;
  uint8_t* s_epi = ring + T::kRing;                       // the epilogue warps' staging
  Bars<S>* bars = &bars_s;
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cta_rank() : 0u;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, units = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      bar_init(smem_addr(&bars->full[s]), 1);
      bar_init(smem_addr(&bars->empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(smem_addr(&bars->acc_full[s]), 1);
      bar_init(smem_addr(&bars->acc_empty[s]), (PAIR ? 2 : 1) * kEpiWarps);
    }
    for (int s = 0; s < kReady; ++s) bar_init(smem_addr(&bars->ready[s]), 1);
    bar_init(smem_addr(&bars->done), 1);
    bars->abort = 0;
    bar_init_fence();
    fence_async_smem();
  }
  if (warp == 1) tmem_alloc<PAIR>(smem_addr(&bars->tmem), T::kTmemCols);
  fence_before();
  __syncthreads();
  if constexpr (PAIR) pair_sync();  // both CTAs' barriers and TMEM exist before any remote use
  fence_after();
  const uint32_t tmem = bars->tmem;

  // ---- |G|_F and X0
  uint32_t phase = 0;
  bool ok = true;
  if (!g.prepared) {
    const bool f32 = g.dtype == PG_F32;
    for (int w = blockIdx.x; w < g.batch * g.parts; w += gridDim.x)
      f32 ? norm_part<PG_F32, kThreads>(g, w / g.parts, w % g.parts, s_sum)
          : norm_part<PG_BF16, kThreads>(g, w / g.parts, w % g.parts, s_sum);
    ok = grid_meet(g, bars, &phase);
    if (ok) {
      f32 ? scale_rows<PG_F32, kThreads>(g, &s_scale) : scale_rows<PG_BF16, kThreads>(g, &s_scale);
      ok = grid_meet(g, bars, &phase);
    }
  }

  // ---- the products; each role walks this unit's tiles of the list, carrying its place in the ring
  // and the accumulators along
  int stage = 0, acc = 0;
  uint32_t ring_phase = 0, acc_phase = 0;
  const int total = ok ? g.steps * g.batch * (g.tiles[0] + g.tiles[1] + g.tiles[2]) : 0;
  if (warp == 0) {
    if (lane == 0) {
      bool fine = true;
      uint32_t nth = 0;
      for (int t = unit; fine && t < total; t += units, ++nth) {
        const Work w = work_at<PAIR>(g, t);
        const Product pr = product_of<PAIR>(g, maps, w.step, w.kind);
        if (!wait_stored(g, w.b, static_cast<uint32_t>(w.before) * ((PAIR ? 2 : 1) * kEpiWarps), abort)) {
          fine = false;
          break;
        }
        bar_arrive(smem_addr(&bars->ready[nth % kReady]));
        fence_async_global();  // what the epilogues stored, before the TMA reads it
        const int high_kb = (pr.K + kBK - 1) / kBK, num_kb = high_kb + pr.low;
        const int p0 = w.i * T::kM + static_cast<int>(rank) * kRowsP, q0 = w.j * T::kN + static_cast<int>(rank) * T::kRowsQ;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait<PAIR>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u, abort)) {
            fine = false;
            break;
          }
          const uint32_t full = smem_addr(&bars->full[stage]);
          const uint32_t dp = smem_addr(ring + stage * (T::kPBytes + T::kQBytes)), dq = dp + T::kPBytes;
          const uint32_t bar = PAIR ? in_cta(full, 0) : full;
          if (rank == 0) bar_expect(full, (PAIR ? 2 : 1) * (T::kPBytes + T::kQBytes));
          const bool low = kb == high_kb;  // (P2 is K-major or Bm, Q2 MN-major or Bm: Qrows serves both)
          const int k0 = low ? 0 : kb * kBK;
          const CUtensorMap* P = low ? pr.P2 : pr.P;
          load_operand<PAIR, kRowsP>(dp, P, P, reads_mn<PAIR>(pr.p_in, w.i * T::kM, k0), p0, k0, w.b, bar);
          load_operand<PAIR, T::kRowsQ>(dq, low ? pr.Q2 : pr.Q, pr.Qrows, reads_mn<PAIR>(pr.q_in, w.j * T::kN, k0), q0, k0,
                                        w.b, bar);
          if (++stage == S) {
            stage = 0;
            ring_phase ^= 1u;
          }
        }
      }
      if (!fine) {
        atomicOr(g.err_word, kErrOrtho);
        *abort = 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      bool fine = true;
      for (int t = unit; fine && t < total; t += units) {
        const Work w = work_at<PAIR>(g, t);
        const Product pr = product_of<PAIR>(g, maps, w.step, w.kind);
        if (!wait<PAIR>(smem_addr(&bars->acc_empty[acc]), acc_phase ^ 1u, abort)) {
          fine = false;
          break;
        }
        fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * T::kN);
        const int high_kb = (pr.K + kBK - 1) / kBK, num_kb = high_kb + pr.low;
        for (int kb = 0; kb < num_kb; ++kb) {
          const int k0 = kb == high_kb ? 0 : kb * kBK;
          if (!wait<PAIR>(smem_addr(&bars->full[stage]), ring_phase, abort)) {
            fine = false;
            break;
          }
          fence_after();
          const uint32_t sp = smem_addr(ring + stage * (T::kPBytes + T::kQBytes));
          const bool p_mn = reads_mn<PAIR>(pr.p_in, w.i * T::kM, k0), q_mn = reads_mn<PAIR>(pr.q_in, w.j * T::kN, k0);
          const uint64_t dp = operand_desc(sp, p_mn), dq = operand_desc(sp + T::kPBytes, q_mn);
          const uint32_t idesc = T::kIdesc | (p_mn ? 1u << 15 : 0u) | (q_mn ? 1u << 16 : 0u);
          // 16 k further: 32 bytes along a K-major line (after four, the deeper half), two 8-k
          // groups of an MN-major tile
          const uint32_t step_p = p_mn ? 2048 >> 4 : 32 >> 4, step_q = q_mn ? 2048 >> 4 : 32 >> 4;
          const uint32_t half_p = p_mn ? 4 * step_p : T::kPBytes / 2 >> 4, half_q = q_mn ? 4 * step_q : T::kQBytes / 2 >> 4;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma_f16<PAIR>(d, dp + (k / 4) * half_p + (k % 4) * step_p, dq + (k / 4) * half_q + (k % 4) * step_q, idesc,
                          (kb | k) != 0);
          commit<PAIR>(smem_addr(&bars->empty[stage]));
          if (++stage == S) {
            stage = 0;
            ring_phase ^= 1u;
          }
        }
        if (!fine) break;
        commit<PAIR>(smem_addr(&bars->acc_full[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!fine) {
        atomicOr(g.err_word, kErrOrtho);
        *abort = 1;
      }
    }
  } else {
    bool fine = true;
    uint32_t nth = 0;
    for (int t = unit; fine && t < total; t += units, ++nth) {
      const Work w = work_at<PAIR>(g, t);
      const Product pr = product_of<PAIR>(g, maps, w.step, w.kind);
      auto make_x = [&](auto tall) {
        constexpr bool kTall = decltype(tall)::value;
        if (pr.D && pr.C) return epilogue<PAIR, kMakeX, kTall>(g, pr, w, bars, s_epi, tmem, rank, acc, acc_phase, nth);
        if (pr.D) return epilogue<PAIR, kMakeXPlain, kTall>(g, pr, w, bars, s_epi, tmem, rank, acc, acc_phase, nth);
        return epilogue<PAIR, kMakeOut, kTall>(g, pr, w, bars, s_epi, tmem, rank, acc, acc_phase, nth);
      };
      if (w.kind == 0)
        fine = epilogue<PAIR, kMakeA, false>(g, pr, w, bars, s_epi, tmem, rank, acc, acc_phase, nth);
      else if (w.kind == 1)
        fine = epilogue<PAIR, kMakeB, false>(g, pr, w, bars, s_epi, tmem, rank, acc, acc_phase, nth);
      else
        fine = g.m > g.n ? make_x(std::true_type{}) : make_x(std::false_type{});
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (!fine) {
      if (lane == 0) atomicOr(g.err_word, kErrOrtho);
      *abort = 1;
    }
  }
  __syncwarp();

  // ---- teardown: every copy has landed and every MMA and commit has finished before the CTA
  // (or its peer) may exit and its TMEM is given back
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      const uint64_t t0 = now_ns();
      while (!poll<PAIR>(smem_addr(&bars->empty[stage]), ring_phase ^ 1u) && now_ns() - t0 < kAsyncWaitNs / 8) {
      }
      if (++stage == S) {
        stage = 0;
        ring_phase ^= 1u;
      }
    }
  }
  if (warp == 1 && lane == 0 && rank == 0) {
    commit_here<PAIR>(smem_addr(&bars->done));
    const uint64_t t0 = now_ns();
    while (!poll<PAIR>(smem_addr(&bars->done), 0) && now_ns() - t0 < kAsyncWaitNs) {
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (PAIR) pair_sync();
  if (warp == 1) tmem_free<PAIR>(tmem, T::kTmemCols);
}

// Block 0 of two waits for the other at the grid barrier and for a tile that nothing stores.
__global__ void __launch_bounds__(64) ortho_wait_selftest_kernel(OrthoCtrl* ctrl, int* gave_up, int* err_word) {
  __shared__ Bars<1> bars;
  if (blockIdx.x != 0) return;
  if (threadIdx.x == 0) bars.abort = 0;
  __syncthreads();
  OrthoArgs g = {};
  g.ctrl = ctrl;
  g.err_word = err_word;
  uint32_t phase = 0;
  if (!grid_meet(g, &bars, &phase) && threadIdx.x == 0) gave_up[0] = 1;
  if (threadIdx.x == 0 && !wait_stored(g, 0, 1u, &bars.abort)) {
    gave_up[1] = 1;
    atomicOr(err_word, kErrOrtho);
  }
}

// ------------------------------------------------------------------------------ host side

size_t ctrl_bytes(int64_t batch) { return offsetof(OrthoCtrl, stored) + batch * sizeof(uint32_t); }

size_t carve_ortho(uint8_t* base, int64_t batch, int m, int n, OrthoArgs* o) {
  uint8_t* first = base ? reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(base) + 127) & ~uintptr_t(127)) : nullptr;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* ptr = first ? first + at : nullptr;
    at += (bytes + 127) / 128 * 128;
    return ptr;
  };
  const int p = std::min(m, n);
  o->ldx = (n + 63) / 64 * 64;  // rows start on 128 bytes
  o->ldp = (p + 63) / 64 * 64;
  o->ctrl = reinterpret_cast<OrthoCtrl*>(take(ctrl_bytes(batch)));
  o->partial = reinterpret_cast<float*>(take(batch * kNormParts * 3 * sizeof(float)));
  for (int i = 0; i < 2; ++i) o->X[i] = reinterpret_cast<__half*>(take(sizeof(__half) * batch * m * o->ldx));
  o->A = reinterpret_cast<__half*>(take(sizeof(__half) * batch * p * o->ldp));
  o->Bm = reinterpret_cast<__half*>(take(sizeof(__half) * batch * p * o->ldp));
  o->dA = reinterpret_cast<float2*>(take(sizeof(float2) * batch * o->ldp));
  o->rB = reinterpret_cast<float*>(take(sizeof(float) * batch * o->ldp));
  o->lo_product = p <= kBK;
  for (int i = 0; i < 2; ++i)
    o->L[i] = i && !o->lo_product ? o->L[0] : reinterpret_cast<__half*>(take(sizeof(__half) * batch * m * o->ldx));
  return at + 128;
}

// [batch, rows, cols] fp16 with row stride ld, boxes of 64 columns, 128-byte swizzle.
bool held_map(CUtensorMap* map, const void* ptr, int batch, int rows, int cols, int ld, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(rows) * ld * 2};
  cuuint32_t box[3] = {kLine, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;
// From this many values on, norm and scaling are launches of their own, with more threads an SM
// than the products leave them: 5 x 2560 x 1280 366 -> 355 us, and below the two launches cost more
// than they save (1280 x 2560 221 -> 225, 768 x 1024 110 -> 115).
constexpr int64_t kPrepareFrom = 4 << 20;

// Units (CTAs, or CTA pairs) of the kernel that are resident at once on the current device.
template <bool PAIR>
pg_status resident_units(int* units) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return PG_ERR_DEVICE;
  *units = known[dev].load(std::memory_order_relaxed);
  if (*units) return PG_OK;
  auto kern = ortho_kernel<PAIR>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(Tile<PAIR>::kSmem));
  if (e != cudaSuccess) return cuda_fail(e);
  int n = 0;
  if (PAIR) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * static_cast<unsigned>(sm_count()));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Tile<PAIR>::kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
  } else {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kThreads, Tile<PAIR>::kSmem);
    n = std::min(n, 1) * sm_count();
  }
  if (e != cudaSuccess) return cuda_fail(e);
  if (n < 1) return PG_ERR_DEVICE;
  known[dev].store(n, std::memory_order_relaxed);
  *units = n;
  return PG_OK;
}

template <bool PAIR>
pg_status launch_ortho(OrthoArgs g, cudaStream_t stream) {
  int units;
  pg_status st = resident_units<PAIR>(&units);
  if (st != PG_OK) return st;
  Maps maps;
  auto encode = [&](CUtensorMap (&X)[2], CUtensorMap& A, CUtensorMap& Bm, int box_rows) {
    return held_map(&X[0], g.X[0], g.batch, g.m, g.n, g.ldx, box_rows) &&
           held_map(&X[1], g.X[1], g.batch, g.m, g.n, g.ldx, box_rows) &&
           held_map(&A, g.A, g.batch, g.p, g.p, g.ldp, box_rows) && held_map(&Bm, g.Bm, g.batch, g.p, g.p, g.ldp, box_rows);
  };
  for (int i = 0; g.lo_product && i < 2; ++i)
    if (!held_map(&maps.L[i], g.L[i], g.batch, g.m, g.n, g.ldx, kRowsP)) return PG_ERR_CUDA;
  if (!encode(maps.X, maps.A, maps.Bm, kRowsP) || (!PAIR && !encode(maps.Xq, maps.Aq, maps.Bmq, Tile<false>::kRowsQ)))
    return PG_ERR_CUDA;
  g.tiles[0] = g.tiles[1] = tiles_of<PAIR>(g.p, g.p, true);
  g.tiles[2] = tiles_of<PAIR>(g.m, g.n, false);
  if (static_cast<int64_t>(g.steps) * g.batch * (g.tiles[0] + g.tiles[1] + g.tiles[2]) >= (1ll << 31)) return PG_ERR_SHAPE;
  // no more units than the widest phase has work for: the fewer blocks, the quicker they meet
  const int64_t tiles = static_cast<int64_t>(g.batch) * std::max(tiles_of<PAIR>(g.m, g.n, false), tiles_of<PAIR>(g.p, g.p, true));
  const int64_t piece = 8 * kThreads;  // what a block's threads read at a time in the norm and the scaling
  const int64_t reads = (static_cast<int64_t>(g.batch) * g.size + piece - 1) / piece;
  units = static_cast<int>(std::min<int64_t>(units, std::max(tiles, PAIR ? (reads + 1) / 2 : reads)));
  // one round of partial sums over the blocks
  g.prepared = static_cast<int64_t>(g.batch) * g.size >= kPrepareFrom;
  const int blocks = g.prepared ? 2 * sm_count() : (PAIR ? 2 : 1) * units;
  g.parts = static_cast<int>(std::min<int64_t>({kNormParts, std::max(1, blocks / g.batch), (g.size + piece - 1) / piece}));
  cudaError_t e = cudaMemsetAsync(g.ctrl, 0, ctrl_bytes(g.batch), stream);
  if (e != cudaSuccess) return cuda_fail(e);
  if (g.prepared) {
    const bool f32 = g.dtype == PG_F32;
    (f32 ? ortho_norm_kernel<PG_F32> : ortho_norm_kernel<PG_BF16>)<<<g.batch * g.parts, kPrepThreads, 0, stream>>>(g);
    if ((st = after_launch(1)) != PG_OK) return st;
    (f32 ? ortho_scale_kernel<PG_F32> : ortho_scale_kernel<PG_BF16>)<<<blocks, kPrepThreads, 0, stream>>>(g);
    if ((st = after_launch(1)) != PG_OK) return st;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PAIR ? 2 : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((PAIR ? 2u : 1u) * static_cast<unsigned>(units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tile<PAIR>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, ortho_kernel<PAIR>, maps, g);
  if (e != cudaSuccess) return cuda_fail(e);
  return after_launch(1);
}

// Whether 256 x 256 pair tiles finish sooner than 128 x 64 tiles. A step takes the k-blocks that a
// unit walks (those of one matrix alone, product after product, or all of them spread evenly,
// whichever is more) at 0.62 us each (a pair's MMAs) against 0.53 us (a single CTA's 48 KB from L2),
// and 6.4 us more for a pair's pipeline to fill and empty three times. Measured over 5 steps, pair
// and single, in us: 768 x 1024 158 / 110, 4 of them 166 / 140; 1280 x 1280 189 / 166; 1280 x 2560
// 222 / 222; 5 of 640 x 1280 169 / 145; 5 of 2560 x 1280 356 / 696.
bool use_pairs(const OrthoArgs& g, int sms) {
  const int q = std::max(g.m, g.n);
  auto step = [&](bool pair) {
    const int units = pair ? sms / 2 : sms;
    double alone = 0, all = 0;
    auto product = [&](int M, int N, int K, bool sym) {
      const int tiles = pair ? tiles_of<true>(M, N, sym) : tiles_of<false>(M, N, sym), blocks = (K + kBK - 1) / kBK;
      alone += static_cast<double>((tiles + units - 1) / units) * blocks;
      all += static_cast<double>(g.batch) * tiles * blocks / units;
    };
    product(g.p, g.p, q, true);
    product(g.p, g.p, g.p, true);
    product(g.m, g.n, g.p, false);
    return std::max(alone, all);
  };
  return 0.62 * step(true) + 6.4 < 0.53 * step(false);
}

}  // namespace

pg_status launch_ortho_wait_selftest(void* counters, int* gave_up, cudaStream_t stream) {
  ortho_wait_selftest_kernel<<<2, 64, 0, stream>>>(static_cast<OrthoCtrl*>(counters), gave_up, device_error_word());
  return after_launch(1);
}

}  // namespace pg

using namespace pg;

extern "C" pg_status pg_orthogonalize_workspace_size(int32_t batch, int32_t m, int32_t n, size_t* bytes) {
  if (!bytes) return PG_ERR_NULL;
  if (batch < 0 || batch > kMaxBatch || m < 1 || n < 1 || m > kMaxSide || n > kMaxSide) return PG_ERR_SHAPE;
  OrthoArgs o;
  *bytes = batch == 0 ? 0 : carve_ortho(nullptr, batch, m, n, &o);
  return PG_OK;
}

extern "C" pg_status pg_orthogonalize(const void* G, int32_t dtype, int32_t batch, int32_t m, int32_t n, int32_t steps,
                                      float a, float b, float c, float eps, float scale, void* out, void* workspace,
                                      size_t workspace_bytes, pg_stream_t stream) {
  size_t need;
  pg_status st = pg_orthogonalize_workspace_size(batch, m, n, &need);
  if (st != PG_OK) return st;
  if (steps < 1 || steps > 32) return PG_ERR_SHAPE;
  if (!real_dtype(dtype)) return PG_ERR_DTYPE;
  // a I is held as fp16 times 2^10: infinite from 64 on, whatever G is
  if (!(std::fabs(a) < 63.f) || !std::isfinite(b) || !std::isfinite(c)) return PG_ERR_UNSUPPORTED;
  if (batch == 0) return PG_OK;
  if (!G || !out) return PG_ERR_NULL;
  if (!aligned(G, dtype_bytes(dtype)) || !aligned(out, 2) || !aligned(workspace, 16)) return PG_ERR_ALIGN;
  if (workspace_bytes < need || !workspace) return PG_ERR_WORKSPACE;
  if (device_cc() != 103) return PG_ERR_DEVICE;

  OrthoArgs g = {};
  g.G = G;
  g.out = static_cast<__nv_bfloat16*>(out);
  g.err_word = device_error_word();
  g.size = static_cast<int64_t>(m) * n;
  g.batch = batch;
  g.m = m;
  g.n = n;
  g.p = std::min(m, n);
  carve_ortho(static_cast<uint8_t*>(workspace), batch, m, n, &g);
  g.steps = steps;
  g.dtype = dtype;
  g.g_vec = n % 8 == 0 && aligned(G, vec_bytes(dtype));
  g.out_vec = n % 8 == 0 && aligned(out, 16);
  g.a = a;
  g.b = b;
  g.c = c;
  g.eps = eps;
  g.scale = scale;
  return use_pairs(g, sm_count()) ? launch_ortho<true>(g, stream) : launch_ortho<false>(g, stream);
}
