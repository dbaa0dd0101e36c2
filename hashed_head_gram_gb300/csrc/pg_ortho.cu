// Orthogonalised updates by Newton-Schulz steps (pg_orthogonalize), for a batch of matrices.
//
// With p = min(m, n), q = max(m, n) and X [p, q] (G or its transpose, divided by its Frobenius
// norm), a step is three products:
//   A  = X X^T             [p, p], symmetric
//   Bm = b A + c A A       [p, p], symmetric
//   X  <- a X + Bm X       [p, q]
// Each is D = alpha P Q^T + beta C with P and Q row-major: X is kept in both orientations (XT
// [q, p] is the second operand of the last product), and the symmetric matrices are their own
// transposes. So one kernel does all three; it writes a tile where it belongs and, transposed,
// in the second array, which for the symmetric products is the mirrored tile of the same
// matrix: their tiles below the diagonal are never computed.
//
// Between the products X, A and Bm are held as fp16 scaled by 2^10 (pg.h): 11 significant
// bits, against the 8 of the bf16 result.
#include <cuda_fp16.h>

#include "pg_vec.cuh"

namespace pg {
namespace {

constexpr int kMaxSide = 16384;
constexpr int kMaxBatch = 4096;
constexpr float kHold = 1024.f;         // X, A and Bm are stored times 2^10
constexpr float kUnhold = 1.f / 1024.f;
constexpr int kNormBlocks = 64;         // blocks of partial sums per matrix, at most
constexpr int kTr = 32;                 // tile of the transposing passes

// Sums of squares over one matrix's share, of x, 2^64 x and 2^-64 x: whichever of the three
// neither overflows nor vanishes gives the norm.
__global__ void __launch_bounds__(256) ortho_norm_kernel(const void* __restrict__ G, int dtype, int64_t size,
                                                         float* __restrict__ partial) {
  __shared__ float s[3][8];
  const int64_t base = static_cast<int64_t>(blockIdx.y) * size;
  float sum[3] = {};
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < size; i += gridDim.x * 256ll) {
    float x[1];
    if (dtype == PG_F32)
      load_cols<PG_F32, 1>(G, base + i, x);
    else
      load_cols<PG_BF16, 1>(G, base + i, x);
    const float up = x[0] * 0x1p64f, down = x[0] * 0x1p-64f;
    sum[0] = fmaf(x[0], x[0], sum[0]);
    sum[1] = fmaf(up, up, sum[1]);
    sum[2] = fmaf(down, down, sum[2]);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
    if ((threadIdx.x & 31) == 0) s[k][threadIdx.x >> 5] = sum[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = 0.f;
    for (int w = 0; w < 8; ++w) t += s[threadIdx.x][w];
    partial[(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 3 + threadIdx.x] = t;
  }
}

// 2^10 / (|G|_F + eps) from the partial sums, added in their order.
__device__ __forceinline__ float held_scale(const float* partial, int parts, float eps) {
  float s[3] = {};
  for (int i = 0; i < parts; ++i)
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += partial[3 * i + k];
  float norm;
  if (s[0] > 0x1p-60f && s[0] < 0x1p120f)
    norm = sqrtf(s[0]);
  else if (s[0] <= 0x1p-60f)
    norm = sqrtf(s[1]) * 0x1p-64f;
  else
    norm = sqrtf(s[2]) * 0x1p64f;  // also NaN and infinities
  return kHold / (norm + eps);
}

// X0 in both orientations from G: dst[i, j] and dstT[j, i] of G's own orientation.
__global__ void __launch_bounds__(256) ortho_scale_kernel(const void* __restrict__ G, int dtype, int m, int n,
                                                          const float* __restrict__ partial, int parts, float eps,
                                                          __half* dst, int ld, int64_t dst_size, __half* dstT, int ldT,
                                                          int64_t dstT_size) {
  __shared__ float s_scale;
  __shared__ __half tile[kTr][kTr + 1];
  const int64_t b = blockIdx.z;
  if (threadIdx.x == 0) s_scale = held_scale(partial + b * parts * 3, parts, eps);
  __syncthreads();
  const float scale = s_scale;
  const int j0 = blockIdx.x * kTr, i0 = blockIdx.y * kTr;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  for (int r = ty; r < kTr; r += 8) {
    const int i = i0 + r, j = j0 + tx;
    if (i < m && j < n) {
      const int64_t at = (b * m + i) * n + j;
      float x[1];
      if (dtype == PG_F32)
        load_cols<PG_F32, 1>(G, at, x);
      else
        load_cols<PG_BF16, 1>(G, at, x);
      const __half h = __float2half_rn(x[0] * scale);
      tile[r][tx] = h;
      dst[b * dst_size + static_cast<int64_t>(i) * ld + j] = h;
    }
  }
  __syncthreads();
  for (int r = ty; r < kTr; r += 8) {
    const int j = j0 + r, i = i0 + tx;
    if (i < m && j < n) dstT[b * dstT_size + static_cast<int64_t>(j) * ldT + i] = tile[tx][r];
  }
}

// D = alpha P Q^T + beta C for one batch entry; see the top of the file.
struct Product {
  const __half* P;
  const __half* Q;
  const __half* C;       // laid out as D, or null
  __half* D;             // [M, N] (ld), null for the last product of the last step
  __half* DT;            // D transposed [N, M] (ldT); symmetric: D itself
  __nv_bfloat16* out;    // last product: scale * D, as [M, N] or, flip, [N, M], dense
  int64_t sP, sQ, sC, sD, sDT, sOut;  // batch strides, elements
  int ldP, ldQ, ldC, ldD, ldDT;
  int M, N, K;
  float alpha, beta, scale;
  int symmetric, flip;
};

constexpr int kSimt = 64;

__global__ void __launch_bounds__(256) ortho_product_kernel(const Product g) {
  if (g.symmetric && blockIdx.x < blockIdx.y) return;  // below the diagonal: the mirrored tile
  __shared__ float sp[16][kSimt + 1], sq[16][kSimt + 1];
  const int64_t b = blockIdx.z;
  const int i0 = blockIdx.y * kSimt, j0 = blockIdx.x * kSimt;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += 16) {
    for (int e = threadIdx.x; e < kSimt * 16; e += 256) {
      const int r = e >> 4, k = e & 15;
      sp[k][r] = i0 + r < g.M && k0 + k < g.K
                     ? __half2float(g.P[b * g.sP + static_cast<int64_t>(i0 + r) * g.ldP + k0 + k]) : 0.f;
      sq[k][r] = j0 + r < g.N && k0 + k < g.K
                     ? __half2float(g.Q[b * g.sQ + static_cast<int64_t>(j0 + r) * g.ldQ + k0 + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sp[k][ty + 16 * i], sq[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
      if (r >= g.M || c >= g.N) continue;
      float x = g.alpha * acc[i][j];
      if (g.C) x = fmaf(g.beta, __half2float(g.C[b * g.sC + static_cast<int64_t>(r) * g.ldC + c]), x);
      if (g.out) {
        g.out[b * g.sOut + (g.flip ? static_cast<int64_t>(c) * g.M + r : static_cast<int64_t>(r) * g.N + c)] =
            __float2bfloat16_rn(x * g.scale);
      } else {
        const __half h = __float2half_rn(x);
        g.D[b * g.sD + static_cast<int64_t>(r) * g.ldD + c] = h;
        if (!g.symmetric || blockIdx.x != blockIdx.y) g.DT[b * g.sDT + static_cast<int64_t>(c) * g.ldDT + r] = h;
      }
    }
}

struct OrthoBuffers {
  float* partial;
  __half *X[2], *XT[2], *A, *Bm;
  int ldq, ldp;  // row strides: q and p rounded up to 8 (16 bytes)
};

size_t carve_ortho(uint8_t* base, int64_t batch, int p, int q, OrthoBuffers* o) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* ptr = base ? base + at : nullptr;
    at += (bytes + 15) / 16 * 16;
    return ptr;
  };
  o->ldq = (q + 7) / 8 * 8;
  o->ldp = (p + 7) / 8 * 8;
  o->partial = reinterpret_cast<float*>(take(batch * kNormBlocks * 3 * sizeof(float)));
  for (int i = 0; i < 2; ++i) {
    o->X[i] = reinterpret_cast<__half*>(take(sizeof(__half) * batch * p * o->ldq));
    o->XT[i] = reinterpret_cast<__half*>(take(sizeof(__half) * batch * q * o->ldp));
  }
  o->A = reinterpret_cast<__half*>(take(sizeof(__half) * batch * p * o->ldp));
  o->Bm = reinterpret_cast<__half*>(take(sizeof(__half) * batch * p * o->ldp));
  return at;
}

pg_status launch_product(const Product& g, int batch, cudaStream_t stream) {
  const dim3 grid((g.N + kSimt - 1) / kSimt, (g.M + kSimt - 1) / kSimt, batch);
  ortho_product_kernel<<<grid, 256, 0, stream>>>(g);
  return after_launch(1);
}

}  // namespace
}  // namespace pg

using namespace pg;

extern "C" pg_status pg_orthogonalize_workspace_size(int32_t batch, int32_t m, int32_t n, size_t* bytes) {
  if (!bytes) return PG_ERR_NULL;
  if (batch < 0 || batch > kMaxBatch || m < 1 || n < 1 || m > kMaxSide || n > kMaxSide) return PG_ERR_SHAPE;
  OrthoBuffers o;
  *bytes = batch == 0 ? 0 : carve_ortho(nullptr, batch, m < n ? m : n, m < n ? n : m, &o);
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
  if (batch == 0) return PG_OK;
  if (!G || !out) return PG_ERR_NULL;
  if (!aligned(G, dtype_bytes(dtype)) || !aligned(out, 2) || !aligned(workspace, 16)) return PG_ERR_ALIGN;
  if (workspace_bytes < need || !workspace) return PG_ERR_WORKSPACE;
  if (device_cc() != 103) return PG_ERR_DEVICE;

  const bool flip = m > n;  // X = G^T
  const int p = flip ? n : m, q = flip ? m : n;
  OrthoBuffers o;
  carve_ortho(static_cast<uint8_t*>(workspace), batch, p, q, &o);
  const int64_t sX = static_cast<int64_t>(p) * o.ldq, sXT = static_cast<int64_t>(q) * o.ldp;
  const int64_t sA = static_cast<int64_t>(p) * o.ldp, size = static_cast<int64_t>(m) * n;
  const int parts = static_cast<int>(min(static_cast<int64_t>(kNormBlocks), (size + 4095) / 4096));
  ortho_norm_kernel<<<dim3(parts, batch), 256, 0, stream>>>(G, dtype, size, o.partial);
  st = after_launch(1);
  if (st != PG_OK) return st;
  ortho_scale_kernel<<<dim3((n + kTr - 1) / kTr, (m + kTr - 1) / kTr, batch), 256, 0, stream>>>(
      G, dtype, m, n, o.partial, parts, eps, flip ? o.XT[0] : o.X[0], flip ? o.ldp : o.ldq, flip ? sXT : sX,
      flip ? o.X[0] : o.XT[0], flip ? o.ldq : o.ldp, flip ? sX : sXT);
  st = after_launch(1);
  if (st != PG_OK) return st;

  int cur = 0;
  for (int s = 0; s < steps; ++s) {
    Product g = {};
    // A = X X^T
    g.P = g.Q = o.X[cur];
    g.sP = g.sQ = sX;
    g.ldP = g.ldQ = o.ldq;
    g.D = g.DT = o.A;
    g.sD = g.sDT = sA;
    g.ldD = g.ldDT = o.ldp;
    g.M = g.N = p;
    g.K = q;
    g.alpha = kUnhold;
    g.symmetric = 1;
    if ((st = launch_product(g, batch, stream)) != PG_OK) return st;
    // Bm = b A + c A A
    g.P = g.Q = g.C = o.A;
    g.sP = g.sQ = g.sC = sA;
    g.ldP = g.ldQ = g.ldC = o.ldp;
    g.D = g.DT = o.Bm;
    g.K = p;
    g.alpha = c * kUnhold;
    g.beta = b;
    if ((st = launch_product(g, batch, stream)) != PG_OK) return st;
    // X <- a X + Bm X
    g.P = o.Bm;
    g.Q = o.XT[cur];
    g.sQ = sXT;
    g.C = o.X[cur];
    g.sC = sX;
    g.ldC = o.ldq;
    g.D = o.X[cur ^ 1];
    g.sD = sX;
    g.ldD = o.ldq;
    g.DT = o.XT[cur ^ 1];
    g.sDT = sXT;
    g.ldDT = o.ldp;
    g.N = q;
    g.alpha = kUnhold;
    g.beta = a;
    g.symmetric = 0;
    if (s + 1 == steps) {
      g.D = g.DT = nullptr;
      g.out = static_cast<__nv_bfloat16*>(out);
      g.sOut = size;
      g.scale = scale * kUnhold;
      g.flip = flip;
    }
    if ((st = launch_product(g, batch, stream)) != PG_OK) return st;
    cur ^= 1;
  }
  return PG_OK;
}
