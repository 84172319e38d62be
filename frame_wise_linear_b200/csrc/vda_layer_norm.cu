// Layer norm over the last dimension, forward and backward, optionally with
// the normalised row kept in 8 bits for the backward.
//
//   forward    m = sum x / D, r = 1 / sqrt(sum (x - m)^2 / D + eps),
//              xh = (x - m) r, y = xh w + b
//   backward   g = dy w, dx = r (g - mean(g) - xh mean(g xh)),
//              dw = sum over rows of dy xh, db = sum over rows of dy
//
// Both are bound by HBM: a row is read once, stays in registers between its
// sums and its outputs, and is written once.  A row belongs to `tpr` threads,
// each with 8 of its elements (one 16-byte vector of bf16, two of float32, or
// 8 single elements where the row is not 16-byte aligned); up to 32 threads a
// row is summed by shuffles, above that through shared memory.  The variance
// is the mean of the squared differences from the mean that is already known
// (two sums, no cancellation).  Everything is float32; an output is rounded
// once.
//
// The gradients of w and b are sums over all rows.  A thread holds the same
// columns of every row that its CTA takes, so it keeps their sums in
// registers; each CTA writes one row of partial sums, and a second kernel
// adds those rows in a fixed order (no atomics: the result does not depend on
// the order in which CTAs run).
#include "vda_internal.cuh"
#include "vda_tokops.cuh"

namespace vda {
namespace {

using namespace tokops;

constexpr int kPer = 8;   // elements of a row that one thread holds

struct NormArgs {
  const void* X;       // forward: input; backward: input (or null: codes)
  const void* dY;      // backward
  const void* W;       // or null
  const void* bias;    // or null
  void* Y;             // forward: Y; backward: dX
  float* mean;         // forward: written (or null); backward: read
  float* rstd;
  uint8_t* codes;      // forward: written (or null); backward: read (or null)
  uint8_t* scales;
  float* partial;      // backward: [gridDim.x][2 D] (dw then db), or null
  int64_t tokens, ld_x, ld_y;   // ld_x: X (and dX); ld_y: Y, dY
  int heads, D, tpr;
  float eps, inv_d;
  int w_bf16;
};

__device__ __forceinline__ float load_w(const void* w, int i, int w_bf16) {
  return w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}

// A row's place: token and head, advanced by a fixed number of rows.
struct RowPos {
  int64_t row, tok;
  int head;
  __device__ __forceinline__ RowPos(int64_t r, int heads) : row(r) {
    if (heads == 1) {
      tok = r;
      head = 0;
    } else {
      tok = r / heads;
      head = (int)(r - tok * heads);
    }
  }
  __device__ __forceinline__ void advance(int64_t by, int64_t dtok, int dhead, int heads) {
    row += by;
    tok += dtok;
    head += dhead;
    if (head >= heads) {
      head -= heads;
      ++tok;
    }
  }
};

// Sums of v over the threads of a row; every thread gets them.  Rows of up to
// 32 threads: shuffles.  Above: the row's warps leave their sums in one half
// of `red` (the halves alternate from call to call, so one barrier a call is
// enough), and every thread adds them in the same order.
struct RowSum {
  float2* red;   // [2][32]
  int tpr, warps, first, half;
  __device__ __forceinline__ RowSum(float2* r, int t) : red(r), tpr(t), half(0) {
    warps = t >> 5;
    first = warps ? ((int)threadIdx.x / t) * warps : 0;
  }
  __device__ __forceinline__ float2 operator()(float2 v) {
    for (int o = (tpr < 32 ? tpr : 32) / 2; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (tpr <= 32) return v;
    float2* r = red + half * 32;
    half ^= 1;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = r[first];
    for (int i = 1; i < warps; ++i) {
      const float2 o = r[first + i];
      v.x += o.x;
      v.y += o.y;
    }
    return v;
  }
};

// Vectors of VE elements, NV = kPer / VE a thread: vector k of thread t of a
// row is number t + k tpr.
template <typename T, int VE>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormArgs a) {
  constexpr int NV = kPer / VE;
  __shared__ float2 red[64];
  const int t = (int)threadIdx.x % a.tpr, group = (int)threadIdx.x / a.tpr;
  const int groups = (int)blockDim.x / a.tpr;
  const int nvec = a.D / VE, nblk = (a.D + kBlock - 1) / kBlock;
  float w[kPer], b[kPer];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const int v = t + k * a.tpr, c = v * VE + i;
      w[k * VE + i] = a.W && v < nvec ? load_w(a.W, c, a.w_bf16) : 1.f;
      b[k * VE + i] = a.bias && v < nvec ? load_w(a.bias, c, a.w_bf16) : 0.f;
    }
  RowSum sum(red, a.tpr);
  const int64_t rows = a.tokens * a.heads, by = (int64_t)gridDim.x * groups;
  const int64_t dtok = by / a.heads;
  const int dhead = (int)(by - dtok * a.heads);
  RowPos p((int64_t)blockIdx.x * groups + group, a.heads);
  // Every thread of the block makes the same number of trips: the sums and
  // the block maxima need them all.
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < rows; r0 += by) {
    const bool live = p.row < rows;
    const T* xr = static_cast<const T*>(a.X) + p.tok * a.ld_x + (int64_t)p.head * a.D;
    float x[kPer];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = t + k * a.tpr;
      Pack<T, VE> q;
      if (live && v < nvec) q.load(xr + (int64_t)v * VE);
      else q.zero();
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        x[k * VE + i] = q.get(i);
        s.x += x[k * VE + i];
      }
    }
    const float mean = sum(s).x * a.inv_d;
    s.x = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const bool in = t + k * a.tpr < nvec;
        x[k * VE + i] = in ? x[k * VE + i] - mean : 0.f;
        s.x += x[k * VE + i] * x[k * VE + i];
      }
    const float rstd = 1.f / sqrtf(sum(s).x * a.inv_d + a.eps);
    T* yr = static_cast<T*>(a.Y) + p.tok * a.ld_y + (int64_t)p.head * a.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = t + k * a.tpr;
      const bool in = live && v < nvec;
      Pack<T, VE> q;
      float xh[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        xh[i] = x[k * VE + i] * rstd;
        q.set(i, xh[i] * w[k * VE + i] + b[k * VE + i]);
      }
      if (in) q.store(yr + (int64_t)v * VE);
      if (a.codes) {
        // A thread without this vector adds nothing to the block's maximum.
        if (!in) {
#pragma unroll
          for (int i = 0; i < VE; ++i) xh[i] = 0.f;
        }
        uint8_t c[VE];
        const int sb = encode_block<VE>(xh, c);
        if (in) {
          store_codes<VE>(a.codes + p.row * a.D + (int64_t)v * VE, c);
          if (v % (kBlock / VE) == 0) a.scales[p.row * nblk + v / (kBlock / VE)] = (uint8_t)sb;
        }
      }
    }
    if (live && t == 0) {
      if (a.mean) a.mean[p.row] = mean;
      if (a.rstd) a.rstd[p.row] = rstd;
    }
    p.advance(by, dtok, dhead, a.heads);
  }
}

// The backward: X with mean and rstd, or (kCodes) the 8-bit normalised row
// with rstd.  Writes dX, and with a.partial the CTA's sums of dy xh and dy.
template <typename T, int VE, bool kCodes>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const NormArgs a) {
  constexpr int NV = kPer / VE;
  extern __shared__ float fold[];   // groups > 1: [groups][2 D]
  __shared__ float2 red[64];
  const int t = (int)threadIdx.x % a.tpr, group = (int)threadIdx.x / a.tpr;
  const int groups = (int)blockDim.x / a.tpr;
  const int nvec = a.D / VE, nblk = (a.D + kBlock - 1) / kBlock;
  float w[kPer], dw[kPer], db[kPer];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const int v = t + k * a.tpr;
      w[k * VE + i] = a.W && v < nvec ? load_w(a.W, v * VE + i, a.w_bf16) : 1.f;
      dw[k * VE + i] = db[k * VE + i] = 0.f;
    }
  RowSum sum(red, a.tpr);
  const int64_t rows = a.tokens * a.heads, by = (int64_t)gridDim.x * groups;
  const int64_t dtok = by / a.heads;
  const int dhead = (int)(by - dtok * a.heads);
  RowPos p((int64_t)blockIdx.x * groups + group, a.heads);
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < rows; r0 += by) {
    const bool live = p.row < rows;
    const int64_t at_x = p.tok * a.ld_x + (int64_t)p.head * a.D, at_y = p.tok * a.ld_y + (int64_t)p.head * a.D;
    const float mean = !kCodes && live ? a.mean[p.row] : 0.f, rstd = live ? a.rstd[p.row] : 0.f;
    float g[kPer], xh[kPer];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = t + k * a.tpr;
      const bool in = live && v < nvec;
      Pack<T, VE> q;
      if (in) q.load(static_cast<const T*>(a.dY) + at_y + (int64_t)v * VE);
      else q.zero();
      float x[VE];
      if constexpr (kCodes) {
        CodePack<VE> c;
        float sc = 0.f;
        if (in) {
          c.load(a.codes + p.row * a.D + (int64_t)v * VE);
          sc = scale_of(a.scales[p.row * nblk + v / (kBlock / VE)]);
          c.values(sc, x);
        }
      } else {
        Pack<T, VE> u;
        if (in) {
          u.load(static_cast<const T*>(a.X) + at_x + (int64_t)v * VE);
#pragma unroll
          for (int i = 0; i < VE; ++i) x[i] = (u.get(i) - mean) * rstd;
        }
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const int e = k * VE + i;
        const float dy = q.get(i);
        xh[e] = in ? x[i] : 0.f;
        g[e] = dy * w[e];
        dw[e] += dy * xh[e];
        db[e] += dy;
        s.x += g[e];
        s.y += g[e] * xh[e];
      }
    }
    s = sum(s);
    s.x *= a.inv_d;
    s.y *= a.inv_d;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = t + k * a.tpr;
      Pack<T, VE> q;
#pragma unroll
      for (int i = 0; i < VE; ++i) q.set(i, rstd * (g[k * VE + i] - s.x - xh[k * VE + i] * s.y));
      if (live && v < nvec) q.store(static_cast<T*>(a.Y) + at_x + (int64_t)v * VE);
    }
    p.advance(by, dtok, dhead, a.heads);
  }
  if (!a.partial) return;
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.D;
  if (groups > 1) out = fold + (int64_t)group * 2 * a.D;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = t + k * a.tpr;
    if (v < nvec) {
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        out[v * VE + i] = dw[k * VE + i];
        out[a.D + v * VE + i] = db[k * VE + i];
      }
    }
  }
  if (groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += blockDim.x) {
      float v = 0.f;
      for (int q = 0; q < groups; ++q) v += fold[q * 2 * a.D + c];
      a.partial[(int64_t)blockIdx.x * 2 * a.D + c] = v;
    }
  }
}

// dW and db from the CTAs' partial sums [parts][2 D]: 32 columns a block,
// thread (x, y) adds rows y, y + 8, ...; then the 8 sums of a column in order.
__global__ void __launch_bounds__(256) norm_fold_kernel(const float* partial, int parts, int D, float* dW, float* db) {
  __shared__ float sh[8][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float v = 0.f;
  if (c < 2 * D)
    for (int i = y; i < parts; i += 8) v += partial[(int64_t)i * 2 * D + c];
  sh[y][x] = v;
  __syncthreads();
  if (y == 0 && c < 2 * D) {
    for (int i = 1; i < 8; ++i) v += sh[i][x];
    if (c < D) {
      if (dW) dW[c] = v;
    } else if (db) {
      db[c - D] = v;
    }
  }
}

// y = xh w + b from the 8-bit normalised rows.
template <typename T, int VE>
__global__ void __launch_bounds__(1024) norm_apply_kernel(const NormArgs a) {
  constexpr int NV = kPer / VE;
  const int t = (int)threadIdx.x % a.tpr, group = (int)threadIdx.x / a.tpr;
  const int groups = (int)blockDim.x / a.tpr;
  const int nvec = a.D / VE, nblk = (a.D + kBlock - 1) / kBlock;
  float w[kPer], b[kPer];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const int v = t + k * a.tpr, c = v * VE + i;
      w[k * VE + i] = a.W && v < nvec ? load_w(a.W, c, a.w_bf16) : 1.f;
      b[k * VE + i] = a.bias && v < nvec ? load_w(a.bias, c, a.w_bf16) : 0.f;
    }
  const int64_t rows = a.tokens * a.heads, by = (int64_t)gridDim.x * groups;
  const int64_t dtok = by / a.heads;
  const int dhead = (int)(by - dtok * a.heads);
  RowPos p((int64_t)blockIdx.x * groups + group, a.heads);
  for (; p.row < rows; p.advance(by, dtok, dhead, a.heads)) {
    T* yr = static_cast<T*>(a.Y) + p.tok * a.ld_y + (int64_t)p.head * a.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = t + k * a.tpr;
      if (v >= nvec) continue;
      CodePack<VE> c;
      float x[VE];
      c.load(a.codes + p.row * a.D + (int64_t)v * VE);
      c.values(scale_of(a.scales[p.row * nblk + v / (kBlock / VE)]), x);
      Pack<T, VE> q;
#pragma unroll
      for (int i = 0; i < VE; ++i) q.set(i, x[i] * w[k * VE + i] + b[k * VE + i]);
      q.store(yr + (int64_t)v * VE);
    }
  }
}

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Threads of a row and of a block, and rows of a block.  A row takes as many
// threads as it has groups of 8 elements: a power of two up to 32 (at least
// the lanes of one 32-element block of codes), or whole warps.
struct Shape {
  int tpr, threads, groups;
};
Shape shape_for(int D, int ve) {
  const int need = ((D + ve - 1) / ve + kPer / ve - 1) / (kPer / ve);
  int tpr = kBlock / ve;
  while (tpr < 32 && tpr < need) tpr *= 2;
  if (need > 32) tpr = (need + 31) / 32 * 32;
  const int groups = tpr >= 256 ? 1 : 256 / tpr;
  return Shape{tpr, tpr * groups, groups};
}

// CTAs for `rows` rows: enough for every SM to hold 2048 threads' worth, or
// fewer where there are fewer rows.
int grid_for(int64_t rows, const Shape& s) {
  const int64_t blocks = (rows + s.groups - 1) / s.groups;
  const int64_t most = 148 * (s.threads > 1024 ? 1 : 1024 / s.threads);
  return (int)(blocks < most ? blocks : most);
}

// 16-byte vectors where the width, the strides and the pointers allow them.
template <typename T>
bool wide(const NormArgs& a) {
  const int ve = 16 / (int)sizeof(T);
  const bool c = !a.codes || (aligned_to(a.codes, ve) && a.D % ve == 0);
  return c && a.D % ve == 0 && a.ld_x % ve == 0 && a.ld_y % ve == 0 && aligned_to(a.X, 16) && aligned_to(a.dY, 16) &&
         aligned_to(a.Y, 16);
}

template <typename T, int VE>
cudaError_t fwd(NormArgs a, cudaStream_t st) {
  const Shape s = shape_for(a.D, VE);
  a.tpr = s.tpr;
  norm_fwd_kernel<T, VE><<<grid_for(a.tokens * a.heads, s), s.threads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int VE>
cudaError_t bwd(NormArgs a, float* dW, float* db, cudaStream_t st) {
  const Shape s = shape_for(a.D, VE);
  a.tpr = s.tpr;
  const int grid = grid_for(a.tokens * a.heads, s);
  const size_t sh = a.partial && s.groups > 1 ? (size_t)s.groups * 2 * a.D * sizeof(float) : 0;
  if (a.codes) norm_bwd_kernel<T, VE, true><<<grid, s.threads, sh, st>>>(a);
  else norm_bwd_kernel<T, VE, false><<<grid, s.threads, sh, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  norm_fold_kernel<<<(2 * a.D + 31) / 32, 256, 0, st>>>(a.partial, grid, a.D, dW, db);
  return cudaGetLastError();
}

template <typename T, int VE>
cudaError_t apply(NormArgs a, cudaStream_t st) {
  const Shape s = shape_for(a.D, VE);
  a.tpr = s.tpr;
  norm_apply_kernel<T, VE><<<grid_for(a.tokens * a.heads, s), s.threads, 0, st>>>(a);
  return cudaGetLastError();
}

NormArgs args_for(const vda_norm_problem& p) {
  NormArgs a{};
  a.tokens = p.tokens;
  a.heads = p.heads;
  a.D = p.D;
  a.ld_x = p.ld_x ? p.ld_x : (int64_t)p.heads * p.D;
  a.ld_y = p.ld_y ? p.ld_y : (int64_t)p.heads * p.D;
  // Tokens without gaps are rows like any others.
  if (a.ld_x == (int64_t)p.heads * p.D && a.ld_y == a.ld_x) {
    a.tokens *= p.heads;
    a.heads = 1;
    a.ld_x = a.ld_y = p.D;
  }
  a.eps = p.eps;
  a.inv_d = 1.f / (float)p.D;
  a.w_bf16 = p.w_dtype == VDA_DTYPE_BF16;
  return a;
}

}  // namespace

// The partial sums' rows: as many as CTAs, whichever variant runs.
size_t norm_backward_workspace_bytes(const vda_norm_problem& p) {
  const int64_t rows = p.tokens * p.heads;
  if (rows == 0) return 0;
  int parts = 0;
  for (int ve : {1, 4, 8}) {
    const int g = grid_for(rows, shape_for(p.D, ve));
    parts = g > parts ? g : parts;
  }
  return align_up((size_t)parts * 2 * p.D * sizeof(float), 256);
}

cudaError_t launch_layer_norm(const vda_norm_problem& p, const void* X, const void* W, const void* bias, void* Y,
                              float* mean, float* rstd, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  NormArgs a = args_for(p);
  if (a.tokens == 0) return cudaSuccess;
  a.X = X;
  a.W = W;
  a.bias = bias;
  a.Y = Y;
  a.mean = mean;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  if (p.dtype == VDA_DTYPE_BF16)
    return wide<__nv_bfloat16>(a) ? fwd<__nv_bfloat16, 8>(a, st) : fwd<__nv_bfloat16, 1>(a, st);
  return wide<float>(a) ? fwd<float, 4>(a, st) : fwd<float, 1>(a, st);
}

cudaError_t launch_layer_norm_backward(const vda_norm_problem& p, const void* dY, const void* X, const float* mean,
                                       const float* rstd, const uint8_t* codes, const uint8_t* scales, const void* W,
                                       void* dX, float* dW, float* db, float* partial, cudaStream_t st) {
  NormArgs a = args_for(p);
  if (a.tokens == 0) {
    cudaError_t e = dW ? cudaMemsetAsync(dW, 0, (size_t)p.D * sizeof(float), st) : cudaSuccess;
    if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)p.D * sizeof(float), st);
    return e;
  }
  a.X = X;
  a.dY = dY;
  a.W = W;
  a.Y = dX;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.partial = dW || db ? partial : nullptr;
  if (p.dtype == VDA_DTYPE_BF16)
    return wide<__nv_bfloat16>(a) ? bwd<__nv_bfloat16, 8>(a, dW, db, st) : bwd<__nv_bfloat16, 1>(a, dW, db, st);
  return wide<float>(a) ? bwd<float, 4>(a, dW, db, st) : bwd<float, 1>(a, dW, db, st);
}

cudaError_t launch_layer_norm_from_checkpoint(const vda_norm_problem& p, const uint8_t* codes, const uint8_t* scales,
                                              const void* W, const void* bias, void* Y, cudaStream_t st) {
  NormArgs a = args_for(p);
  if (a.tokens == 0) return cudaSuccess;
  a.W = W;
  a.bias = bias;
  a.Y = Y;
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  if (p.dtype == VDA_DTYPE_BF16)
    return wide<__nv_bfloat16>(a) ? apply<__nv_bfloat16, 8>(a, st) : apply<__nv_bfloat16, 1>(a, st);
  return wide<float>(a) ? apply<float, 4>(a, st) : apply<float, 1>(a, st);
}

}  // namespace vda
