// Layer norm's backward from X, and the last sum of the weights' gradients.
#include "vda_layer_norm_bwd.cuh"

namespace vda {
namespace {

template <int kPass, typename T, int VE, int NV, int kRows, int F>
cudaError_t launch_pass(const NormArgs& a, const Shape& s, int grid, cudaStream_t st) {
  return launch_backward<T, VE, NV, kRows, F, false>(a, s, grid, st);
}

// dW and db from the CTAs' partial sums [parts][2 D]: 32 columns a block,
// thread (x, y) adds rows y, y + 32, ...; then a warp the 32 sums of a column.
// The rows come from L2, and there are at most kMostParts of them: a thread's
// loads are all on their way before the first is added (296 rows of 2002
// columns: 4.6 us one after the other).
constexpr int kMostParts = 320;
static_assert(kMostParts >= 148 * ctas_of(16) && kMostParts % 32 == 0, "every CTA's row is added");
__global__ void __launch_bounds__(1024) norm_fold_kernel(const float* partial, int parts, int D, float* dW, float* db) {
  __shared__ float sh[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  cudaGridDependencySynchronize();
  float part[kMostParts / 32];
#pragma unroll
  for (int j = 0; j < kMostParts / 32; ++j) {
    const int i = y + j * 32;
    part[j] = c < 2 * D && i < parts ? partial[(int64_t)i * 2 * D + c] : 0.f;
  }
  float v = part[0];
#pragma unroll
  for (int j = 1; j < kMostParts / 32; ++j) v += part[j];
  sh[y][x] = v;
  __syncthreads();
  // Warp y adds column y's 32 sums.
  v = sh[x][y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + y;
  if (x == 0 && col < 2 * D) {
    if (col < D) {
      if (dW) dW[col] = v;
    } else if (db) {
      db[col - D] = v;
    }
  }
}

}  // namespace

// The partial sums' rows: as many as CTAs, whichever variant runs.
size_t norm_backward_workspace_bytes(const vda_norm_problem& p) {
  const int64_t rows = p.tokens * p.heads;
  if (rows == 0) return 0;
  int parts = 0;
  for (int ve : {1, 4, 8})
    for (int kinds : {0, ve > 1 ? kinds_for(p.D, ve, rows) : 0}) {
      const Shape s = shape_for(p.D, ve, kinds);
      const int g = s.groups ? grid_for(rows, s, 1) : 0;
      parts = g > parts ? g : parts;
    }
  return align_up((size_t)parts * 2 * p.D * sizeof(float), 256);
}

cudaError_t launch_norm_fold(const vda_norm_problem& p, const float* partial, int parts, float* dW, float* db,
                             cudaStream_t st) {
  if (p.tokens == 0) {   // no rows: the sums are 0
    cudaError_t e = dW ? cudaMemsetAsync(dW, 0, (size_t)p.D * sizeof(float), st) : cudaSuccess;
    if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)p.D * sizeof(float), st);
    return e;
  }
  // Launched while the pass over the rows still runs (4097 x 1001 float32, both:
  // 21.3 us a call against 22.6).
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((2 * p.D + 31) / 32));
  c.blockDim = dim3(1024);
  c.stream = st;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, norm_fold_kernel, partial, parts, (int)p.D, dW, db);
}

cudaError_t launch_layer_norm_backward(const vda_norm_problem& p, const void* dY, const void* X, const float* mean,
                                       const float* rstd, const void* W, void* dX, float* dW, float* db,
                                       float* partial, cudaStream_t st) {
  NormArgs a = args_for(p);
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    a.X = X;
    a.dY = dY;
    a.W = W;
    a.Y = dX;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.partial = dW || db ? partial : nullptr;
    e = run_pass<kBackward>(p.dtype, a, &parts, st);
  }
  return e == cudaSuccess && (dW || db) ? launch_norm_fold(p, partial, parts, dW, db, st) : e;
}

}  // namespace vda
