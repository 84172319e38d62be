// Layer norm from the 8-bit normalised rows: the backward, and y again.
//
// 45360 x 4096 bf16: 191 and 101 us, 0.75 and 0.85 of the copy rate, bound by the
// instructions that decode next to HBM.  45360 x 1001 bf16: 131 and 68 us, 0.27
// and 0.31, 59 and 27 instructions of a warp for 32 elements: a shifted vector may
// hold elements of two blocks, so each pair takes its own scales.
#include "vda_layer_norm_bwd.cuh"

namespace vda {
namespace {

// y = xh w + b.
template <typename T, int VE, int NV, int kRows, bool kAsync, int F>
__global__ void __launch_bounds__(kThreads, ctas_of(NV * VE)) norm_apply_kernel(const NormArgs a) {
  constexpr int kChunks = NV / kOf<VE>, kSize = Chunk<VE>::kSize;
  extern __shared__ __align__(16) uint8_t ring[];
  const Place<VE, NV, F> p(a);
  const int nblk = (a.D + kBlock - 1) / kBlock;
  const Batch<uint8_t, VE, NV, kRows, kAsync> in(ring, a.codes, a);
  int sb[kRows][NV] = {}, next_sb[kRows][NV] = {};
  const int64_t span = (int64_t)p.groups * kRows, step = p.ctas * span;
  auto fetch = [&](int buf, int64_t row0) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      if (at < p.rows) {
        in.fetch(buf, r, a.codes + row * a.D, p);
        load_scales(a, row, nblk, p, next_sb[r]);
      }
    }
  };
  int64_t row0 = p.cta * span;
  fetch(0, row0);
  async_commit();
  Chunk<VE> w[kChunks], b[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    get_columns(a.W, a, p, c, 1.f, w[c]);
    get_columns(a.bias, a, p, c, 0.f, b[c]);
  }
  for (int buf = 0; row0 < p.rows; row0 += step, buf ^= 1) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int k = 0; k < NV; ++k) sb[r][k] = next_sb[r][k];
    fetch(buf ^ 1, row0 + step);
    async_commit();
    async_wait<1>();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
        if (at >= p.rows) continue;
        Chunk<VE> x;
        get_codes(in, buf, r, a.codes + row * a.D, p, sb[r], 1.f, c, x);
#pragma unroll
        for (int j = 0; j < kSize / 2; ++j) x.p[j] = fma2(x.p[j], w[c].p[j], b[c].p[j]);
        put_chunk(static_cast<T*>(a.Y) + row_at(a, row, a.ld_y), p, c, x);
      }
    }
  }
}

template <int kPass, typename T, int VE, int NV, int kRows, int F>
cudaError_t launch_pass(const NormArgs& a, const Shape& s, int grid, cudaStream_t st) {
  constexpr bool kAsync = VE > 1;
  if constexpr (kPass == kApply)
    return launch(norm_apply_kernel<T, VE, NV, kRows, kAsync, F>, grid, s.threads,
                  Batch<uint8_t, VE, NV, kRows, kAsync>::kBytes, a, st);
  else
    return launch_backward<T, VE, NV, kRows, F, true>(a, s, grid, st);
}

}  // namespace

cudaError_t launch_layer_norm_backward_from_checkpoint(const vda_norm_problem& p, const void* dY,
                                                       const uint8_t* codes, const uint8_t* scales, const float* rstd,
                                                       const void* W, void* dX, float* dW, float* db, float* partial,
                                                       cudaStream_t st) {
  NormArgs a = args_for(p);
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    a.dY = dY;
    a.W = W;
    a.Y = dX;
    a.rstd = const_cast<float*>(rstd);
    a.codes = const_cast<uint8_t*>(codes);
    a.scales = const_cast<uint8_t*>(scales);
    a.partial = dW || db ? partial : nullptr;
    e = run_pass<kBackwardCodes>(p.dtype, a, &parts, st);
  }
  return e == cudaSuccess && (dW || db) ? launch_norm_fold(p, partial, parts, dW, db, st) : e;
}

cudaError_t launch_layer_norm_from_checkpoint(const vda_norm_problem& p, const uint8_t* codes, const uint8_t* scales,
                                              const void* W, const void* bias, void* Y, cudaStream_t st) {
  NormArgs a = args_for(p);
  if (a.rows == 0) return cudaSuccess;
  a.W = W;
  a.bias = bias;
  a.Y = Y;
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  int ctas = 0;
  return run_pass<kApply>(p.dtype, a, &ctas, st);
}

}  // namespace vda
