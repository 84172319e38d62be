// Layer norm's backward kernel (vda_layer_norm.cuh has the plan), for the two
// files that compile it: from X (vda_layer_norm_bwd.cu) and from the 8-bit
// normalised rows (vda_layer_norm_ckpt.cu).
#pragma once

#include "vda_layer_norm.cuh"

namespace vda {
namespace {

// The columns of a thread to a row of sums in global or shared memory (16-byte
// aligned where rows are vectors of 4 or 8).
template <int VE, int NV, int F>
__device__ __forceinline__ void put_columns(float* to, const Place<VE, NV, F>& p, int c, const Chunk<VE>& v) {
  if constexpr (VE > 1 && F != kShift) {
    if (!p.has(c)) return;
#pragma unroll
    for (int j = 0; j < VE; j += 4)
      *reinterpret_cast<float4*>(to + p.col(c) + j) =
          make_float4(v.p[j / 2].x, v.p[j / 2].y, v.p[j / 2 + 1].x, v.p[j / 2 + 1].y);
  } else {
#pragma unroll
    for (int k = 0; k < kOf<VE>; ++k)
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (p.in(c * kOf<VE> + k, i)) to[p.col(c * kOf<VE> + k) + i] = v.get(k * VE + i);
  }
}

// X with mean and rstd, or (kCodes) the 8-bit normalised row with rstd.  Writes
// dX, and with a.partial the CTA's sums of dy xh and dy.  A batch's elements
// are read twice from shared memory, for the sums and for dX: kept in
// registers they would cost 32 a row, and the occupancy with them.
template <typename T, int VE, int NV, int kRows, bool kAsync, int F, bool kCodes>
__global__ void __launch_bounds__(kThreads, ctas_of(NV * VE)) norm_bwd_kernel(const NormArgs a) {
  constexpr int kChunks = NV / kOf<VE>, kSize = Chunk<VE>::kSize, kSb = kCodes ? NV : 1;
  using U = typename std::conditional<kCodes, uint8_t, T>::type;   // what xh comes from
  using InY = Batch<T, VE, NV, kRows, kAsync>;
  using InX = Batch<U, VE, NV, kRows, kAsync>;
  extern __shared__ __align__(16) uint8_t ring[];   // afterwards: groups > 1: [groups][2 D] partial sums
  __shared__ float red[2][2 * kRows][kThreads / 32];
  const Place<VE, NV, F> p(a);
  const int nblk = (a.D + kBlock - 1) / kBlock;
  const T* dY = static_cast<const T*>(a.dY);
  const U* X = kCodes ? reinterpret_cast<const U*>(a.codes) : static_cast<const U*>(a.X);
  const InY iny(ring, dY, a);
  const InX inx(ring + InY::kBytes, X, a);
  auto x_at = [&](int64_t row) { return kCodes ? row * a.D : row_at(a, row, a.ld_x); };
  // rstd, and mean or the scale bytes, of the batch that is worked on and of
  // the next: loaded with it, so that they too are there when it is.
  float mean[kRows] = {}, rstd[kRows] = {}, next_mean[kRows] = {}, next_rstd[kRows] = {};
  int sb[kRows][kSb] = {}, next_sb[kRows][kSb] = {};
  const int64_t span = (int64_t)p.groups * kRows, step = p.ctas * span;
  auto fetch = [&](int buf, int64_t row0, auto whole) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      if (decltype(whole)::value || at < p.rows) {
        iny.fetch(buf, r, dY + row_at(a, row, a.ld_y), p);
        inx.fetch(buf, r, X + x_at(row), p);
        next_rstd[r] = a.rstd[row];
        if constexpr (kCodes) load_scales(a, row, nblk, p, next_sb[r]);
        else next_mean[r] = a.mean[row];
      }
    }
  };
  // Chunk c of dy, and of xh (of codes: times `by`), of row r.
  auto get = [&](int buf, int r, int64_t row, float by, int c, Chunk<VE>& dy, Chunk<VE>& xh) {
    get_chunk(iny, buf, r, dY + row_at(a, row, a.ld_y), p, c, dy);
    if constexpr (kCodes) {
      get_codes(inx, buf, r, X + x_at(row), p, sb[r], by, c, xh);
    } else {
      get_plus(inx, buf, r, X + x_at(row), p, c, -mean[r], xh);
      // Where a vector is missing x is 0, and -mean rstd overflows for constant
      // rows from 3.4e38 sqrt(eps) up.
#pragma unroll
      for (int j = 0; j < kSize / 2; ++j) {
        const int k = VE > 1 ? c : 2 * c, k1 = VE > 1 ? c : 2 * c + 1;
        const float2 rs = F != kSome ? both(rstd[r]) : make_float2(p.has(k) ? rstd[r] : 0.f, p.has(k1) ? rstd[r] : 0.f);
        xh.p[j] = mul2(xh.p[j], rs);
      }
    }
  };
  // The last sum may be launched from here on; it waits for this grid's end.
  cudaTriggerProgrammaticLaunchCompletion();
  int64_t row0 = p.cta * span;
  fetch(0, row0, std::false_type());
  async_commit();
  Chunk<VE> w[kChunks], dw[kChunks], db[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) get_columns(a.W, a, p, c, 1.f, w[c]);
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < kSize / 2; ++j) dw[c].p[j] = db[c].p[j] = both(0.f);
  auto body = [&](int buf, int64_t row0, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    float2 s1[kRows], s2[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) s1[r] = s2[r] = both(0.f);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
        if (!kWhole && at >= p.rows) continue;
        Chunk<VE> dy, xh;
        get(buf, r, row, 1.f, c, dy, xh);
        // Where the thread has no element dy is 0 and xh finite: nothing is added.
#pragma unroll
        for (int j = 0; j < kSize / 2; ++j) {
          const float2 t = mul2(dy.p[j], xh.p[j]);
          dw[c].p[j] = add2(dw[c].p[j], t);
          db[c].p[j] = add2(db[c].p[j], dy.p[j]);
          s1[r] = fma2(dy.p[j], w[c].p[j], s1[r]);
          s2[r] = fma2(t, w[c].p[j], s2[r]);
        }
      }
    }
    float s[2 * kRows];   // of g, then of g xh
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      s[r] = s1[r].x + s1[r].y;
      s[kRows + r] = s2[r].x + s2[r].y;
    }
    lanes_sum(s, p.lanes);
    if (p.warps > 1) {
      if (p.lane == 0) {
#pragma unroll
        for (int n = 0; n < 2 * kRows; ++n) red[buf][n][p.warp] = s[n];
      }
      // A warp that writes this half again has passed the barrier of the batch
      // between, as has every reader after reading.
      __syncthreads();
#pragma unroll
      for (int n = 0; n < 2 * kRows; n += 2) {
        const int peer = p.lane & 15;
        const float sum = half_warp_sum(peer < p.warps ? red[buf][n + (p.lane >> 4)][p.first + peer] : 0.f);
        s[n] = __shfl_sync(0xffffffffu, sum, 0);
        s[n + 1] = __shfl_sync(0xffffffffu, sum, 16);
      }
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
        if (!kWhole && at >= p.rows) continue;
        const float2 c1 = both(-s[r] * a.inv_d), c2 = both(-s[kRows + r] * a.inv_d), rs = both(rstd[r]);
        Chunk<VE> dy, xh;
        get(buf, r, row, c2.x, c, dy, xh);
#pragma unroll
        for (int j = 0; j < kSize / 2; ++j) {
          const float2 t = kCodes ? add2(xh.p[j], c1) : fma2(xh.p[j], c2, c1);
          xh.p[j] = mul2(rs, fma2(dy.p[j], w[c].p[j], t));
        }
        put_chunk(static_cast<T*>(a.Y) + row_at(a, row, a.ld_x), p, c, xh);
      }
    }
  };
  for (int buf = 0; row0 < p.rows; row0 += step, buf ^= 1) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      mean[r] = next_mean[r];
      rstd[r] = next_rstd[r];
#pragma unroll
      for (int k = 0; k < kSb; ++k) sb[r][k] = next_sb[r][k];
    }
    if (row0 + step + span <= p.rows) fetch(buf ^ 1, row0 + step, std::true_type());
    else fetch(buf ^ 1, row0 + step, std::false_type());
    async_commit();
    async_wait<1>();
    if (row0 + span <= p.rows) body(buf, row0, std::true_type());
    else body(buf, row0, std::false_type());
  }
  if (!a.partial) return;
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.D;
  float* fold = reinterpret_cast<float*>(ring);
  if (p.groups > 1) {
    async_wait<0>();
    __syncthreads();   // every thread has read its last rows
    out = fold + p.group * 2 * a.D;
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    put_columns(out, p, c, dw[c]);
    put_columns(out + a.D, p, c, db[c]);
  }
  if (p.groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += blockDim.x) {
      float v = 0.f;
      for (int q = 0; q < p.groups; ++q) v += fold[q * 2 * a.D + c];
      a.partial[(int64_t)blockIdx.x * 2 * a.D + c] = v;
    }
  }
}

template <typename T, int VE, int NV, int kRows, int F, bool kCodes>
cudaError_t launch_backward(const NormArgs& a, const Shape& s, int grid, cudaStream_t st) {
  constexpr bool kAsync = VE > 1;
  using U = typename std::conditional<kCodes, uint8_t, T>::type;
  const int sh = Batch<T, VE, NV, kRows, kAsync>::kBytes + Batch<U, VE, NV, kRows, kAsync>::kBytes;
  const int fold = a.partial && s.groups > 1 ? s.groups * 2 * a.D * (int)sizeof(float) : 0;
  return launch(norm_bwd_kernel<T, VE, NV, kRows, kAsync, F, kCodes>, grid, s.threads, sh > fold ? sh : fold, a, st);
}

}  // namespace
}  // namespace vda
