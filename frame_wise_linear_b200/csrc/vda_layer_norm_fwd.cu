// Layer norm's forward (vda_layer_norm.cuh has the plan).
#include "vda_layer_norm.cuh"

namespace vda {
namespace {

template <typename T, int VE, int NV, int kRows, bool kAsync, int F, bool kCodes>
__global__ void __launch_bounds__(kThreads, ctas_of(NV * VE)) norm_fwd_kernel(const NormArgs a) {
  constexpr int kChunks = NV / kOf<VE>, kSize = Chunk<VE>::kSize;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][kRows][kThreads / 32];   // (mean, squares) of each warp's part of a row
  const Place<VE, NV, F> p(a);
  const int nblk = (a.D + kBlock - 1) / kBlock;
  const T* X = static_cast<const T*>(a.X);
  const Batch<T, VE, NV, kRows, kAsync> in(ring, X, a);
  // Row r of a batch that starts at row0: row0 + r groups + group.
  const int64_t span = (int64_t)p.groups * kRows, step = p.ctas * span;
  auto fetch = [&](int buf, int64_t row0, auto whole) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      if (decltype(whole)::value || at < p.rows) in.fetch(buf, r, X + row_at(a, row, a.ld_x), p);
    }
  };
  int64_t row0 = p.cta * span;
  fetch(0, row0, std::false_type());
  async_commit();
  Chunk<VE> w[kChunks], b[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    get_columns(a.W, a, p, c, 1.f, w[c]);
    get_columns(a.bias, a, p, c, 0.f, b[c]);
  }
  const int n_t = p.elements();
  const float count_t = (float)n_t, inv_t = 1.f / (float)(n_t > 1 ? n_t : 1);
  const int n_w = p.warps > 1 ? p.warp_elements(p.warp - p.first) : a.D;
  const float inv_w = n_w > 0 ? 1.f / (float)n_w : 0.f;
  // In the exchange lanes 0 - 15 and 16 - 31 look at one warp each of two rows.
  const int peer = p.lane & 15;
  const bool in_row = peer < p.warps;
  const float weight = in_row ? (float)p.warp_elements(peer) * a.inv_d : 0.f;
  auto body = [&](int buf, int64_t row0, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    float mean[kRows], rstd[kRows], s[kRows], m2[kRows], own[kRows];
    // One float32 row stays in registers until it is written; of several each is
    // read again from shared memory (kept, they spill: 144 us against 133 for
    // 45360 x 4096 bf16).
    constexpr bool kKeep = kRows == 1 && sizeof(T) == 4;
    [[maybe_unused]] Chunk<VE> kept[kChunks];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      s[r] = m2[r] = own[r] = 0.f;
      if (kWhole || at < p.rows) {
        const T* xr = X + row_at(a, row, a.ld_x);
        Pack<T, VE> q[NV];
        float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          q[k] = in.get(buf, r, k, xr, p);
          if constexpr (VE > 1) {
#pragma unroll
            for (int i = 0; i < VE; i += 2) sum[i / 2 % 2] = plus2(q[k], i, sum[i / 2 % 2]);
          } else {
            sum[k / 2 % 2].x += q[k].get(0);
          }
        }
        sum[0] = add2(sum[0], sum[1]);
        s[r] = sum[0].x + sum[0].y;
        own[r] = s[r] * inv_t;   // the thread's own mean
        float2 sq[2] = {both(0.f), both(0.f)};
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int j = 0; j < kSize / 2; ++j) {
            [[maybe_unused]] const int e = c * kSize + 2 * j;   // of the thread's NV VE
            float2 d;
            if constexpr (VE > 1) d = plus2(q[c], 2 * j, both(-own[r]));
            else d = make_float2(q[e].get(0) - own[r], q[e + 1].get(0) - own[r]);
            if constexpr (kKeep) {
              if constexpr (VE > 1) kept[c].p[j] = q[c].get2(2 * j);
              else kept[c].p[j] = make_float2(q[e].get(0), q[e + 1].get(0));
            }
            if constexpr (F != kAll) {
              if (!p.in(e / VE, e % VE)) d.x = 0.f;
              if (!p.in((e + 1) / VE, (e + 1) % VE)) d.y = 0.f;
            }
            sq[j % 2] = fma2(d, d, sq[j % 2]);
          }
        sq[0] = add2(sq[0], sq[1]);
        m2[r] = sq[0].x + sq[0].y;
      }
    }
    lanes_sum(s, p.lanes);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      mean[r] = s[r] * inv_w;
      const float d = own[r] - mean[r];
      m2[r] += F == kAll || n_t > 0 ? count_t * d * d : 0.f;
    }
    lanes_sum(m2, p.lanes);
    if (p.warps > 1) {
      if (p.lane == 0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) red[buf][r][p.warp] = make_float2(mean[r], m2[r]);
      }
      // A warp that writes this half again has passed the barrier of the batch
      // between, as has every reader after reading.
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRows; r += 2) {
        const int of = kRows > 1 ? r + (p.lane >> 4) : 0;
        const float2 e = in_row ? red[buf][of][p.first + peer] : make_float2(0.f, 0.f);
        const float m = half_warp_sum(e.x * weight);
        const float d = e.x - m;
        const float var = half_warp_sum(in_row ? e.y * a.inv_d + weight * d * d : 0.f);
        const float rs = 1.f / sqrtf(var + a.eps);
        mean[r] = __shfl_sync(0xffffffffu, m, 0);
        rstd[r] = __shfl_sync(0xffffffffu, rs, 0);
        if (kRows > 1) {
          mean[r + 1 < kRows ? r + 1 : r] = __shfl_sync(0xffffffffu, m, 16);
          rstd[r + 1 < kRows ? r + 1 : r] = __shfl_sync(0xffffffffu, rs, 16);
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < kRows; ++r) rstd[r] = 1.f / sqrtf(m2[r] * a.inv_d + a.eps);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
        if (!kWhole && at >= p.rows) continue;
        Chunk<VE> x, y;
        if constexpr (kKeep) {
#pragma unroll
          for (int j = 0; j < kSize / 2; ++j) x.p[j] = add2(kept[c].p[j], both(-mean[r]));
        } else {
          get_plus(in, buf, r, X + row_at(a, row, a.ld_x), p, c, -mean[r], x);
        }
#pragma unroll
        for (int j = 0; j < kSize / 2; ++j) {
          x.p[j] = mul2(x.p[j], both(rstd[r]));
          y.p[j] = fma2(x.p[j], w[c].p[j], b[c].p[j]);
        }
        put_chunk(static_cast<T*>(a.Y) + row_at(a, row, a.ld_y), p, c, y);
        if constexpr (kCodes) {
          static_assert(F != kShift, "a block's lanes are those of one vector of four or eight");
#pragma unroll
          for (int k = 0; k < kOf<VE>; ++k) {
            // A thread without this vector adds nothing to the block's maximum.
            // |xh| is at most sqrt(D) (or NaN).
            const int n = c * kOf<VE> + k;
            float xh[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) xh[i] = p.has(n) ? x.get(k * VE + i) : 0.f;
            Pack<uint8_t, VE> q;
            const int sb = encode_block<VE, true>(xh, q, kWhole ? 0xffffffffu : lane_group<kBlock / VE>());
            if (p.has(n)) {
              q.store(a.codes + row * a.D + p.vec(n) * VE);
              if (p.vec(n) % (kBlock / VE) == 0) a.scales[row * nblk + p.vec(n) / (kBlock / VE)] = (uint8_t)sb;
            }
          }
        }
      }
    }
    if (p.t == 0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
        if (!kWhole && at >= p.rows) continue;
        if (a.mean) a.mean[row] = mean[r];
        if (a.rstd) a.rstd[row] = rstd[r];
      }
    }
  };
  for (int buf = 0; row0 < p.rows; row0 += step, buf ^= 1) {
    if (row0 + step + span <= p.rows) fetch(buf ^ 1, row0 + step, std::true_type());
    else fetch(buf ^ 1, row0 + step, std::false_type());
    async_commit();
    async_wait<1>();
    // All but a batch that the rows' end cuts off need no test of each row.
    if (row0 + span <= p.rows) body(buf, row0, std::true_type());
    else body(buf, row0, std::false_type());
  }
}

template <int kPass, typename T, int VE, int NV, int kRows, int F>
cudaError_t launch_pass(const NormArgs& a, const Shape& s, int grid, cudaStream_t st) {
  constexpr bool kAsync = VE > 1;
  return launch(norm_fwd_kernel<T, VE, NV, kRows, kAsync, F, kPass == kForwardCodes>, grid, s.threads,
                Batch<T, VE, NV, kRows, kAsync>::kBytes, a, st);
}

}  // namespace

cudaError_t launch_layer_norm(const vda_norm_problem& p, const void* X, const void* W, const void* bias, void* Y,
                              float* mean, float* rstd, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  NormArgs a = args_for(p);
  if (a.rows == 0) return cudaSuccess;
  a.X = X;
  a.W = W;
  a.bias = bias;
  a.Y = Y;
  a.mean = mean;
  a.rstd = rstd;
  int ctas = 0;
  if (!codes) return run_pass<kForward>(p.dtype, a, &ctas, st);
  // Odd widths: shifted vectors do not give a block of codes its elements in
  // neighbouring lanes.  Y and the statistics first, then the codes from X and
  // those, one more pass over X (45360 x 1001 bf16, with the codes unpacked: 190
  // us, against 372 in one pass by single elements).  That pass is left where X
  // is written over or the statistics are not wanted.
  const bool again = X != Y && mean && rstd &&
                     (p.dtype == VDA_DTYPE_BF16 ? !wide<__nv_bfloat16>(a) && shifted<__nv_bfloat16>(a)
                                                : !wide<float>(a) && shifted<float>(a));
  if (again) {
    cudaError_t e = run_pass<kForward>(p.dtype, a, &ctas, st);
    if (e != cudaSuccess) return e;
    const vda_checkpoint_problem q = {a.rows, 0, p.D, p.dtype};
    return launch_checkpoint_pack_normalised(q, X, mean, rstd, codes, scales, st);
  }
  a.codes = codes;
  a.scales = scales;
  return run_pass<kForwardCodes>(p.dtype, a, &ctas, st);
}

}  // namespace vda
