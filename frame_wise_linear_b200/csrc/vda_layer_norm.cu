// Layer norm over the last dimension, forward and backward, optionally with
// the normalised row kept in 8 bits for the backward.
//
//   forward    m = sum x / D, r = 1 / sqrt(sum (x - m)^2 / D + eps),
//              xh = (x - m) r, y = xh w + b
//   backward   g = dy w, dx = r (g - mean(g) - xh mean(g xh)),
//              dw = sum over rows of dy xh, db = sum over rows of dy
//
// Both are bound by HBM: a row is read once, stays on the SM between its sums
// and its outputs, and is written once.  A row belongs to `tpr` threads, each
// with 16 of its elements as 16-byte vectors (single elements where rows are
// not 16-byte aligned).  A CTA walks over batches of rows, with the next batch
// already on its way: every thread copies its own vectors into its own places
// in shared memory (cp.async), so they need no barrier, cost no registers and
// keep HBM busy while a batch is summed and written.  Several rows a batch
// let the chains of their sums overlap, and share the barrier of a row's
// warps.  Next to HBM the instructions count (a row of 4096 has 550 ns on its
// SM in the backward), hence float32 in pairs.
//
// The row's sums: shuffles within a warp, and where a row has several warps
// one exchange through shared memory with one barrier a batch.  In the forward
// each thread takes the mean of its own elements first and the squares of the
// differences from that; lanes and warps join (count, mean, squares):
// sum of squares = sum_i M2_i + n_i (m_i - m)^2, exact algebra without the
// cancellation of sum x^2 - D m^2, and no second pass over the row before m
// is known.
//
// The gradients of w and b are sums over all rows.  A thread holds the same
// columns of every row that its CTA takes, so it keeps their sums in
// registers; each CTA writes one row of partial sums, and a second kernel
// adds those rows in a fixed order (no atomics: the result does not depend on
// the order in which CTAs run).  Everything is float32; an output is rounded
// once.
#include <type_traits>

#include "vda_internal.cuh"
#include "vda_tokops.cuh"

namespace vda {
namespace {

using namespace tokops;
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
  int64_t rows, ld_x, ld_y;   // ld_x: X (and dX); ld_y: Y, dY; from one token to the next
  uint64_t by_heads;   // ceil(2^64 / heads), or 0: every row is a token
  int heads, D, tpr;
  int shift, kinds;    // rows of any width: where row 0 starts in a vector, and after how many rows that repeats
  float eps, inv_d;
  int w_bf16;
};

// Element offset of a row: token row / heads, head row % heads.  The quotient
// by multiplication is exact: row * heads < 2^64.
__device__ __forceinline__ int64_t row_at(const NormArgs& a, int64_t row, int64_t ld) {
  if (a.by_heads == 0) return row * ld;
  const int64_t tok = (int64_t)__umul64hi((uint64_t)row, a.by_heads);
  return tok * ld + (row - tok * a.heads) * a.D;
}

__device__ __forceinline__ float load_w(const void* w, int i, int w_bf16) {
  return w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]) : static_cast<const float*>(w)[i];
}
// Sums over a group of neighbouring lanes (lanes: a power of two).
template <int N>
__device__ __forceinline__ void lanes_sum(float (&v)[N], int lanes) {
  if (lanes == 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  } else {
    for (int o = lanes / 2; o > 0; o >>= 1) {
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    }
  }
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kThreads = 256;   // of a CTA at most, and the ring's stride

// Which of the vectors of VE elements that a row's threads may hold it has.
//   kAll: rows are vectors, and every thread has all of its NV.
//   kSome: rows are vectors, and some threads have fewer.
//   kShift: dense rows of any width.  A row starts `shift` elements into an
//   aligned vector, and the shift repeats every `kinds` rows; a CTA takes rows
//   of one kind, so that its threads keep their columns.  The first and last
//   vector of a row hold elements of its neighbours, too: read and left alone.
enum Fill { kAll, kSome, kShift };

// What a thread is in its CTA, and which columns it holds: vectors t + k tpr,
// k < NV; vector v is columns v VE - shift .. + VE - 1.
template <int VE, int NV, int F>
struct Place {
  int t, group, groups, tpr, nvec, lanes, warps, lane, warp, first, D, shift, kind, kinds;
  int64_t rows, cta, ctas;   // rows of this CTA's kind, its place among the CTAs that share them
  __device__ __forceinline__ explicit Place(const NormArgs& a) {
    tpr = a.tpr;
    t = (int)threadIdx.x % a.tpr;
    group = (int)threadIdx.x / a.tpr;
    groups = (int)blockDim.x / a.tpr;
    D = a.D;
    if constexpr (F == kShift) {
      kinds = a.kinds;
      kind = blockIdx.x % kinds;
      cta = blockIdx.x / kinds;
      ctas = gridDim.x / kinds;
      rows = (a.rows - kind + kinds - 1) / kinds;
      shift = (a.shift + kind * a.D) % VE;
    } else {
      kinds = 1;
      kind = shift = 0;
      cta = blockIdx.x;
      ctas = gridDim.x;
      rows = a.rows;
    }
    nvec = (a.D + shift + VE - 1) / VE;
    lanes = a.tpr < 32 ? a.tpr : 32;
    warps = a.tpr < 32 ? 1 : a.tpr >> 5;
    lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    first = warp / warps * warps;   // the row's first warp
  }
  // Row i of this kind among all rows.
  __device__ __forceinline__ int64_t real(int64_t i) const { return F == kShift ? i * kinds + kind : i; }
  __device__ __forceinline__ int vec(int k) const { return t + k * tpr; }
  __device__ __forceinline__ int col(int k) const { return vec(k) * VE - shift; }
  __device__ __forceinline__ bool has(int k) const { return F == kAll || vec(k) < nvec; }
  // Element i of vector k is one of the row's; all of vector k's are.
  __device__ __forceinline__ bool in(int k, int i) const {
    return F == kShift ? (unsigned)(col(k) + i) < (unsigned)D : has(k);
  }
  __device__ __forceinline__ bool whole(int k) const {
    return F == kShift ? col(k) >= 0 && col(k) + VE <= D : has(k);
  }
  // Columns of the row among n that start at column c.
  __device__ __forceinline__ int columns(int c, int n) const {
    const int lo = c > 0 ? c : 0, hi = c + n < D ? c + n : D;
    return hi > lo ? hi - lo : 0;
  }
  __device__ __forceinline__ int elements() const {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) n += F == kAll ? VE : columns(col(k), VE);
    return n;
  }
  // Elements that warp i of a row holds: vectors 32 i + k tpr .. + 31.
  __device__ __forceinline__ int warp_elements(int i) const {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) n += columns((i * 32 + k * tpr) * VE - shift, 32 * VE);
    return n;
  }
};

// A thread's elements of a row as pairs: element e = k VE + i is half e % 2 of
// pair e / 2.
template <int N>
struct Pairs {
  float2 p[N / 2];
  __device__ __forceinline__ void set(int e, float v) { (e % 2 ? p[e / 2].y : p[e / 2].x) = v; }
  __device__ __forceinline__ float get(int e) const { return e % 2 ? p[e / 2].y : p[e / 2].x; }
};

// The columns of w (or `none`) that a thread holds; 16 bytes at a time where a
// vector's columns start at a multiple of that.
template <int VE, int NV, int F>
__device__ __forceinline__ void load_columns(const void* w, const NormArgs& a, const Place<VE, NV, F>& p,
                                             float none, Pairs<NV * VE>& out) {
  const bool aligned = VE >= 4 && F != kShift && w && ((uintptr_t)w & 15) == 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int i = 0; i < VE; ++i) out.set(k * VE + i, none);
    if (!w || !p.has(k)) continue;
    if constexpr (VE >= 4) {
      if (aligned) {
        if (a.w_bf16) {
          Pack<__nv_bfloat16, VE> q;
          q.load(static_cast<const __nv_bfloat16*>(w) + p.vec(k) * VE);
#pragma unroll
          for (int i = 0; i < VE; ++i) out.set(k * VE + i, q.get(i));
        } else {
#pragma unroll
          for (int j = 0; j < VE; j += 4) {
            Pack<float, 4> q;
            q.load(static_cast<const float*>(w) + p.vec(k) * VE + j);
#pragma unroll
            for (int i = 0; i < 4; ++i) out.set(k * VE + j + i, q.get(i));
          }
        }
        continue;
      }
    }
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (p.in(k, i)) out.set(k * VE + i, load_w(w, p.col(k) + i, a.w_bf16));
  }
}

// The columns of a thread to a row of sums in global or shared memory (16-byte
// aligned where rows are vectors of 4 or 8).
template <int VE, int NV, int F>
__device__ __forceinline__ void store_columns(float* to, const Place<VE, NV, F>& p, const Pairs<NV * VE>& v) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!p.has(k)) continue;
    if constexpr (VE >= 4 && F != kShift) {
#pragma unroll
      for (int j = 0; j < VE; j += 4) {
        const int e = (k * VE + j) / 2;
        *reinterpret_cast<float4*>(to + p.vec(k) * VE + j) =
            make_float4(v.p[e].x, v.p[e].y, v.p[e + 1].x, v.p[e + 1].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (p.in(k, i)) to[p.col(k) + i] = v.get(k * VE + i);
    }
  }
}

// Where the threads of a CTA find the elements of a batch: kRows rows of every
// row group, two batches on the SM, one being worked on and one on its way.
// kAsync: in shared memory, [2][kRows][NV][kThreads] vectors from `base`, each
// thread's own, filled by its own cp.async (so no barrier is needed to read
// them).  Else (single elements) straight from global memory, the second time
// from the caches.  Rows are given by their first element.
template <typename T, int VE, int NV, int kRows, bool kAsync>
struct Batch {
  static constexpr int kBytes = kAsync ? 2 * kRows * NV * VE * (int)sizeof(T) * kThreads : 0;
  T* place;
  const T *begin, *end;   // the tensor, where its rows are dense
  __device__ __forceinline__ Batch(void* base, const T* tensor, const NormArgs& a)
      : place(static_cast<T*>(base) + (int)threadIdx.x * VE), begin(tensor), end(tensor + a.rows * a.D) {}
  __device__ __forceinline__ T* slot(int buf, int r, int k) const {
    return place + buf * (kRows * NV * kThreads * VE) + (r * NV + k) * (kThreads * VE);
  }
  template <int F>
  __device__ __forceinline__ void fetch(int buf, int r, const T* row, const Place<VE, NV, F>& p) const {
    if constexpr (kAsync) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!p.has(k)) continue;
        const T* from = row + p.col(k);
        if (F != kShift || p.whole(k) || (from >= begin && from + VE <= end)) {
          async_copy<VE * (int)sizeof(T)>(slot(buf, r, k), from);
        } else {   // the tensor's first or last vector reaches beyond it
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (p.in(k, i)) slot(buf, r, k)[i] = from[i];
        }
      }
    }
  }
  // The thread's vector k of row r, zeros where it has no element.
  template <int F>
  __device__ __forceinline__ Pack<T, VE> get(int buf, int r, int k, const T* row, const Place<VE, NV, F>& p) const {
    Pack<T, VE> q;
    if constexpr (F != kAll) q.zero();
    if (p.has(k)) q.load(kAsync ? slot(buf, r, k) : row + p.col(k));
    if constexpr (F == kShift) {
      if (!p.whole(k)) {
        Pack<T, VE> none;
        none.zero();
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (!p.in(k, i)) q.e[i] = none.e[i];
      }
    }
    return q;
  }
  // All of the thread's elements of a row.
  template <int F>
  __device__ __forceinline__ void get(int buf, int r, const T* row, const Place<VE, NV, F>& p,
                                      Pairs<NV * VE>& out) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const Pack<T, VE> q = get(buf, r, k, row, p);
#pragma unroll
      for (int i = 0; i < VE; ++i) out.set(k * VE + i, q.get(i));
    }
  }
};

// A thread's elements to a row, rounded to its type.
template <typename T, int VE, int NV, int F>
__device__ __forceinline__ void put(T* row, const Place<VE, NV, F>& p, const Pairs<NV * VE>& v) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    Pack<T, VE> q;
    if constexpr (VE > 1) {
#pragma unroll
      for (int i = 0; i < VE; i += 2) q.set2(i, v.p[(k * VE + i) / 2]);
    } else {
      q.set(0, v.get(k));
    }
    if (p.whole(k)) {
      q.store(row + p.col(k));
    } else if constexpr (F == kShift) {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (p.in(k, i)) row[p.col(k) + i] = q.e[i];
    }
  }
}

// CTAs of an SM that the kernels are compiled for, by the elements a thread
// holds (two: up to 128 registers a thread; with three the rows of a batch
// spill: 45360 x 4096 bf16 forward 190 us against 148, backward 234 against
// 205).
constexpr int ctas_of(int per) { return per == 32 ? 1 : 2; }

template <typename T, int VE, int NV, int kRows, bool kAsync, int F, bool kCodes>
__global__ void __launch_bounds__(kThreads, ctas_of(NV * VE)) norm_fwd_kernel(const NormArgs a) {
  constexpr int N = NV * VE;
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
  Pairs<N> w, b;
  load_columns(a.W, a, p, 1.f, w);
  load_columns(a.bias, a, p, 0.f, b);
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
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      s[r] = m2[r] = own[r] = 0.f;
      if (kWhole || at < p.rows) {
        Pairs<N> x;
        in.get(buf, r, X + row_at(a, row, a.ld_x), p, x);
        float2 sum = x.p[0];
#pragma unroll
        for (int j = 1; j < N / 2; ++j) sum = add2(sum, x.p[j]);
        s[r] = sum.x + sum.y;
        own[r] = s[r] * inv_t;   // the thread's own mean
        float2 sq = both(0.f);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          float2 d = add2(x.p[j], both(-own[r]));
          if constexpr (F != kAll) {
            if (!p.in(2 * j / VE, 2 * j % VE)) d.x = 0.f;
            if (!p.in((2 * j + 1) / VE, (2 * j + 1) % VE)) d.y = 0.f;
          }
          sq = fma2(d, d, sq);
        }
        m2[r] = sq.x + sq.y;
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
        const int at = kRows > 1 ? r + (p.lane >> 4) : 0;
        const float2 e = in_row ? red[buf][at][p.first + peer] : make_float2(0.f, 0.f);
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
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      if (!kWhole && at >= p.rows) break;
      const T* xr = X + row_at(a, row, a.ld_x);
      T* yr = static_cast<T*>(a.Y) + row_at(a, row, a.ld_y);
      Pairs<N> x, y;
      in.get(buf, r, xr, p, x);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        x.p[j] = mul2(add2(x.p[j], both(-mean[r])), both(rstd[r]));
        y.p[j] = fma2(x.p[j], w.p[j], b.p[j]);
      }
      put(yr, p, y);
      if constexpr (kCodes) {
        static_assert(F != kShift, "a block's lanes are those of one vector of four or eight");
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          // A thread without this vector adds nothing to the block's maximum.
          // |xh| is at most sqrt(D) (or NaN).
          float xh[VE];
#pragma unroll
          for (int i = 0; i < VE; ++i) xh[i] = p.has(k) ? x.get(k * VE + i) : 0.f;
          Pack<uint8_t, VE> c;
          const int sb = encode_block<VE, true>(xh, c, kWhole ? 0xffffffffu : lane_group<kBlock / VE>());
          if (p.has(k)) {
            c.store(a.codes + row * a.D + p.vec(k) * VE);
            if (p.vec(k) % (kBlock / VE) == 0) a.scales[row * nblk + p.vec(k) / (kBlock / VE)] = (uint8_t)sb;
          }
        }
      }
      if (p.t == 0) {
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

// The scale bytes of a thread's vectors of a row; a shifted vector may reach
// from one block into the next, whose byte is then the second.
template <int VE, int NV, int F>
__device__ __forceinline__ void load_scales(const NormArgs& a, int64_t row, int nblk, const Place<VE, NV, F>& p,
                                            int (&sb)[NV]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!p.has(k)) continue;
    if constexpr (F == kShift) {
      const int lo = p.col(k) > 0 ? p.col(k) : 0, hi = p.col(k) + VE <= a.D ? p.col(k) + VE - 1 : a.D - 1;
      sb[k] = a.scales[row * nblk + lo / kBlock] | a.scales[row * nblk + hi / kBlock] << 8;
    } else {
      sb[k] = a.scales[row * nblk + p.vec(k) / (kBlock / VE)];
    }
  }
}

// All of a thread's elements of a row of codes, each times its block's scale
// times `by`.
template <int VE, int NV, int kRows, bool kAsync, int F>
__device__ __forceinline__ void get_codes(const Batch<uint8_t, VE, NV, kRows, kAsync>& in, int buf, int r,
                                          const uint8_t* row, const Place<VE, NV, F>& p, const int (&sb)[NV],
                                          float by, Pairs<NV * VE>& out) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const float scale = scale_of(sb[k] & 255) * by;
    float2 x[VE > 1 ? VE / 2 : 1];
    decode_pairs<VE>(in.get(buf, r, k, row, p), x);
    if constexpr (F == kShift) {
      // Elements up to the end of the first one's block.
      const int split = kBlock - (p.col(k) > 0 ? p.col(k) % kBlock : p.col(k));
      const float next = scale_of(sb[k] >> 8) * by;
#pragma unroll
      for (int j = 0; j < VE / 2; ++j)
        out.p[k * VE / 2 + j] =
            mul2(x[j], make_float2(2 * j < split ? scale : next, 2 * j + 1 < split ? scale : next));
    } else if constexpr (VE > 1) {
#pragma unroll
      for (int j = 0; j < VE / 2; ++j) out.p[k * VE / 2 + j] = mul2(x[j], both(scale));
    } else {
      out.set(k, x[0].x * scale);
    }
  }
}

// The backward: X with mean and rstd, or (kCodes) the 8-bit normalised row
// with rstd.  Writes dX, and with a.partial the CTA's sums of dy xh and dy.
// A batch's elements are read twice from shared memory, for the sums and for
// dX: kept in registers they would cost 32 a row, and the occupancy with them.
template <typename T, int VE, int NV, int kRows, bool kAsync, int F, bool kCodes>
__global__ void __launch_bounds__(kThreads, ctas_of(NV * VE)) norm_bwd_kernel(const NormArgs a) {
  constexpr int N = NV * VE, kSb = kCodes ? NV : 1;
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
  float mean[kRows], rstd[kRows], next_mean[kRows], next_rstd[kRows];
  int sb[kRows][kSb], next_sb[kRows][kSb];
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
  // The thread's dy, and xh (of codes: times `by`), of row r.
  auto get = [&](int buf, int r, int64_t row, float by, Pairs<N>& dy, Pairs<N>& xh) {
    iny.get(buf, r, dY + row_at(a, row, a.ld_y), p, dy);
    if constexpr (kCodes) {
      get_codes(inx, buf, r, X + x_at(row), p, sb[r], by, xh);
    } else {
      inx.get(buf, r, X + x_at(row), p, xh);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) xh.p[j] = mul2(add2(xh.p[j], both(-mean[r])), both(rstd[r]));
    }
  };
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    next_mean[r] = next_rstd[r] = 0.f;
#pragma unroll
    for (int k = 0; k < kSb; ++k) next_sb[r][k] = 0;
  }
  int64_t row0 = p.cta * span;
  fetch(0, row0, std::false_type());
  async_commit();
  Pairs<N> w, dw, db;
  load_columns(a.W, a, p, 1.f, w);
#pragma unroll
  for (int j = 0; j < N / 2; ++j) dw.p[j] = db.p[j] = both(0.f);
  auto body = [&](int buf, int64_t row0, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    float s[2 * kRows];   // of g, then of g xh
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      float2 s1 = both(0.f), s2 = both(0.f);
      if (kWhole || at < p.rows) {
        Pairs<N> dy, xh;
        get(buf, r, row, 1.f, dy, xh);
        // Where the thread has no vector dy is 0: nothing is added.
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float2 t = mul2(dy.p[j], xh.p[j]);
          dw.p[j] = add2(dw.p[j], t);
          db.p[j] = add2(db.p[j], dy.p[j]);
          s1 = fma2(dy.p[j], w.p[j], s1);
          s2 = fma2(t, w.p[j], s2);
        }
      }
      s[r] = s1.x + s1.y;
      s[kRows + r] = s2.x + s2.y;
    }
    lanes_sum(s, p.lanes);
    if (p.warps > 1) {
      if (p.lane == 0) {
#pragma unroll
        for (int n = 0; n < 2 * kRows; ++n) red[buf][n][p.warp] = s[n];
      }
      __syncthreads();   // the halves alternate: see the forward
#pragma unroll
      for (int n = 0; n < 2 * kRows; n += 2) {
        const int peer = p.lane & 15;
        const float sum = half_warp_sum(peer < p.warps ? red[buf][n + (p.lane >> 4)][p.first + peer] : 0.f);
        s[n] = __shfl_sync(0xffffffffu, sum, 0);
        s[n + 1] = __shfl_sync(0xffffffffu, sum, 16);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      if (!kWhole && at >= p.rows) break;
      T* dx = static_cast<T*>(a.Y) + row_at(a, row, a.ld_x);
      const float2 c1 = both(-s[r] * a.inv_d), c2 = both(-s[kRows + r] * a.inv_d), rs = both(rstd[r]);
      Pairs<N> dy, xh;
      get(buf, r, row, c2.x, dy, xh);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const float2 t = kCodes ? add2(xh.p[j], c1) : fma2(xh.p[j], c2, c1);
        xh.p[j] = mul2(rs, fma2(dy.p[j], w.p[j], t));
      }
      put(dx, p, xh);
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
  store_columns(out, p, dw);
  store_columns(out + a.D, p, db);
  if (p.groups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += blockDim.x) {
      float v = 0.f;
      for (int q = 0; q < p.groups; ++q) v += fold[q * 2 * a.D + c];
      a.partial[(int64_t)blockIdx.x * 2 * a.D + c] = v;
    }
  }
}

// dW and db from the CTAs' partial sums [parts][2 D]: 32 columns a block,
// thread (x, y) adds rows y, y + 32, ...; then a warp the 32 sums of a column.
// The rows come from L2; there are at most 296 of them, so a thread has ten
// loads, all on their way at once.
__global__ void __launch_bounds__(1024) norm_fold_kernel(const float* partial, int parts, int D, float* dW, float* db) {
  __shared__ float sh[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float v = 0.f;
  if (c < 2 * D) {
#pragma unroll 10
    for (int i = y; i < parts; i += 32) v += partial[(int64_t)i * 2 * D + c];
  }
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

// y = xh w + b from the 8-bit normalised rows.
template <typename T, int VE, int NV, int kRows, bool kAsync, int F>
__global__ void __launch_bounds__(kThreads, ctas_of(NV * VE)) norm_apply_kernel(const NormArgs a) {
  constexpr int N = NV * VE;
  extern __shared__ __align__(16) uint8_t ring[];
  const Place<VE, NV, F> p(a);
  const int nblk = (a.D + kBlock - 1) / kBlock;
  const Batch<uint8_t, VE, NV, kRows, kAsync> in(ring, a.codes, a);
  int sb[kRows][NV], next_sb[kRows][NV] = {};
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
  Pairs<N> w, b;
  load_columns(a.W, a, p, 1.f, w);
  load_columns(a.bias, a, p, 0.f, b);
  for (int buf = 0; row0 < p.rows; row0 += step, buf ^= 1) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int k = 0; k < NV; ++k) sb[r][k] = next_sb[r][k];
    fetch(buf ^ 1, row0 + step);
    async_commit();
    async_wait<1>();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = row0 + r * p.groups + p.group, row = p.real(at);
      if (at >= p.rows) break;
      T* yr = static_cast<T*>(a.Y) + row_at(a, row, a.ld_y);
      Pairs<N> x;
      get_codes(in, buf, r, a.codes + row * a.D, p, sb[r], 1.f, x);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) x.p[j] = fma2(x.p[j], w.p[j], b.p[j]);
      put(yr, p, x);
    }
  }
}

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Threads of a row and of a CTA, and rows of a CTA.  A thread holds 16
// elements of a row (8 where a row would not fill the lanes of a block of
// codes with 16, 32 where a row would need more than 256 threads); a row
// takes a power of two up to 32 threads, at least the lanes of one block, or
// whole warps.
struct Shape {
  int per, tpr, threads, groups, kinds;
  Fill fill;
};
Shape shape_for(int D, int ve, int kinds = 0) {
  const int least = kBlock / ve, nvec = kinds ? (D + 2 * ve - 2) / ve : D / ve;   // kinds: at any shift
  const int per = nvec * ve <= 8 * least ? 8 : (nvec * ve <= 16 * kThreads ? 16 : 32);
  const int need = (nvec + per / ve - 1) / (per / ve);
  int tpr = least;
  while (tpr < 32 && tpr < need) tpr *= 2;
  if (need > 32) tpr = (need + 31) / 32 * 32;
  const int groups = tpr > kThreads ? 0 : kThreads / tpr;   // 0: more than the CTA's threads
  return Shape{per,    tpr, tpr * groups, groups, kinds ? kinds : 1, kinds ? kShift
                                                                     : nvec == tpr * (per / ve) ? kAll : kSome};
}

// CTAs for `rows` rows in batches of `n` rows a group: as many as are resident
// at once, or as there are batches; as many for each kind.
int grid_for(int64_t rows, const Shape& s, int n) {
  const int64_t each = (rows + s.kinds - 1) / s.kinds, batches = (each + (int64_t)s.groups * n - 1) / ((int64_t)s.groups * n);
  const int64_t most = 148 * ctas_of(s.per) / s.kinds;
  return (int)(batches < most ? batches : most) * s.kinds;
}
// Batches of several rows where every CTA gets one all the same.
bool batched(int64_t rows, const Shape& s, int n) { return rows >= (int64_t)grid_for(rows, s, 1) * s.groups * n; }

// 16-byte vectors where the width, the strides and the pointers allow them.
template <typename T>
bool wide(const NormArgs& a) {
  const int ve = 16 / (int)sizeof(T);
  return a.D % ve == 0 && a.ld_x % ve == 0 && a.ld_y % ve == 0 && aligned_to(a.X, 16) && aligned_to(a.dY, 16) &&
         aligned_to(a.Y, 16) && aligned_to(a.codes, ve);
}

// Rows of any width by vectors: dense tensors that start at the same place of a
// vector.  Rows narrower than four vectors would leave most of a vector unused.
template <typename T>
bool shifted(const NormArgs& a) {
  const int ve = 16 / (int)sizeof(T);
  if (a.D < 4 * ve || a.ld_x != a.D || a.ld_y != a.D || a.heads != 1) return false;
  const int place = (int)((uintptr_t)a.Y / sizeof(T) % ve);
  auto same = [&](const void* x) { return !x || (int)((uintptr_t)x / sizeof(T) % ve) == place; };
  return same(a.X) && same(a.dY) && (!a.codes || (int)((uintptr_t)a.codes % ve) == place) &&
         shape_for(a.D, ve, 1).groups > 0;
}
// After how many rows of D elements the place in a vector repeats, or the rows
// there are.
int kinds_for(int D, int ve, int64_t rows) {
  int n = 1;
  while (n * D % ve) n *= 2;
  return rows < n ? (int)rows : n;
}

template <typename Kernel>
cudaError_t launch(Kernel k, int grid, int threads, int sh, const NormArgs& a, cudaStream_t st) {
  if (sh > 46 * 1024) {   // with the static part, what a launch may have without asking is 48 KB
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sh);
    if (e != cudaSuccess) return e;
  }
  k<<<grid, threads, sh, st>>>(a);
  return cudaGetLastError();
}

enum Pass { kForward, kBackward, kApply };

template <typename T, int VE, int NV, int kRows, int F>
cudaError_t run_rows(Pass pass, const NormArgs& a, const Shape& s, cudaStream_t st) {
  constexpr bool kX = VE > 1, kC = VE > 1, kBoth = kX && kC;
  const int grid = grid_for(a.rows, s, kRows);
  if (pass == kForward) {
    auto k = norm_fwd_kernel<T, VE, NV, kRows, kX, F, false>;
    if constexpr (F != kShift) {
      if (a.codes) k = norm_fwd_kernel<T, VE, NV, kRows, kX, F, true>;
    }
    return launch(k, grid, s.threads, Batch<T, VE, NV, kRows, kX>::kBytes, a, st);
  }
  if (pass == kApply)
    return launch(norm_apply_kernel<T, VE, NV, kRows, kC, F>, grid, s.threads,
                  Batch<uint8_t, VE, NV, kRows, kC>::kBytes, a, st);
  const int fold = a.partial && s.groups > 1 ? s.groups * 2 * a.D * (int)sizeof(float) : 0;
  if (a.codes) {
    const int sh = Batch<T, VE, NV, kRows, kBoth>::kBytes + Batch<uint8_t, VE, NV, kRows, kBoth>::kBytes;
    return launch(norm_bwd_kernel<T, VE, NV, kRows, kBoth, F, true>, grid, s.threads, sh > fold ? sh : fold, a, st);
  }
  const int sh = 2 * Batch<T, VE, NV, kRows, kX>::kBytes;
  return launch(norm_bwd_kernel<T, VE, NV, kRows, kX, F, false>, grid, s.threads, sh > fold ? sh : fold, a, st);
}

// Rows of a batch: 128 bytes of a thread's loads on their way, where there are
// rows enough.
constexpr int batch_rows(int element, int per, bool backward) {
  const int n = 128 / (per * element) / (backward ? 2 : 1);
  return n < 1 ? 1 : n > 4 ? 4 : n;
}

template <typename T, int VE, int NV, int F>
cudaError_t run_shape(Pass pass, const NormArgs& a, const Shape& s, float* dW, float* db, cudaStream_t st) {
  // Single elements: one row a batch (their loads are not ahead of their use).
  constexpr int most = VE == 1 ? 1 : batch_rows(sizeof(T), VE * NV, false);
  constexpr int most_backward = VE == 1 ? 1 : batch_rows(sizeof(T), VE * NV, true);
  if (pass != kBackward)
    return batched(a.rows, s, most) ? run_rows<T, VE, NV, most, F>(pass, a, s, st)
                                    : run_rows<T, VE, NV, 1, F>(pass, a, s, st);
  const bool many = batched(a.rows, s, most_backward);
  cudaError_t e =
      many ? run_rows<T, VE, NV, most_backward, F>(pass, a, s, st) : run_rows<T, VE, NV, 1, F>(pass, a, s, st);
  if (e != cudaSuccess || !a.partial) return e;
  const int parts = grid_for(a.rows, s, many ? most_backward : 1);
  norm_fold_kernel<<<(2 * a.D + 31) / 32, 1024, 0, st>>>(a.partial, parts, a.D, dW, db);
  return cudaGetLastError();
}

template <typename T, int VE, int NV>
cudaError_t run_fill(Pass pass, const NormArgs& a, const Shape& s, float* dW, float* db, cudaStream_t st) {
  if constexpr (VE > 1) {
    if (s.fill == kAll) return run_shape<T, VE, NV, kAll>(pass, a, s, dW, db, st);
    if (s.fill == kShift) return run_shape<T, VE, NV, kShift>(pass, a, s, dW, db, st);
  }
  return run_shape<T, VE, NV, kSome>(pass, a, s, dW, db, st);   // single elements too
}

template <typename T, int VE>
cudaError_t run_per(Pass pass, NormArgs& a, const Shape& s, float* dW, float* db, cudaStream_t st) {
  a.tpr = s.tpr;
  a.kinds = s.kinds;
  if (s.per == 8) return run_fill<T, VE, 8 / VE>(pass, a, s, dW, db, st);
  if (s.per == 16) return run_fill<T, VE, 16 / VE>(pass, a, s, dW, db, st);
  return run_fill<T, VE, 32 / VE>(pass, a, s, dW, db, st);
}

template <typename T>
cudaError_t run_type(Pass pass, NormArgs& a, float* dW, float* db, cudaStream_t st) {
  constexpr int VE = 16 / (int)sizeof(T);
  if (wide<T>(a)) return run_per<T, VE>(pass, a, shape_for(a.D, VE), dW, db, st);
  // (A block of codes that is being made needs its elements in neighbouring
  // lanes, which shifted vectors do not give.)
  if (shifted<T>(a) && !(pass == kForward && a.codes)) {
    a.shift = (int)((uintptr_t)a.Y / sizeof(T) % VE);
    return run_per<T, VE>(pass, a, shape_for(a.D, VE, kinds_for(a.D, VE, a.rows)), dW, db, st);
  }
  return run_per<T, 1>(pass, a, shape_for(a.D, 1), dW, db, st);
}

cudaError_t run(Pass pass, int dtype, NormArgs& a, float* dW, float* db, cudaStream_t st) {
  return dtype == VDA_DTYPE_BF16 ? run_type<__nv_bfloat16>(pass, a, dW, db, st)
                                 : run_type<float>(pass, a, dW, db, st);
}

NormArgs args_for(const vda_norm_problem& p) {
  NormArgs a{};
  a.rows = p.tokens * p.heads;
  a.heads = p.heads;
  a.D = p.D;
  const int64_t dense = (int64_t)p.heads * p.D;
  a.ld_x = p.ld_x ? p.ld_x : dense;
  a.ld_y = p.ld_y ? p.ld_y : dense;
  // Tokens without gaps are rows like any others.
  if (a.ld_x == dense && a.ld_y == dense) {
    a.heads = 1;
    a.ld_x = a.ld_y = p.D;
  }
  a.by_heads = a.heads > 1 ? ~0ull / (uint64_t)a.heads + 1 : 0;
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
  for (int ve : {1, 4, 8})
    for (int kinds : {0, ve > 1 ? kinds_for(p.D, ve, rows) : 0}) {
      const Shape s = shape_for(p.D, ve, kinds);
      const int g = s.groups ? grid_for(rows, s, 1) : 0;
      parts = g > parts ? g : parts;
    }
  return align_up((size_t)parts * 2 * p.D * sizeof(float), 256);
}

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
  a.codes = codes;
  a.scales = scales;
  return run(kForward, p.dtype, a, nullptr, nullptr, st);
}

cudaError_t launch_layer_norm_backward(const vda_norm_problem& p, const void* dY, const void* X, const float* mean,
                                       const float* rstd, const uint8_t* codes, const uint8_t* scales, const void* W,
                                       void* dX, float* dW, float* db, float* partial, cudaStream_t st) {
  NormArgs a = args_for(p);
  if (a.rows == 0) {
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
  return run(kBackward, p.dtype, a, dW, db, st);
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
  return run(kApply, p.dtype, a, nullptr, nullptr, st);
}

}  // namespace vda
