// Layer norm over the last dimension, forward and backward, optionally with
// the normalised row kept in 8 bits for the backward: what the passes share
// (vda_layer_norm_fwd.cu, vda_layer_norm_bwd.cu, vda_layer_norm_ckpt.cu).
//
//   forward    m = sum x / D, r = 1 / sqrt(sum (x - m)^2 / D + eps),
//              xh = (x - m) r, y = xh w + b
//   backward   g = dy w, dx = r (g - mean(g) - xh mean(g xh)),
//              dw = sum over rows of dy xh, db = sum over rows of dy
//
// Both are bound by HBM: a row is read once, stays on the SM between its sums
// and its outputs, and is written once.  A row belongs to `tpr` threads, each
// with 16 of its elements as 16-byte vectors (Fill, below, has what is done
// where rows are not 16-byte aligned).  A CTA walks over batches of rows, with the next batch
// already on its way: every thread copies its own vectors into its own places
// in shared memory (cp.async), so they need no barrier, cost no registers and
// keep HBM busy while a batch is summed and written.  Several rows a batch
// let the chains of their sums overlap, and share the barrier of a row's
// warps.  Next to HBM the instructions count (a row of 4096 bf16 has 550 ns on
// its SM in the backward, and the clock falls under the power cap), hence
// float32 in pairs and bf16 added to float32 as it is.  45360 x 4096 bf16, in a
// run of calls: forward 123 to 128 us by the box (0.92 to 0.89 of the copy rate),
// backward 190 to 201 us (0.90 to 0.85).
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
#pragma once

#include <type_traits>

#include "vda_internal.cuh"
#include "vda_tokops.cuh"

namespace vda {
namespace {   // each source file that includes this compiles its own kernels

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
  int w_aligned;       // W and bias start at multiples of 16 bytes
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
//   kSome: rows are vectors, and some threads have fewer.  (Vectors of one
//   element: rows with gaps at odd places, and narrow odd rows.)
//   kShift: dense rows of any width.  A row starts `shift` elements into an
//   aligned vector, and the shift repeats every `kinds` rows; a CTA takes rows
//   of one kind, so that its threads keep their columns.  The first and last
//   vector of a row hold elements of its neighbours, too: read and left alone.
//   Every vector is tested for that, and the forward's squares element by
//   element: 27 and 37 instructions of a warp for 32 elements, where whole
//   vectors take 13 and 19, and they are what bounds it.  45360 x 1001 bf16:
//   forward 67 us, backward 84 us; by single elements 126 and 190 us.
enum Fill { kAll, kSome, kShift };

// What a thread is in its CTA, and which columns it holds: vectors t + k tpr,
// k < NV; vector v is columns v VE - shift .. + VE - 1.
template <int VE, int NV, int F>
struct Place {
  int t, group, groups, tpr, nvec, lanes, warps, lane, warp, first, D, shift, kind, kinds;
  uint32_t has_bits, whole_bits;   // by vector
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
    has_bits = whole_bits = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      has_bits |= (vec(k) < nvec ? 1u : 0u) << k;
      whole_bits |= (F == kShift ? col(k) >= 0 && col(k) + VE <= D : vec(k) < nvec) ? 1u << k : 0u;
    }
  }
  // Row i of this kind among all rows.
  __device__ __forceinline__ int64_t real(int64_t i) const { return F == kShift ? i * kinds + kind : i; }
  __device__ __forceinline__ int vec(int k) const { return t + k * tpr; }
  __device__ __forceinline__ int col(int k) const { return vec(k) * VE - shift; }
  __device__ __forceinline__ bool has(int k) const { return F == kAll || (has_bits >> k & 1); }
  // Element i of vector k is one of the row's; all of vector k's are.
  __device__ __forceinline__ bool in(int k, int i) const {
    return F == kShift ? (unsigned)(col(k) + i) < (unsigned)D : has(k);
  }
  __device__ __forceinline__ bool whole(int k) const {
    return F == kAll || (whole_bits >> k & 1);
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

// A thread's elements go in chunks, pairs of them in registers: chunk c is
// vector c, or two single elements.
template <int VE>
struct Chunk {
  static constexpr int kSize = VE > 1 ? VE : 2;
  float2 p[kSize / 2];
  __device__ __forceinline__ void set(int e, float v) { (e % 2 ? p[e / 2].y : p[e / 2].x) = v; }
  __device__ __forceinline__ float get(int e) const { return e % 2 ? p[e / 2].y : p[e / 2].x; }
};
// Vectors of a chunk: chunk c is vectors c kOf .. c kOf + kOf - 1.
template <int VE>
constexpr int kOf = VE > 1 ? 1 : 2;

// The columns of w (or `none`) of chunk c, 16 bytes at a time where they are
// aligned.  A thread loads them once (from L1 for every batch: three CTAs of
// an SM instead of two, but 148 us against 133 for the forward of 45360 x 4096
// bf16, 237 against 214 for the backward).
template <int VE, int NV, int F>
__device__ __forceinline__ void get_columns(const void* w, const NormArgs& a, const Place<VE, NV, F>& p, int c,
                                            float none, Chunk<VE>& out) {
#pragma unroll
  for (int e = 0; e < Chunk<VE>::kSize; ++e) out.set(e, none);
  if (!w) return;
  if constexpr (VE > 1 && F != kShift) {
    if (!p.has(c)) return;
    if (a.w_aligned) {
      if (a.w_bf16) {
        Pack<__nv_bfloat16, VE> q;
        q.load(static_cast<const __nv_bfloat16*>(w) + p.col(c));
#pragma unroll
        for (int i = 0; i < VE; ++i) out.set(i, q.get(i));
      } else {
#pragma unroll
        for (int j = 0; j < VE; j += 4) {
          Pack<float, 4> q;
          q.load(static_cast<const float*>(w) + p.col(c) + j);
#pragma unroll
          for (int i = 0; i < 4; ++i) out.set(j + i, q.get(i));
        }
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < kOf<VE>; ++k)
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (p.in(c * kOf<VE> + k, i)) out.set(k * VE + i, load_w(w, p.col(c * kOf<VE> + k) + i, a.w_bf16));
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
  // The thread's vector k of row r.  Where it has no element: zeros, or `none`
  // in a shifted row's vector.
  template <int F>
  __device__ __forceinline__ Pack<T, VE> get(int buf, int r, int k, const T* row, const Place<VE, NV, F>& p,
                                             T none = T(0.f)) const {
    Pack<T, VE> q;
    if constexpr (F != kAll) q.zero();
    if (p.has(k)) q.load(kAsync ? slot(buf, r, k) : row + p.col(k));
    if constexpr (F == kShift) {
      if (!p.whole(k)) {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (!p.in(k, i)) q.e[i] = none;
      }
    }
    return q;
  }
};

// Chunk c of row r of a batch, zeros where the thread has no element.
template <typename T, int VE, int NV, int kRows, bool kAsync, int F>
__device__ __forceinline__ void get_chunk(const Batch<T, VE, NV, kRows, kAsync>& in, int buf, int r, const T* row,
                                          const Place<VE, NV, F>& p, int c, Chunk<VE>& out) {
#pragma unroll
  for (int k = 0; k < kOf<VE>; ++k) {
    const Pack<T, VE> q = in.get(buf, r, c * kOf<VE> + k, row, p);
    if constexpr (VE > 1) {
#pragma unroll
      for (int i = 0; i < VE; i += 2) out.p[i / 2] = q.get2(i);
    } else {
      out.set(k, q.get(0));
    }
  }
}

// The same plus `by`.  A shifted row's vector has -by in the type where it has
// no element, for a difference next to 0: 0 + by, times rstd, overflows for
// constant rows from 3.4e38 sqrt(eps) up.
template <typename T, int VE, int NV, int kRows, bool kAsync, int F>
__device__ __forceinline__ void get_plus(const Batch<T, VE, NV, kRows, kAsync>& in, int buf, int r, const T* row,
                                         const Place<VE, NV, F>& p, int c, float by, Chunk<VE>& out) {
#pragma unroll
  for (int k = 0; k < kOf<VE>; ++k) {
    const Pack<T, VE> q = in.get(buf, r, c * kOf<VE> + k, row, p, from_f32<T>(F == kShift ? -by : 0.f));
    if constexpr (VE > 1) {
#pragma unroll
      for (int i = 0; i < VE; i += 2) out.p[i / 2] = plus2(q, i, both(by));
    } else {
      out.set(k, q.get(0) + by);
    }
  }
}

// Chunk c of a row, rounded to its type.
template <typename T, int VE, int NV, int F>
__device__ __forceinline__ void put_chunk(T* row, const Place<VE, NV, F>& p, int c, const Chunk<VE>& v) {
#pragma unroll
  for (int k = 0; k < kOf<VE>; ++k) {
    const int n = c * kOf<VE> + k;
    Pack<T, VE> q;
    if constexpr (VE > 1) {
#pragma unroll
      for (int i = 0; i < VE; i += 2) q.set2(i, v.p[i / 2]);
    } else {
      q.set(0, v.get(k));
    }
    if (p.whole(n)) {
      q.store(row + p.col(n));
    } else if constexpr (F == kShift) {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (p.in(n, i)) row[p.col(n) + i] = q.e[i];
    }
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

// Chunk c of a row of codes, each element times its block's scale times `by`.
template <int VE, int NV, int kRows, bool kAsync, int F>
__device__ __forceinline__ void get_codes(const Batch<uint8_t, VE, NV, kRows, kAsync>& in, int buf, int r,
                                          const uint8_t* row, const Place<VE, NV, F>& p, const int (&sb)[NV], float by,
                                          int c, Chunk<VE>& out) {
  if constexpr (VE == 1) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float2 x[1];
      decode_pairs<1>(in.get(buf, r, 2 * c + k, row, p), x);
      out.set(k, x[0].x * (scale_of(sb[2 * c + k]) * by));
    }
  } else {
    const float scale = scale_of(sb[c] & 255) * by;
    float2 x[VE > 1 ? VE / 2 : 1];
    decode_pairs<VE>(in.get(buf, r, c, row, p), x);
    // Elements up to the end of the first one's block; the others are the next one's.
    const int split = F != kShift ? VE : kBlock - (p.col(c) > 0 ? p.col(c) % kBlock : p.col(c));
    const float next = F != kShift ? scale : scale_of(sb[c] >> 8) * by;
#pragma unroll
    for (int j = 0; j < VE / 2; ++j)
      out.p[j] = mul2(x[j], make_float2(2 * j < split ? scale : next, 2 * j + 1 < split ? scale : next));
  }
}

// CTAs of an SM that the kernels are compiled for, by the elements a thread
// holds: two, with up to 128 registers a thread (with three the sums of a batch
// spill: 45360 x 4096 bf16 forward 190 us against 148 at the time, backward 234
// against 205), or one with twice the elements.  These spill all the same: the
// forward of four shifted bf16 rows (12 bytes a thread), and of the single
// elements the float32 forward with 32 of them (16 bytes), the backward from
// codes with 16 or 32 (300 and 560) and y again with 32 (88).
constexpr int ctas_of(int per) { return per == 32 ? 1 : 2; }

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
  const Fill fill = kinds ? kShift : nvec == tpr * (per / ve) ? kAll : kSome;
  return Shape{per, tpr, tpr * groups, groups, kinds ? kinds : 1, fill};
}

// CTAs for `rows` rows in batches of `n` rows a group: as many as are resident
// at once, or as there are batches; as many for each kind.
int grid_for(int64_t rows, const Shape& s, int n) {
  const int64_t each = (rows + s.kinds - 1) / s.kinds, batch = (int64_t)s.groups * n;
  const int64_t batches = (each + batch - 1) / batch;
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

// What a pass over the rows does, and which of the library's source files holds it.
enum Pass { kForward, kForwardCodes, kBackward, kBackwardCodes, kApply };

// The pass's kernel for one shape (defined in the file that holds the pass).
template <int kPass, typename T, int VE, int NV, int kRows, int F>
cudaError_t launch_pass(const NormArgs& a, const Shape& s, int grid, cudaStream_t st);

// Rows of a batch, where there are rows enough: 128 bytes of a thread's loads
// (bf16 forward with 64: 144 us against 129 for 45360 x 4096; backward 220
// against 196, with 256 spilling 214).  The float32 forward takes one row, 64
// bytes, which then stays in registers (45360 x 2048: 122 us against 132).
constexpr int batch_rows(int element, int per, bool backward) {
  const int n = (element == 4 && !backward ? 64 : 128) / (per * element) / (backward ? 2 : 1);
  return n < 1 ? 1 : n > 4 ? 4 : n;
}

template <int kPass, typename T, int VE, int NV, int F>
cudaError_t run_shape(const NormArgs& a, const Shape& s, int* parts, cudaStream_t st) {
  // Single elements: one row a batch (their loads are not ahead of their use).
  constexpr int most =
      VE == 1 ? 1
      : kPass == kBackwardCodes && sizeof(T) == 2 && VE * NV == 16 && F != kShift
          ? 4   // fewer bytes a row: 45360 x 4096, y and gradients, 288 us against 310 with two
          : batch_rows(sizeof(T), VE * NV, kPass == kBackward || kPass == kBackwardCodes);
  const bool many = batched(a.rows, s, most);
  *parts = grid_for(a.rows, s, many ? most : 1);
  return many ? launch_pass<kPass, T, VE, NV, most, F>(a, s, *parts, st)
              : launch_pass<kPass, T, VE, NV, 1, F>(a, s, *parts, st);
}

template <int kPass, typename T, int VE, int NV>
cudaError_t run_fill(const NormArgs& a, const Shape& s, int* parts, cudaStream_t st) {
  if constexpr (VE > 1) {
    if (s.fill == kAll) return run_shape<kPass, T, VE, NV, kAll>(a, s, parts, st);
    // Shifted rows have four vectors at least, and with a fifth for the shift more
    // than the 32 bf16 that 8 a thread are for.
    if constexpr (kPass != kForwardCodes && VE * NV * (int)sizeof(T) > 16) {
      if (s.fill == kShift) return run_shape<kPass, T, VE, NV, kShift>(a, s, parts, st);
    }
  }
  return run_shape<kPass, T, VE, NV, kSome>(a, s, parts, st);   // single elements too
}

template <int kPass, typename T, int VE>
cudaError_t run_per(NormArgs& a, const Shape& s, int* parts, cudaStream_t st) {
  a.tpr = s.tpr;
  a.kinds = s.kinds;
  if (s.per == 8) return run_fill<kPass, T, VE, 8 / VE>(a, s, parts, st);
  if (s.per == 16) return run_fill<kPass, T, VE, 16 / VE>(a, s, parts, st);
  return run_fill<kPass, T, VE, 32 / VE>(a, s, parts, st);
}

template <int kPass, typename T>
cudaError_t run_type(NormArgs& a, int* parts, cudaStream_t st) {
  constexpr int VE = 16 / (int)sizeof(T);
  a.w_aligned = aligned_to(a.W, 16) && aligned_to(a.bias, 16);
  if (wide<T>(a)) return run_per<kPass, T, VE>(a, shape_for(a.D, VE), parts, st);
  // (A block of codes that is being made needs its elements in neighbouring
  // lanes, which shifted vectors do not give.)
  if (kPass != kForwardCodes && shifted<T>(a)) {
    a.shift = (int)((uintptr_t)a.Y / sizeof(T) % VE);
    return run_per<kPass, T, VE>(a, shape_for(a.D, VE, kinds_for(a.D, VE, a.rows)), parts, st);
  }
  return run_per<kPass, T, 1>(a, shape_for(a.D, 1), parts, st);
}

// The pass over all rows; *parts: CTAs of it, the rows of partial sums.
template <int kPass>
cudaError_t run_pass(int dtype, NormArgs& a, int* parts, cudaStream_t st) {
  return dtype == VDA_DTYPE_BF16 ? run_type<kPass, __nv_bfloat16>(a, parts, st) : run_type<kPass, float>(a, parts, st);
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
}  // namespace vda
