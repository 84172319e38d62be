// Activation checkpoints in 8 bits: a [rows, D] tensor into e4m3 codes with a
// power-of-two scale per 32 neighbours of a row (vda_tokops.cuh has the
// format), and back.
//
// Both directions are one pass over the data, bound by HBM: element size + 1
// + 1/32 bytes an element.  Three forms, by alignment alone:
//   - rows of 16-byte vectors: eight neighbouring lanes (float32) or four (bf16)
//     hold a block, 16 bytes each, and find its largest magnitude by shuffles
//     (1451520 x 128 bf16, both directions: 185 to 190 us, 0.93 to 0.90 of the
//     copy rate);
//   - dense rows at any alignment (odd widths): a CTA's blocks are one stretch of
//     memory, copied through shared memory 16 bytes at a time on both sides.
//     Elements pass shared memory one by one and codes byte by byte, 42 and 29
//     instructions of a warp for 32 bf16 elements, which bound it (45360 x 4090
//     bf16, both directions: 414 us, 0.41; 22680 x 4095 float32: 231 us, 0.62);
//   - rows with gaps at any alignment: one element a lane, a warp a block (45360 x
//     4090 bf16 with rows 4091 apart: 1245 us, 0.14).
#include "vda_internal.cuh"
#include "vda_tokops.cuh"

namespace vda {
namespace {

using namespace tokops;

// A unit is VE elements of a row; a row's count is rounded up to whole blocks,
// so that a block's lanes are neighbours in one warp.
struct Rows {
  int64_t units;      // of all rows
  int per_row;        // units of a row
  uint64_t by;        // ceil(2^64 / per_row) where the quotient by it is exact, else 0
  int64_t ld;         // of the tensor
  int D, nblk;
  int flat;           // blocks of a CTA in the any-alignment form, at most kFlat
  int whole;          // codes and tensor are dense and D is whole blocks: unit u is elements u VE ..
};

template <int VE>
struct Unit {
  int64_t row;
  int v;
  bool in;
  int64_t at, code, scale;   // element offsets in the tensor and the codes, and the scale byte's
  __device__ __forceinline__ Unit(const Rows& r, int64_t u) {
    if (r.whole) {
      in = u < r.units;
      at = code = u * VE;
      scale = u / (kBlock / VE);
      return;
    }
    row = r.by ? (int64_t)__umul64hi((uint64_t)u, r.by) : u / r.per_row;
    v = (int)(u - row * r.per_row);
    in = u < r.units && v * VE < r.D;
    at = row * r.ld + v * VE;
    code = row * r.D + v * VE;
    scale = row * r.nblk + v / (kBlock / VE);
  }
};

constexpr int kUnits = 4;   // of a thread, all on their way before the first is used

template <typename T, int VE>
__global__ void __launch_bounds__(256) pack_kernel(const T* X, const Rows r, uint8_t* codes, uint8_t* scales) {
  const int64_t u0 = (int64_t)blockIdx.x * (256 * kUnits) + threadIdx.x;
  Pack<T, VE> q[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Unit<VE> u(r, u0 + j * 256);
    q[j].zero();
    if (u.in) q[j].load(X + u.at);
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Unit<VE> u(r, u0 + j * 256);
    float x[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = q[j].get(i);
    Pack<uint8_t, VE> c;
    const int s = encode_block<VE, false>(x, c, 0xffffffffu);
    if (u.in) {
      c.store(codes + u.code);
      if (threadIdx.x % (kBlock / VE) == 0) scales[u.scale] = (uint8_t)s;
    }
  }
}

template <typename T, int VE>
__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t* codes, const uint8_t* scales, const Rows r, T* X) {
  const int64_t u0 = (int64_t)blockIdx.x * (256 * kUnits) + threadIdx.x;
  Pack<uint8_t, VE> c[kUnits];
  int s[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Unit<VE> u(r, u0 + j * 256);
    c[j].zero();
    s[j] = 0;
    if (u.in) {
      c[j].load(codes + u.code);
      s[j] = scales[u.scale];
    }
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const Unit<VE> u(r, u0 + j * 256);
    float2 x[VE > 1 ? VE / 2 : 1];
    decode_pairs<VE>(c[j], x);
    const float2 scale = both(scale_of(s[j]));
    Pack<T, VE> q;
    if constexpr (VE > 1) {
#pragma unroll
      for (int i = 0; i < VE; i += 2) q.set2(i, mul2(x[i / 2], scale));
    } else {
      q.set(0, x[0].x * scale.x);
    }
    if (u.in) q.store(X + u.at);
  }
}

// ---- dense rows at any alignment
constexpr int kFlat = 256;                 // blocks of a CTA, at most
constexpr int kStretch = kFlat * kBlock;   // their elements

// The elements of blocks b0 .. b0 + count - 1: neighbours in memory, from
// element `first` on; block i starts `offs[i]` elements behind it, and
// offs[count] is their number.
struct Stretch {
  int64_t first, row0;   // row0: the first block's row
  int count;
};
// `in_row`, where given: each block's row, counted from the first one's.
__device__ __forceinline__ Stretch stretch_of(const Rows& r, int64_t rows, int* offs, int* in_row = nullptr) {
  const int64_t b0 = (int64_t)blockIdx.x * r.flat, row0 = b0 / r.nblk;
  const int col0 = (int)(b0 - row0 * r.nblk);   // first block's place in its row
  const int64_t left = rows * r.nblk - b0;
  const int count = left < r.flat ? (int)left : r.flat;
  for (int i = threadIdx.x; i <= count; i += 256) {
    const int n = col0 + i, row = n / r.nblk, col = n - row * r.nblk;
    offs[i] = row * r.D + (col - col0) * kBlock;   // below kStretch: full blocks, or short ones
    if (in_row) in_row[i] = row;
  }
  return Stretch{row0 * r.D + (int64_t)col0 * kBlock, row0, count};
}

// n elements between global memory at `g` and shared memory, where element j
// is at byte (g & 15) + j sizeof(T): 16 bytes at a time, single elements where
// a vector at either end holds others too.
template <typename T>
__device__ __forceinline__ void stretch_in(const T* g, int n, uint8_t* shared) {
  const int shift = (int)((uintptr_t)g & 15), bytes = shift + n * (int)sizeof(T);
  const uint8_t* base = reinterpret_cast<const uint8_t*>(g) - shift;
  for (int v = threadIdx.x * 16; v < bytes; v += 256 * 16) {
    if (v >= shift && v + 16 <= bytes) {
      async_copy<16>(shared + v, base + v);
    } else {
      const int end = v + 16 < bytes ? v + 16 : bytes;
      for (int b = v < shift ? shift : v; b < end; b += (int)sizeof(T))
        *reinterpret_cast<T*>(shared + b) = *reinterpret_cast<const T*>(base + b);
    }
  }
  async_commit();
  async_wait<0>();
}
template <typename T>
__device__ __forceinline__ void stretch_out(T* g, int n, const uint8_t* shared) {
  const int shift = (int)((uintptr_t)g & 15), bytes = shift + n * (int)sizeof(T);
  uint8_t* base = reinterpret_cast<uint8_t*>(g) - shift;
  for (int v = threadIdx.x * 16; v < bytes; v += 256 * 16) {
    if (v >= shift && v + 16 <= bytes) {
      *reinterpret_cast<uint4*>(base + v) = *reinterpret_cast<const uint4*>(shared + v);
    } else {
      const int end = v + 16 < bytes ? v + 16 : bytes;
      for (int b = v < shift ? shift : v; b < end; b += (int)sizeof(T))
        *reinterpret_cast<T*>(base + b) = *reinterpret_cast<const T*>(shared + b);
    }
  }
}

// A block is eight neighbouring lanes', four elements each; lane q of group
// `sub` takes elements q + 8 ((m + sub) & 3), m < 4, so that the four groups of
// a warp read different banks.
__device__ __forceinline__ int element_of(int lane, int m) { return (lane & 7) + 8 * ((m + (lane >> 3)) & 3); }

// kNorm: packs (x - mean) rstd, each row with its own, in place of x.
template <typename T, bool kNorm>
__global__ void __launch_bounds__(256) pack_flat_kernel(const T* X, const Rows r, int64_t rows, const float* mean,
                                                        const float* rstd, uint8_t* codes, uint8_t* scales) {
  __shared__ __align__(16) uint8_t in[kStretch * sizeof(T) + 16], out[kStretch + 16];
  __shared__ int offs[kFlat + 1], in_row[kNorm ? kFlat + 1 : 1];
  __shared__ uint8_t sb[kFlat];
  const Stretch st = stretch_of(r, rows, offs, kNorm ? in_row : nullptr);
  __syncthreads();
  const int n = offs[st.count];
  stretch_in(X + st.first, n, in);
  __syncthreads();
  const T* x = reinterpret_cast<const T*>(in + ((uintptr_t)(X + st.first) & 15));
  uint8_t* c = out + ((uintptr_t)(codes + st.first) & 15);
  const int lane = threadIdx.x & 31;
  for (int i0 = threadIdx.x >> 5 << 2; i0 < st.count; i0 += 32) {
    const int i = i0 + (lane >> 3);
    const int at = offs[i < st.count ? i : st.count], size = i < st.count ? offs[i + 1] - at : 0;
    float shift = 0.f, factor = 1.f;
    if constexpr (kNorm) {
      if (i < st.count) {
        shift = -mean[st.row0 + in_row[i]];
        factor = rstd[st.row0 + in_row[i]];
      }
    }
    float v[4];   // zeros behind the row's end
    float top = 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int e = element_of(lane, m);
      v[m] = e < size ? to_f32(x[at + e]) : 0.f;
      if constexpr (kNorm) v[m] = e < size ? (v[m] + shift) * factor : 0.f;
      top = fmaxf(top, fabsf(v[m]));
    }
    top = lanes_max<8>(top, 0xffffffffu);
    int s = scale_byte(top);
    uint32_t two[2];
    if (top <= kLargeTop) {
      const float2 inv = both(inv_scale_of(s));
      two[0] = encode2(mul2(make_float2(v[0], v[1]), inv));
      two[1] = encode2(mul2(make_float2(v[2], v[3]), inv));
    } else {
      top = fmaxf(fmaxf(block_mag(v[0]), block_mag(v[1])), fmaxf(block_mag(v[2]), block_mag(v[3])));
      top = lanes_max<8>(top, lane_group<8>());
      s = scale_byte(top);
      two[0] = encode2_any(make_float2(v[0], v[1]), inv_scale_of(s), s);
      two[1] = encode2_any(make_float2(v[2], v[3]), inv_scale_of(s), s);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int e = element_of(lane, m);
      if (e < size) c[at + e] = (uint8_t)(two[m / 2] >> (8 * (m % 2)));
    }
    if ((lane & 7) == 0 && i < st.count) sb[i] = (uint8_t)s;
  }
  __syncthreads();
  stretch_out(codes + st.first, n, out);
  if ((int)threadIdx.x < st.count) scales[(int64_t)blockIdx.x * r.flat + threadIdx.x] = sb[threadIdx.x];
}

template <typename T>
__global__ void __launch_bounds__(256) unpack_flat_kernel(const uint8_t* codes, const uint8_t* scales, const Rows r,
                                                          int64_t rows, T* X) {
  __shared__ __align__(16) uint8_t out[kStretch * sizeof(T) + 16], in[kStretch + 16];
  __shared__ int offs[kFlat + 1];
  __shared__ uint8_t sb[kFlat];
  const Stretch st = stretch_of(r, rows, offs);
  if ((int)threadIdx.x < st.count) sb[threadIdx.x] = scales[(int64_t)blockIdx.x * r.flat + threadIdx.x];
  __syncthreads();
  const int n = offs[st.count];
  stretch_in(codes + st.first, n, in);
  __syncthreads();
  T* x = reinterpret_cast<T*>(out + ((uintptr_t)(X + st.first) & 15));
  const uint8_t* c = in + ((uintptr_t)(codes + st.first) & 15);
  const int lane = threadIdx.x & 31;
  for (int i0 = threadIdx.x >> 5 << 2; i0 < st.count; i0 += 32) {
    const int i = i0 + (lane >> 3);
    if (i >= st.count) break;
    const int at = offs[i], size = offs[i + 1] - at;
    const float2 scale = both(scale_of(sb[i]));
#pragma unroll
    for (int m = 0; m < 4; m += 2) {
      const int e0 = element_of(lane, m), e1 = element_of(lane, m + 1);
      const uint32_t c0 = e0 < size ? c[at + e0] : 0, c1 = e1 < size ? c[at + e1] : 0;
      const float2 v = mul2(decode2(c0 | c1 << 8), scale);
      if (e0 < size) x[at + e0] = from_f32<T>(v.x);
      if (e1 < size) x[at + e1] = from_f32<T>(v.y);
    }
  }
  __syncthreads();
  stretch_out(X + st.first, n, out);
}

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <typename T>
bool wide(const void* X, const void* codes, int D, int64_t ld) {
  const int ve = 16 / (int)sizeof(T);
  return D % ve == 0 && ld % ve == 0 && aligned_to(X, 16) && aligned_to(codes, ve);
}

Rows rows_for(const vda_checkpoint_problem& p, int64_t ld, int ve) {
  Rows r{};
  r.nblk = (p.D + kBlock - 1) / kBlock;
  r.per_row = r.nblk * (kBlock / ve);
  r.units = p.rows * r.per_row;
  r.ld = ld;
  r.D = p.D;
  r.whole = ld == p.D && p.D % kBlock == 0;
  // u * ceil(2^64 / n) >> 64 = u / n while u n < 2^64.
  if (r.per_row > 1 && r.units <= (1LL << 62) / r.per_row) r.by = ~0ull / (uint64_t)r.per_row + 1;
  return r;
}

// CTAs of 256 threads: below 2^31, as there are fewer than 2^36 blocks of at most 32 units.
unsigned grid_for(const Rows& r) { return (unsigned)((r.units + 256 * kUnits - 1) / (256 * kUnits)); }

// Blocks of a CTA: 256, or fewer, down to the 32 that eight warps take at once,
// until there are two CTAs for an SM (257 x 1001 float32: 8.6 us with 256).
unsigned flat_grid(const vda_checkpoint_problem& p, Rows& r) {
  const int64_t blocks = p.rows * r.nblk;
  r.flat = kFlat;
  while (r.flat > 32 && blocks < 148LL * 2 * r.flat) r.flat /= 2;
  return (unsigned)((blocks + r.flat - 1) / r.flat);
}

template <typename T, int VE>
cudaError_t pack(const vda_checkpoint_problem& p, const void* X, uint8_t* codes, uint8_t* scales, int64_t ld,
                 cudaStream_t st) {
  Rows r = rows_for(p, ld, VE);
  if (VE == 1 && ld == p.D) {
    const unsigned grid = flat_grid(p, r);
    pack_flat_kernel<T, false><<<grid, 256, 0, st>>>(static_cast<const T*>(X), r, p.rows, nullptr, nullptr, codes,
                                                     scales);
    return cudaGetLastError();
  }
  pack_kernel<T, VE><<<grid_for(r), 256, 0, st>>>(static_cast<const T*>(X), r, codes, scales);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pack_normalised(const vda_checkpoint_problem& p, const void* X, const float* mean, const float* rstd,
                            uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  Rows r = rows_for(p, p.D, 1);
  const unsigned grid = flat_grid(p, r);
  pack_flat_kernel<T, true><<<grid, 256, 0, st>>>(static_cast<const T*>(X), r, p.rows, mean, rstd, codes, scales);
  return cudaGetLastError();
}

template <typename T, int VE>
cudaError_t unpack(const vda_checkpoint_problem& p, const uint8_t* codes, const uint8_t* scales, void* X, int64_t ld,
                   cudaStream_t st) {
  Rows r = rows_for(p, ld, VE);
  if (VE == 1 && ld == p.D) {
    const unsigned grid = flat_grid(p, r);
    unpack_flat_kernel<T><<<grid, 256, 0, st>>>(codes, scales, r, p.rows, static_cast<T*>(X));
    return cudaGetLastError();
  }
  unpack_kernel<T, VE><<<grid_for(r), 256, 0, st>>>(codes, scales, r, static_cast<T*>(X));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_checkpoint_pack(const vda_checkpoint_problem& p, const void* X, uint8_t* codes, uint8_t* scales,
                                   cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  const int64_t ld = p.ld ? p.ld : p.D;
  if (p.dtype == VDA_DTYPE_BF16)
    return wide<__nv_bfloat16>(X, codes, p.D, ld) ? pack<__nv_bfloat16, 8>(p, X, codes, scales, ld, st)
                                                  : pack<__nv_bfloat16, 1>(p, X, codes, scales, ld, st);
  return wide<float>(X, codes, p.D, ld) ? pack<float, 4>(p, X, codes, scales, ld, st)
                                        : pack<float, 1>(p, X, codes, scales, ld, st);
}

cudaError_t launch_checkpoint_pack_normalised(const vda_checkpoint_problem& p, const void* X, const float* mean,
                                              const float* rstd, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  return p.dtype == VDA_DTYPE_BF16 ? pack_normalised<__nv_bfloat16>(p, X, mean, rstd, codes, scales, st)
                                   : pack_normalised<float>(p, X, mean, rstd, codes, scales, st);
}

cudaError_t launch_checkpoint_unpack(const vda_checkpoint_problem& p, const uint8_t* codes, const uint8_t* scales,
                                     void* X, cudaStream_t st) {
  if (p.rows == 0) return cudaSuccess;
  const int64_t ld = p.ld ? p.ld : p.D;
  if (p.dtype == VDA_DTYPE_BF16)
    return wide<__nv_bfloat16>(X, codes, p.D, ld) ? unpack<__nv_bfloat16, 8>(p, codes, scales, X, ld, st)
                                                  : unpack<__nv_bfloat16, 1>(p, codes, scales, X, ld, st);
  return wide<float>(X, codes, p.D, ld) ? unpack<float, 4>(p, codes, scales, X, ld, st)
                                        : unpack<float, 1>(p, codes, scales, X, ld, st);
}

}  // namespace vda
