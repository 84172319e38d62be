// Activation checkpoints in 8 bits: a [rows, D] tensor into e4m3 codes with a
// power-of-two scale per 32 neighbours of a row (vda_tokops.cuh has the
// format), and back.
//
// Both directions are one pass over the data, bound by HBM: element size + 1
// + 1/32 bytes an element.  Eight neighbouring lanes (float32) or four (bf16)
// hold a block, 16 bytes each, and find its largest magnitude by shuffles; a
// row that is not 16-byte aligned takes one element a lane, a warp a block.
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

template <typename T, int VE>
cudaError_t pack(const vda_checkpoint_problem& p, const void* X, uint8_t* codes, uint8_t* scales, int64_t ld,
                 cudaStream_t st) {
  const Rows r = rows_for(p, ld, VE);
  pack_kernel<T, VE><<<grid_for(r), 256, 0, st>>>(static_cast<const T*>(X), r, codes, scales);
  return cudaGetLastError();
}

template <typename T, int VE>
cudaError_t unpack(const vda_checkpoint_problem& p, const uint8_t* codes, const uint8_t* scales, void* X, int64_t ld,
                   cudaStream_t st) {
  const Rows r = rows_for(p, ld, VE);
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
