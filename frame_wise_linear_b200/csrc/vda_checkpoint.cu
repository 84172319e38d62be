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

// Units of VE elements, row by row, each row's count rounded up to whole
// blocks so that a block never straddles two warps.
template <typename T, int VE>
__global__ void __launch_bounds__(256) pack_kernel(const T* X, int64_t rows, int D, int64_t ld, uint8_t* codes,
                                                   uint8_t* scales) {
  const int nblk = (D + kBlock - 1) / kBlock;
  const int per_row = nblk * (kBlock / VE);
  const int64_t units = rows * per_row;
  for (int64_t u0 = (int64_t)blockIdx.x * blockDim.x; u0 < units; u0 += (int64_t)gridDim.x * blockDim.x) {
    const int64_t u = u0 + threadIdx.x;
    const int64_t row = u / per_row;
    const int v = (int)(u - row * per_row);
    const bool in = u < units && v * VE < D;
    Pack<T, VE> q;
    if (in) q.load(X + row * ld + (int64_t)v * VE);
    else q.zero();
    float x[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = q.get(i);
    Pack<uint8_t, VE> c;
    const int s = encode_block<VE>(x, c);
    if (in) {
      c.store(codes + row * D + (int64_t)v * VE);
      if (v % (kBlock / VE) == 0) scales[row * nblk + v / (kBlock / VE)] = (uint8_t)s;
    }
  }
}

template <typename T, int VE>
__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows, int D,
                                                     int64_t ld, T* X) {
  const int nblk = (D + kBlock - 1) / kBlock;
  const int per_row = D / VE;
  const int64_t units = rows * per_row;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < units; u += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = u / per_row;
    const int v = (int)(u - row * per_row);
    Pack<uint8_t, VE> c;
    float x[VE];
    c.load(codes + row * D + (int64_t)v * VE);
    decode_pack<VE>(c, scale_of(scales[row * nblk + v / (kBlock / VE)]), x);
    Pack<T, VE> q;
#pragma unroll
    for (int i = 0; i < VE; ++i) q.set(i, x[i]);
    q.store(X + row * ld + (int64_t)v * VE);
  }
}

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <typename T>
bool wide(const void* X, const void* codes, int D, int64_t ld) {
  const int ve = 16 / (int)sizeof(T);
  return D % ve == 0 && ld % ve == 0 && aligned_to(X, 16) && aligned_to(codes, ve);
}

int grid_for(int64_t units) {
  const int64_t b = (units + 255) / 256;
  return (int)(b < 148 * 64 ? b : 148 * 64);
}

template <typename T, int VE>
cudaError_t pack(const vda_checkpoint_problem& p, const void* X, uint8_t* codes, uint8_t* scales, int64_t ld,
                 cudaStream_t st) {
  const int64_t units = p.rows * ((p.D + kBlock - 1) / kBlock * (kBlock / VE));
  pack_kernel<T, VE><<<grid_for(units), 256, 0, st>>>(static_cast<const T*>(X), p.rows, p.D, ld, codes, scales);
  return cudaGetLastError();
}

template <typename T, int VE>
cudaError_t unpack(const vda_checkpoint_problem& p, const uint8_t* codes, const uint8_t* scales, void* X, int64_t ld,
                   cudaStream_t st) {
  unpack_kernel<T, VE><<<grid_for(p.rows * (p.D / VE)), 256, 0, st>>>(codes, scales, p.rows, p.D, ld,
                                                                    static_cast<T*>(X));
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
