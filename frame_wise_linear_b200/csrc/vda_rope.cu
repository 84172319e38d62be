// Rotary positions over three axes (time, height, width) on Q and K, and the
// gradients.
//
// The first d_t + d_y + d_x channels of a head turn in pairs: pair j of axis a
// (j < d_a / 2) by the angle p_a theta^(-2 j / d_a), p_a the token's position
// on the axis; the pairs of time come first, then height's, then width's.
//     (u, v) -> (u cos - v sin, u sin + v cos)
// The other channels are copied.  The turn is orthogonal, so the gradients
// are the gradients of the output turned back (sin negated).
//
// Bound by HBM: every element of Q and K is read and written once.  A thread
// takes one unit of a token (a vector of VE channels and, where pairs are
// half the width apart, its partner vector), computes that unit's sines and
// cosines once and applies them in every head of Q and K, so they cost one
// evaluation per 2 (H_q + H_k) elements moved and stay in registers.
//
// Angles.  position x frequency is formed in turns (frequencies divided by
// 2 pi in double on the host) and in double: at position 10^6 a float32
// product would be off by 0.03 rad, this one by 10^-10.  The whole turns are
// taken off in double; sincospif then sees an argument in [-1, 1].
#include <math.h>

#include "vda_internal.cuh"
#include "vda_tokops.cuh"

namespace vda {
namespace {

using namespace tokops;

constexpr int kMaxPairs = 128;

struct RopeArgs {
  const void* in[2];    // Q, K
  void* out[2];
  const float* positions;   // [B][N][3], or null: the grid's
  int64_t ld_in[2], ld_out[2];   // token-major: elements between tokens
  int64_t N;            // tokens per batch item
  int64_t threads;      // B N units
  int heads[2];         // H_q, H_k
  int d, rot, units, layout, chunk;   // chunk: heads a thread takes (of H_q + H_k)
  int first[3];         // pairs before axis 1, before axis 2, in all
  int height, width;
  float sign;           // -1: the gradients
  double pos0[3], step[3];
  double turns[kMaxPairs];   // frequency / (2 pi) per pair
};

// kHalves: pair j is channels (j, j + rot / 2); a unit is VE of the first and
// their partners, or VE channels behind the turned ones.  Otherwise pair j is
// channels (2 j, 2 j + 1), a unit VE neighbouring channels (VE even).
template <typename T, int VE, bool kHalves>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int NP = kHalves ? VE : (VE + 1) / 2;   // pairs of a unit
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= a.threads) return;
  const int64_t token = id / a.units;   // over all batch items
  const int unit = (int)(id - token * a.units);
  const int64_t item = token / a.N, tok = token - item * a.N;
  double pos[3];
  if (a.positions) {
#pragma unroll
    for (int i = 0; i < 3; ++i) pos[i] = (double)a.positions[token * 3 + i];
  } else {
    const int64_t row = tok / a.width;
    const int64_t t = row / a.height;
    pos[0] = a.pos0[0] + a.step[0] * (double)t;
    pos[1] = a.pos0[1] + a.step[1] * (double)(row - t * a.height);
    pos[2] = a.pos0[2] + a.step[2] * (double)(tok - row * a.width);
  }
  const int half = a.rot / 2;
  // Channels of the unit, and of its partner where there is one.
  const int lo = kHalves && unit * VE >= half ? a.rot + unit * VE - half : unit * VE;
  const int hi = kHalves && unit * VE < half ? lo + half : -1;
  float c[NP], s[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int j = kHalves ? unit * VE + k : unit * (VE / 2) + k;
    if (j < half) {
      const double at = j >= a.first[1] ? pos[2] : (j >= a.first[0] ? pos[1] : pos[0]);
      const double turn = at * a.turns[j];
      sincospif((float)(2.0 * (turn - rint(turn))), &s[k], &c[k]);
      s[k] *= a.sign;
    } else {
      c[k] = 1.f;
      s[k] = 0.f;
    }
  }
  const int turned = kHalves ? (hi >= 0 ? VE : 0) : (half - unit * (VE / 2));   // pairs of the unit that turn
  const int h0 = (int)blockIdx.y * a.chunk;
  const int total = a.heads[0] + a.heads[1];
  const int h1 = h0 + a.chunk < total ? h0 + a.chunk : total;
#pragma unroll 4
  for (int hh = h0; hh < h1; ++hh) {
    const int which = hh >= a.heads[0] ? 1 : 0;
    const int h = hh - (which ? a.heads[0] : 0), H = a.heads[which];
    const int64_t dense = ((item * H + h) * a.N + tok) * a.d;
    const T* in = static_cast<const T*>(a.in[which]) + (a.layout ? token * a.ld_in[which] + (int64_t)h * a.d : dense);
    T* out = static_cast<T*>(a.out[which]) + (a.layout ? token * a.ld_out[which] + (int64_t)h * a.d : dense);
    if constexpr (kHalves) {
      Pack<T, VE> x, y;
      x.load(in + lo);
      if (hi >= 0) {
        y.load(in + hi);
        Pack<T, VE> u, v;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          u.set(k, x.get(k) * c[k] - y.get(k) * s[k]);
          v.set(k, x.get(k) * s[k] + y.get(k) * c[k]);
        }
        u.store(out + lo);
        v.store(out + hi);
      } else {
        x.store(out + lo);
      }
    } else {
      Pack<T, VE> x, u;
      x.load(in + lo);
#pragma unroll
      for (int k = 0; k < VE / 2; ++k) {
        if (k < turned) {
          u.set(2 * k, x.get(2 * k) * c[k] - x.get(2 * k + 1) * s[k]);
          u.set(2 * k + 1, x.get(2 * k) * s[k] + x.get(2 * k + 1) * c[k]);
        } else {   // copied as they are, not multiplied by (1, 0)
          u.e[2 * k] = x.e[2 * k];
          u.e[2 * k + 1] = x.e[2 * k + 1];
        }
      }
      u.store(out + lo);
    }
  }
}

// Neighbouring pairs at any alignment: one pair (or the last channel of an
// odd d) a thread, element by element.
template <typename T>
__global__ void __launch_bounds__(256) rope_pair_kernel(const __grid_constant__ RopeArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= a.threads) return;
  const int64_t token = id / a.units;
  const int j = (int)(id - token * a.units);
  const int64_t item = token / a.N, tok = token - item * a.N;
  float c = 1.f, s = 0.f;
  const bool turned = j < a.rot / 2;
  if (turned) {
    const int axis = j >= a.first[1] ? 2 : (j >= a.first[0] ? 1 : 0);
    double pos;
    if (a.positions) {
      pos = (double)a.positions[token * 3 + axis];
    } else {
      const int64_t row = tok / a.width, t = row / a.height;
      pos = a.pos0[axis] + a.step[axis] * (double)(axis == 0 ? t : (axis == 1 ? row - t * a.height : tok - row * a.width));
    }
    const double turn = pos * a.turns[j];
    sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
    s *= a.sign;
  }
  const bool two = 2 * j + 1 < a.d;
  const int h0 = (int)blockIdx.y * a.chunk;
  const int total = a.heads[0] + a.heads[1];
  const int h1 = h0 + a.chunk < total ? h0 + a.chunk : total;
#pragma unroll 4
  for (int hh = h0; hh < h1; ++hh) {
    const int which = hh >= a.heads[0] ? 1 : 0;
    const int h = hh - (which ? a.heads[0] : 0), H = a.heads[which];
    const int64_t dense = ((item * H + h) * a.N + tok) * a.d;
    const T* in = static_cast<const T*>(a.in[which]) + (a.layout ? token * a.ld_in[which] + (int64_t)h * a.d : dense);
    T* out = static_cast<T*>(a.out[which]) + (a.layout ? token * a.ld_out[which] + (int64_t)h * a.d : dense);
    const T x = in[2 * j];
    const T y = two ? in[2 * j + 1] : x;
    if (turned) {
      out[2 * j] = from_f32<T>(to_f32(x) * c - to_f32(y) * s);
      out[2 * j + 1] = from_f32<T>(to_f32(x) * s + to_f32(y) * c);
    } else {
      out[2 * j] = x;
      if (two) out[2 * j + 1] = y;
    }
  }
}

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Launch: threads along x, and along y as many slices of the heads as it
// takes to give every SM work where there are few tokens.
template <typename Kernel>
cudaError_t launch(Kernel k, RopeArgs& a, int64_t tokens, int units, cudaStream_t st) {
  a.units = units;
  a.threads = tokens * units;
  const int64_t bx = (a.threads + 255) / 256;
  const int total = a.heads[0] + a.heads[1];
  int chunk = total;
  while (chunk > 1 && bx * ((total + chunk - 1) / chunk) < 148 * 8) chunk = (chunk + 1) / 2;
  a.chunk = chunk;
  k<<<dim3((unsigned)bx, (unsigned)((total + chunk - 1) / chunk)), 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(RopeArgs& a, int64_t tokens, int pairing, cudaStream_t st) {
  const int ve = 16 / (int)sizeof(T);
  // The widest vector that every row start, stride and the width allow.
  auto fits = [&](int n) {
    if (a.d % n) return false;
    if (pairing == VDA_ROPE_HALVES && (a.rot / 2) % n) return false;
    for (int i = 0; i < 2; ++i) {
      if (!a.heads[i]) continue;
      if (a.layout && (a.ld_in[i] % n || a.ld_out[i] % n)) return false;
      if (!aligned_to(a.in[i], n * sizeof(T)) || !aligned_to(a.out[i], n * sizeof(T))) return false;
    }
    return true;
  };
  if (pairing == VDA_ROPE_HALVES) {
    auto units = [&](int n) { return a.rot / 2 / n + (a.d - a.rot) / n; };
    if constexpr (sizeof(T) == 2) {
      if (fits(8)) return launch(rope_kernel<T, 8, true>, a, tokens, units(8), st);
    }
    if (fits(4)) return launch(rope_kernel<T, 4, true>, a, tokens, units(4), st);
    if (fits(2)) return launch(rope_kernel<T, 2, true>, a, tokens, units(2), st);
    return launch(rope_kernel<T, 1, true>, a, tokens, units(1), st);
  }
  if (fits(ve)) return launch(rope_kernel<T, 16 / (int)sizeof(T), false>, a, tokens, a.d / ve, st);
  if (fits(2)) return launch(rope_kernel<T, 2, false>, a, tokens, a.d / 2, st);
  return launch(rope_pair_kernel<T>, a, tokens, (a.d + 1) / 2, st);
}

}  // namespace

cudaError_t launch_rope(const vda_rope_problem& p, const void* Q, const void* K, const float* positions, void* Qo,
                        void* Ko, bool backward, cudaStream_t st) {
  RopeArgs a{};
  a.N = (int64_t)p.T * p.height * p.width;
  const int64_t tokens = p.B * a.N;
  if (tokens == 0 || p.H_q + p.H_k == 0) return cudaSuccess;
  a.in[0] = Q;
  a.in[1] = K;
  a.out[0] = Qo;
  a.out[1] = Ko;
  a.positions = positions;
  a.heads[0] = p.H_q;
  a.heads[1] = p.H_k;
  a.d = p.d;
  a.rot = p.d_t + p.d_y + p.d_x;
  a.layout = p.layout;
  a.height = p.height;
  a.width = p.width;
  a.sign = backward ? -1.f : 1.f;
  const int64_t plain[2] = {p.ld_q, p.ld_k}, turned[2] = {p.ld_qr, p.ld_kr};
  for (int i = 0; i < 2; ++i) {
    const int64_t dense = (int64_t)a.heads[i] * p.d;
    const int64_t u = plain[i] ? plain[i] : dense, v = turned[i] ? turned[i] : dense;
    a.ld_in[i] = backward ? v : u;
    a.ld_out[i] = backward ? u : v;
  }
  const int n[3] = {p.d_t, p.d_y, p.d_x};
  int j = 0;
  for (int ax = 0; ax < 3; ++ax) {
    for (int i = 0; i < n[ax] / 2; ++i) a.turns[j++] = pow(p.theta, -2.0 * i / n[ax]) / (2.0 * M_PI);
    a.first[ax] = j;
    a.pos0[ax] = p.pos0[ax];
    a.step[ax] = p.step[ax];
  }
  return p.dtype == VDA_DTYPE_BF16 ? run<__nv_bfloat16>(a, tokens, p.pairing, st)
                                   : run<float>(a, tokens, p.pairing, st);
}

}  // namespace vda
