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
// Bound by HBM: every element of Q and K is read and written once.  A CTA takes
// a tile of tokens in all heads of Q and K: it computes the tile's cosines and
// sines once, into shared memory, while its first loads are on their way.  A
// thread then stays with one unit of one token (a vector of VE channels and,
// where pairs are half the width apart, its partner vector), holds that unit's
// cosines and sines in registers and walks over heads, the next kAhead heads
// on their way while it turns the last ones.
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
  uint32_t N, tokens;   // per batch item, and of all: below 2^31
  int heads[2];         // H_q, H_k
  int d, rot, units, layout;
  int tile, lanes;      // tokens of a CTA; threads that share a unit of a token, each with every lanes-th head
  int first[3];         // pairs before axis 1, before axis 2, in all
  int height, width;
  float sign;           // -1: the gradients
  double pos0[3], step[3];
  double turns[kMaxPairs];   // frequency / (2 pi) per pair
};

// Cosine and sine of pair j at a token.
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, uint32_t token, int j) {
  const int axis = j >= a.first[1] ? 2 : (j >= a.first[0] ? 1 : 0);
  double pos;
  if (a.positions) {
    pos = (double)a.positions[(int64_t)token * 3 + axis];
  } else {
    const uint32_t tok = token % a.N, row = tok / (uint32_t)a.width, t = row / (uint32_t)a.height;
    const uint32_t i = axis == 0 ? t : (axis == 1 ? row - t * a.height : tok - row * a.width);
    pos = a.pos0[axis] + a.step[axis] * (double)i;
  }
  const double turn = pos * a.turns[j];
  float s, c;
  sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
  return make_float2(c, s * a.sign);
}

// The unit of a thread in each head it takes.
//   kHalves: pair j is channels (j, j + rot / 2); a unit is VE of the first and
//   their partners, or VE channels behind the turned ones.
//   Else: pair j is channels (2 j, 2 j + 1); a unit is VE neighbours, or (kPair)
//   one pair loaded as single elements, or the last channel of an odd d.
// Four CTAs of an SM: with the 80 registers that the compiler would take 8191
// packed tokens take 20.6 us against 18.9, with five CTAs it spills (31 us).  At
// four the 16-byte form of kHalves spills, too: 40 bytes a thread, 48 read back.
// 768p: neighbours 223 us, 1.02 of the copy rate; halves 235 us, 0.96.
template <typename T, int VE, bool kHalves, bool kPair>
__global__ void __launch_bounds__(256, 4) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int NP = kHalves ? VE : (kPair ? 1 : VE / 2);   // pairs of a unit
  constexpr int kLoad = kPair ? 1 : VE;                      // elements of a load
  // Heads on their way: 64 bytes of a thread's loads (with 32 the turned heads
  // wait, 768p 224 us against 218; with 128 registers cost occupancy, 234 us), at
  // most four heads, and two where pairs are loaded element by element.
  constexpr int kLoadBytes = (kHalves || kPair ? 2 : 1) * (kPair ? 1 : VE) * (int)sizeof(T);
  constexpr int kAhead = kHalves && VE == 1 ? 2 : 64 / kLoadBytes < 4 ? 64 / kLoadBytes : 4;
  extern __shared__ float2 table[];   // [tile][rot / 2]
  const int half = a.rot / 2;
  const uint32_t token0 = blockIdx.x * (uint32_t)a.tile;
  // Neighbouring threads: the units of a head, then the lanes' heads, then the tokens.
  const int c0 = (int)threadIdx.x / a.units, unit = (int)threadIdx.x - c0 * a.units;
  const int local = c0 / a.lanes, lane = c0 - local * a.lanes;
  const uint32_t token = token0 + local;
  const bool live = local < a.tile && token < a.tokens;
  // Channels of the unit's two loads (the second: the partner, if any).
  int lo, hi = -1;
  if constexpr (kHalves) {
    lo = unit * VE < half ? unit * VE : a.rot + unit * VE - half;
    if (unit * VE < half) hi = lo + half;
  } else {
    lo = unit * (kPair ? 2 : VE);
    if (kPair && lo + 1 < a.d) hi = lo + 1;
  }
  // Element offset of the token in head 0, and from head to head.
  int64_t at_in[2], at_out[2], next;
  if (a.layout) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      at_in[i] = (int64_t)token * a.ld_in[i] + lo;
      at_out[i] = (int64_t)token * a.ld_out[i] + lo;
    }
    next = a.d;
  } else {
    const int64_t item = token / a.N;
#pragma unroll
    for (int i = 0; i < 2; ++i) at_in[i] = at_out[i] = (item * (a.heads[i] - 1) * a.N + token) * a.d + lo;
    next = (int64_t)a.N * a.d;
  }
  const int total = live ? a.heads[0] + a.heads[1] : 0, step = hi - lo;
  auto input = [&](int h) {
    return h < a.heads[0] ? static_cast<const T*>(a.in[0]) + at_in[0] + h * next
                          : static_cast<const T*>(a.in[1]) + at_in[1] + (h - a.heads[0]) * next;
  };
  auto output = [&](int h) {
    return h < a.heads[0] ? static_cast<T*>(a.out[0]) + at_out[0] + h * next
                          : static_cast<T*>(a.out[1]) + at_out[1] + (h - a.heads[0]) * next;
  };
  constexpr bool kTwo = kHalves || kPair;
  Pack<T, kLoad> x[kAhead], y[kTwo ? kAhead : 1];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * a.lanes;
      if (h < total) {
        const T* p = input(h);
        x[i].load(p);
        if constexpr (kTwo) {
          if (hi >= 0) y[i].load(p + step);
        }
      }
    }
  };
  load(lane);
  for (int e = threadIdx.x; e < a.tile * half; e += 256) {
    const int tl = e / half;
    if (token0 + tl < a.tokens) table[e] = turn_of(a, token0 + tl, e - tl * half);
  }
  __syncthreads();
  const int first_pair = kHalves ? unit * VE : lo / 2;
  const int turned = kHalves ? (hi >= 0 ? VE : 0) : half - first_pair;   // pairs of the unit that turn
  float2 cs[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) cs[k] = live && k < turned ? table[local * half + first_pair + k] : make_float2(1.f, 0.f);
  for (int h0 = lane; h0 < total; h0 += kAhead * a.lanes) {
    Pack<T, kLoad> u[kAhead], v[kTwo ? kAhead : 1];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if constexpr (kTwo) {
        u[i] = x[i];
        v[i] = y[i];
        if (turned > 0) {
          if constexpr (kLoad > 1) {
#pragma unroll
            for (int k = 0; k < NP; k += 2) {
              const float2 p = x[i].get2(k), q = y[i].get2(k);
              const float2 c2 = make_float2(cs[k].x, cs[k + 1].x), s2 = make_float2(cs[k].y, cs[k + 1].y);
              const float2 qs = mul2(q, s2), qc = mul2(q, c2);
              u[i].set2(k, fma2(p, c2, make_float2(-qs.x, -qs.y)));
              v[i].set2(k, fma2(p, s2, qc));
            }
          } else {
            u[i].set(0, x[i].get(0) * cs[0].x - y[i].get(0) * cs[0].y);
            v[i].set(0, x[i].get(0) * cs[0].y + y[i].get(0) * cs[0].x);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          if (k < turned) {
            const float2 v = x[i].get2(2 * k);
            const float p = v.x, q = v.y;
            u[i].set2(2 * k, make_float2(p * cs[k].x - q * cs[k].y, p * cs[k].y + q * cs[k].x));
          } else {   // copied as they are, not multiplied by (1, 0)
            u[i].e[2 * k] = x[i].e[2 * k];
            u[i].e[2 * k + 1] = x[i].e[2 * k + 1];
          }
        }
      }
    }
    load(h0 + kAhead * a.lanes);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * a.lanes;
      if (h < total) {
        T* p = output(h);
        u[i].store(p);
        if constexpr (kTwo) {
          if (hi >= 0) v[i].store(p + step);
        }
      }
    }
  }
}

bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Tokens of a CTA, and threads that share a unit: four, so that the CTA reads
// and writes 1 KB of a token at a time (768p: 218 us; 226 with two, 235 with
// one; with eight 213, but a sequence of 8192 tokens 23 us against 20), and
// more where there would be fewer than two CTAs for an SM (one frame of 1008
// tokens: 7 us; with eight CTAs for an SM small clips pay for the CTAs, 5.1 us
// against 3.4).
template <typename Kernel>
cudaError_t launch(Kernel k, RopeArgs& a, int units, cudaStream_t st) {
  a.units = units;
  a.tile = 256 / (units * 4);
  if (a.tile < 1) a.tile = 1;
  while (a.tile > 1 && (a.tokens + a.tile - 1) / a.tile < 148 * 2) a.tile = (a.tile + 1) / 2;
  a.lanes = 256 / (a.tile * units);
  const uint32_t grid = (a.tokens + a.tile - 1) / a.tile;
  k<<<grid, 256, (size_t)a.tile * (a.rot / 2) * sizeof(float2), st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(RopeArgs& a, int pairing, cudaStream_t st) {
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
      if (fits(8)) return launch(rope_kernel<T, 8, true, false>, a, units(8), st);
    }
    if (fits(4)) return launch(rope_kernel<T, 4, true, false>, a, units(4), st);
    if (fits(2)) return launch(rope_kernel<T, 2, true, false>, a, units(2), st);
    return launch(rope_kernel<T, 1, true, false>, a, units(1), st);
  }
  if (fits(ve)) return launch(rope_kernel<T, 16 / (int)sizeof(T), false, false>, a, a.d / ve, st);
  if (fits(2)) return launch(rope_kernel<T, 2, false, false>, a, a.d / 2, st);
  return launch(rope_kernel<T, 2, false, true>, a, (a.d + 1) / 2, st);
}

}  // namespace

cudaError_t launch_rope(const vda_rope_problem& p, const void* Q, const void* K, const float* positions, void* Qo,
                        void* Ko, bool backward, cudaStream_t st) {
  if (!p.B || !p.T || !p.height || !p.width || p.H_q + p.H_k == 0) return cudaSuccess;
  RopeArgs a{};
  a.N = (uint32_t)((int64_t)p.T * p.height * p.width);   // B N is below 2^31
  a.tokens = (uint32_t)p.B * a.N;
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
  return p.dtype == VDA_DTYPE_BF16 ? run<__nv_bfloat16>(a, p.pairing, st)
                                   : run<float>(a, p.pairing, st);
}

}  // namespace vda
