// Host side of the C ABI declared in include/vda.h: argument checks,
// workspace carve-up and the launch sequence.  No compute happens here.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <type_traits>

#include "vda_internal.cuh"

namespace {

thread_local char g_msg[512] = "";

vda_status fail(vda_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
vda_status fail(vda_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

vda_status cuda_fail(cudaError_t e, const char* where) {
  return fail(VDA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

vda_status check_problem(const vda_problem* p) {
  if (!p) return fail(VDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->B < 1 || p->H < 1 || p->T < 1 || p->n < 1)
    return fail(VDA_ERR_INVALID_ARG, "B, H, T, n must be >= 1 (got %d, %d, %d, %d)", p->B, p->H,
                p->T, p->n);
  if (p->n_txt < 0) return fail(VDA_ERR_INVALID_ARG, "n_txt must be >= 0 (got %d)", p->n_txt);
  if (p->d_k < 1 || p->d_v < 1)
    return fail(VDA_ERR_INVALID_ARG, "d_k, d_v must be >= 1 (got %d, %d)", p->d_k, p->d_v);
  if (!(p->lambda > 0.f) || !isfinite(p->lambda))
    return fail(VDA_ERR_INVALID_ARG, "lambda must be finite and > 0 (got %g)", (double)p->lambda);
  if (p->dtype != VDA_DTYPE_F32 && p->dtype != VDA_DTYPE_BF16 && p->dtype != VDA_DTYPE_E4M3)
    return fail(VDA_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
  if (p->dtype == VDA_DTYPE_E4M3) {
    const float sc[4] = {p->scale_q, p->scale_k, p->scale_v, p->scale_g};
    for (float v : sc)
      if (!(v > 0.f) || !isfinite(v))
        return fail(VDA_ERR_INVALID_ARG, "e4m3 scales must be finite and > 0 (got %g, %g, %g, %g)",
                    (double)sc[0], (double)sc[1], (double)sc[2], (double)sc[3]);
  }
  if (p->layout != VDA_LAYOUT_BHTND && p->layout != VDA_LAYOUT_BTNHD)
    return fail(VDA_ERR_INVALID_ARG, "unknown layout %d", p->layout);
  if (p->test_stall < 0 || p->test_stall > VDA_TEST_STALL_MAX)
    return fail(VDA_ERR_INVALID_ARG, "unknown test_stall site %d", p->test_stall);
  if (p->layout == VDA_LAYOUT_BTNHD && p->dtype == VDA_DTYPE_F32)
    return fail(VDA_ERR_UNSUPPORTED, "the token-major layout is supported for bfloat16 and e4m3 inputs only");
  if (p->dtype == VDA_DTYPE_F32) {
    if (p->d_k % 16 || p->d_v % 16 || p->d_k > 128 || p->d_v > 128)
      return fail(VDA_ERR_UNSUPPORTED,
                  "float32 path supports d_k, d_v multiples of 16 up to 128 (got %d, %d)", p->d_k,
                  p->d_v);
  } else {
    if (p->d_k != 128 || p->d_v != 128)
      return fail(VDA_ERR_UNSUPPORTED, "%s path supports d_k = d_v = 128 (got %d, %d)",
                  p->dtype == VDA_DTYPE_E4M3 ? "e4m3" : "bfloat16", p->d_k, p->d_v);
  }
  // Index arithmetic in the kernels: slots and frames fit 32 bits, element
  // offsets are 64-bit.
  const long long slots = (long long)p->B * p->H * (p->T + 1);
  if (slots > 65535LL * 64)
    return fail(VDA_ERR_UNSUPPORTED, "B*H*(T+1) = %lld is above the supported 4194240", slots);
  if ((long long)p->B * p->H > 65535)
    return fail(VDA_ERR_UNSUPPORTED, "B*H = %lld is above 65535", (long long)p->B * p->H);
  if ((long long)p->B * p->H * p->T > 65535LL * 1024)
    return fail(VDA_ERR_UNSUPPORTED, "B*H*T is too large");
  if (p->n > (1 << 24) || p->n_txt > (1 << 24))
    return fail(VDA_ERR_UNSUPPORTED, "n and n_txt must be <= 2^24");
  return VDA_OK;
}

// Bytes of one input element, and of one element of O (bfloat16 for e4m3 inputs).
size_t elem_size(const vda_problem& p) {
  return p.dtype == VDA_DTYPE_E4M3 ? 1 : p.dtype == VDA_DTYPE_BF16 ? 2 : 4;
}
size_t out_elem_size(const vda_problem& p) { return p.dtype == VDA_DTYPE_F32 ? 4 : 2; }

struct Sizes {
  size_t q, k, v, g, kt, vt, o;
};

Sizes tensor_bytes(const vda_problem& p) {
  const size_t es = elem_size(p);
  const size_t fr = (size_t)p.B * p.H * p.T * p.n;
  const size_t tx = (size_t)p.B * p.H * p.n_txt;
  return Sizes{fr * p.d_k * es, fr * p.d_k * es, fr * p.d_v * es, fr * p.d_v * es,
               tx * p.d_k * es, tx * p.d_v * es, fr * p.d_v * out_elem_size(p)};
}

vda_status check_pointers(const vda_problem& p, const void* Q, const void* K, const void* V,
                          const void* G, const void* Kt, const void* Vt, const void* O) {
  const void* req[5] = {Q, K, V, G, O};
  const char* names[5] = {"Q", "K", "V", "G", "O"};
  for (int i = 0; i < 5; ++i) {
    if (!req[i]) return fail(VDA_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(req[i])) return fail(VDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if (p.n_txt > 0) {
    if (!Kt || !Vt) return fail(VDA_ERR_INVALID_ARG, "K_txt / V_txt NULL with n_txt = %d", p.n_txt);
    if (!aligned16(Kt) || !aligned16(Vt))
      return fail(VDA_ERR_INVALID_ARG, "K_txt / V_txt not 16-byte aligned");
  }
  return VDA_OK;
}

// The float32 path: SIMT Gram, the register-blocked factor, SIMT scan and
// readout; every state and product in float32.
vda_status run_forward_f32(const vda_problem& p, const float* q, const float* k, const float* v, const float* g,
                           const float* kt, const float* vt, float* O, char* ws, cudaStream_t st, float* S_fwd,
                           float* S_bwd, cudaEvent_t const* ev) {
  const vda::Layout L = vda::make_layout(p);
  unsigned* err = reinterpret_cast<unsigned*>(ws + L.err);
  float* M = reinterpret_cast<float*>(ws + L.M);
  float* C = reinterpret_cast<float*>(ws + L.C);
  // The states live in the workspace unless the caller wants them.
  float* SF = S_fwd ? S_fwd : reinterpret_cast<float*>(ws + L.SF);
  float* SB = S_bwd ? S_bwd : reinterpret_cast<float*>(ws + L.SB);
  cudaError_t e = cudaMemsetAsync(err, 0, 256, st);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the error word");
  auto mark = [&](int i) -> cudaError_t { return ev ? cudaEventRecord(ev[i], st) : cudaSuccess; };
  if ((e = mark(0)) != cudaSuccess) return cuda_fail(e, "event record");
  if ((e = vda::launch_gram_simt<float>(p, k, v, kt, vt, M, C, st)) != cudaSuccess) return cuda_fail(e, "gram launch");
  if ((e = mark(1)) != cudaSuccess) return cuda_fail(e, "event record");
  if ((e = vda::launch_factor(p, M, err, st)) != cudaSuccess) return cuda_fail(e, "factor launch");
  if ((e = mark(2)) != cudaSuccess) return cuda_fail(e, "event record");
  if ((e = vda::launch_scan_simt(p, M, C, SF, SB, st)) != cudaSuccess) return cuda_fail(e, "scan launch");
  if ((e = mark(3)) != cudaSuccess) return cuda_fail(e, "event record");
  if ((e = vda::launch_readout_simt<float>(p, q, g, SF, SB, O, st)) != cudaSuccess)
    return cuda_fail(e, "readout launch");
  if ((e = mark(4)) != cudaSuccess) return cuda_fail(e, "event record");
  return VDA_OK;
}

// The tensor-core path (bfloat16 or e4m3 inputs, d = 128): the fused
// Gram+factor kernel (A_t never leaves TMEM), the scan, the readout.  The
// workspace holds bf16 states for the readout; the caller's float32 state
// buffers, if any, are written besides.
vda_status run_forward_tc(const vda_problem& p, const void* q, const void* k, const void* v, const void* g,
                          const void* kt, const void* vt, void* O, char* ws, cudaStream_t st, float* S_fwd,
                          float* S_bwd, cudaEvent_t const* ev) {
  const vda::Layout L = vda::make_layout(p);
  unsigned* err = reinterpret_cast<unsigned*>(ws + L.err);
  float* M = reinterpret_cast<float*>(ws + L.M);
  float* C = reinterpret_cast<float*>(ws + L.C);
  __nv_bfloat16* SFb = reinterpret_cast<__nv_bfloat16*>(ws + L.SF);
  __nv_bfloat16* SBb = reinterpret_cast<__nv_bfloat16*>(ws + L.SB);
  cudaError_t e = cudaMemsetAsync(err, 0, 256, st);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the error word");
  auto mark = [&](int i) -> cudaError_t { return ev ? cudaEventRecord(ev[i], st) : cudaSuccess; };
  if ((e = mark(0)) != cudaSuccess) return cuda_fail(e, "event record");
  // Gram and factor in one kernel: the factor interval between events 1 and
  // 2 is empty on this path.
  if ((e = vda::launch_gramfactor_tc(p, k, v, kt, vt, M, C, err, st)) != cudaSuccess)
    return cuda_fail(e, "gram+factor launch");
  if ((e = mark(1)) != cudaSuccess) return cuda_fail(e, "event record");
  if ((e = mark(2)) != cudaSuccess) return cuda_fail(e, "event record");
  if ((e = vda::launch_scan_tc(p, M, C, SFb, SBb, S_fwd, S_bwd, err, st)) != cudaSuccess)
    return cuda_fail(e, "scan launch");
  if ((e = mark(3)) != cudaSuccess) return cuda_fail(e, "event record");
  if ((e = vda::launch_readout_tc(p, q, g, SFb, SBb, static_cast<__nv_bfloat16*>(O), err, st)) != cudaSuccess)
    return cuda_fail(e, "readout launch");
  if ((e = mark(4)) != cudaSuccess) return cuda_fail(e, "event record");
  return VDA_OK;
}

vda_status forward_impl(const vda_problem* p, const void* Q, const void* K, const void* V,
                        const void* G, const void* Kt, const void* Vt, void* O, void* workspace,
                        size_t workspace_bytes, void* stream, float* S_fwd, float* S_bwd,
                        cudaEvent_t const* ev = nullptr) {
  g_msg[0] = 0;
  vda_status s = check_problem(p);
  if (s != VDA_OK) return s;
  if ((s = check_pointers(*p, Q, K, V, G, Kt, Vt, O)) != VDA_OK) return s;
  const vda::Layout L = vda::make_layout(*p);
  if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)workspace & 255u) return fail(VDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < L.total)
    return fail(VDA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, L.total);
  if ((S_fwd && !aligned16(S_fwd)) || (S_bwd && !aligned16(S_bwd)))
    return fail(VDA_ERR_INVALID_ARG, "S_fwd / S_bwd not 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (p->dtype != VDA_DTYPE_F32) return run_forward_tc(*p, Q, K, V, G, Kt, Vt, O, ws, st, S_fwd, S_bwd, ev);
  auto f = [](const void* x) { return static_cast<const float*>(x); };
  return run_forward_f32(*p, f(Q), f(K), f(V), f(G), f(Kt), f(Vt), static_cast<float*>(O), ws, st, S_fwd, S_bwd, ev);
}

}  // namespace

namespace vda {
void set_error_message(const char* msg) { snprintf(g_msg, sizeof(g_msg), "%s", msg); }
}  // namespace vda

extern "C" {

vda_status vda_workspace_size(const vda_problem* p, size_t* bytes) {
  g_msg[0] = 0;
  vda_status s = check_problem(p);
  if (s != VDA_OK) return s;
  if (!bytes) return fail(VDA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = vda::make_layout(*p).total;
  return VDA_OK;
}

vda_status vda_forward(const vda_problem* p, const void* Q, const void* K, const void* V,
                       const void* G, const void* K_txt, const void* V_txt, void* O,
                       void* workspace, size_t workspace_bytes, void* stream) {
  return forward_impl(p, Q, K, V, G, K_txt, V_txt, O, workspace, workspace_bytes, stream, nullptr,
                      nullptr);
}

vda_status vda_forward_states(const vda_problem* p, const void* Q, const void* K, const void* V,
                              const void* G, const void* K_txt, const void* V_txt, void* O,
                              void* workspace, size_t workspace_bytes, void* stream,
                              float* S_fwd, float* S_bwd) {
  if (!S_fwd || !S_bwd) return fail(VDA_ERR_INVALID_ARG, "S_fwd / S_bwd is NULL");
  return forward_impl(p, Q, K, V, G, K_txt, V_txt, O, workspace, workspace_bytes, stream, S_fwd,
                      S_bwd);
}

vda_status vda_forward_timed(const vda_problem* p, const void* Q, const void* K, const void* V,
                             const void* G, const void* K_txt, const void* V_txt, void* O,
                             void* workspace, size_t workspace_bytes, void* stream,
                             void* const* events, int n_events) {
  if (!events || n_events != VDA_TIMED_EVENTS)
    return fail(VDA_ERR_INVALID_ARG, "events must hold %d cudaEvent_t handles", VDA_TIMED_EVENTS);
  for (int i = 0; i < n_events; ++i)
    if (!events[i]) return fail(VDA_ERR_INVALID_ARG, "events[%d] is NULL", i);
  return forward_impl(p, Q, K, V, G, K_txt, V_txt, O, workspace, workspace_bytes, stream, nullptr,
                      nullptr, reinterpret_cast<cudaEvent_t const*>(events));
}

vda_status vda_host_workspace_size(const vda_problem* p, size_t* bytes) {
  g_msg[0] = 0;
  vda_status s = check_problem(p);
  if (s != VDA_OK) return s;
  if (!bytes) return fail(VDA_ERR_INVALID_ARG, "bytes is NULL");
  const Sizes z = tensor_bytes(*p);
  size_t off = 0;
  const size_t parts[7] = {z.q, z.k, z.v, z.g, z.kt, z.vt, z.o};
  for (size_t b : parts) off = vda::align_up(off + b, 256);
  *bytes = off + vda::make_layout(*p).total;
  return VDA_OK;
}

vda_status vda_forward_host(const vda_problem* p, const void* Q, const void* K, const void* V,
                            const void* G, const void* K_txt, const void* V_txt, void* O,
                            void* workspace, size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  vda_status s = check_problem(p);
  if (s != VDA_OK) return s;
  if ((s = check_pointers(*p, Q, K, V, G, K_txt, V_txt, O)) != VDA_OK) return s;
  size_t need = 0;
  vda_host_workspace_size(p, &need);
  if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)workspace & 255u) return fail(VDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < need)
    return fail(VDA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  const Sizes z = tensor_bytes(*p);
  char* base = static_cast<char*>(workspace);
  const void* src[6] = {Q, K, V, G, K_txt, V_txt};
  const size_t len[6] = {z.q, z.k, z.v, z.g, z.kt, z.vt};
  void* dev[7];
  size_t off = 0;
  for (int i = 0; i < 6; ++i) {
    dev[i] = base + off;
    off = vda::align_up(off + len[i], 256);
  }
  dev[6] = base + off;
  off = vda::align_up(off + z.o, 256);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int i = 0; i < 6; ++i) {
    if (len[i] == 0) continue;
    cudaError_t e = cudaMemcpyAsync(dev[i], src[i], len[i], cudaMemcpyHostToDevice, st);
    if (e != cudaSuccess) return cuda_fail(e, "host-to-device copy");
  }
  s = forward_impl(p, dev[0], dev[1], dev[2], dev[3], p->n_txt ? dev[4] : nullptr,
                   p->n_txt ? dev[5] : nullptr, dev[6], base + off, workspace_bytes - off, stream,
                   nullptr, nullptr);
  if (s != VDA_OK) return s;
  cudaError_t e = cudaMemcpyAsync(O, dev[6], z.o, cudaMemcpyDeviceToHost, st);
  if (e != cudaSuccess) return cuda_fail(e, "device-to-host copy");
  return vda_sync_status(base + off, stream);
}

vda_status vda_backward_workspace_size(const vda_problem* p, size_t* bytes) {
  g_msg[0] = 0;
  vda_status s = check_problem(p);
  if (s != VDA_OK) return s;
  if (p->dtype != VDA_DTYPE_BF16)
    return fail(VDA_ERR_UNSUPPORTED, "the backward supports bfloat16 inputs only");
  if (!bytes) return fail(VDA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = vda::backward_workspace_bytes(*p);
  return VDA_OK;
}

namespace {

vda_status check_backward_pointers(const vda_problem& p, const void* Q, const void* K, const void* V, const void* G,
                                   const void* K_txt, const void* V_txt, const void* dO, const void* dQ,
                                   const void* dK, const void* dV, const void* dG, const void* dK_txt,
                                   const void* dV_txt) {
  vda_status s = check_pointers(p, Q, K, V, G, K_txt, V_txt, dO);
  if (s != VDA_OK) return s;
  const void* outs[4] = {dQ, dK, dV, dG};
  const char* names[4] = {"dQ", "dK", "dV", "dG"};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) return fail(VDA_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(outs[i])) return fail(VDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if (p.n_txt > 0 && (!dK_txt || !dV_txt || !aligned16(dK_txt) || !aligned16(dV_txt)))
    return fail(VDA_ERR_INVALID_ARG, "dK_txt / dV_txt NULL or not 16-byte aligned with n_txt = %d", p.n_txt);
  return VDA_OK;
}

vda_status backward_impl(const vda_problem* p, const void* Q, const void* K, const void* V, const void* G,
                         const void* K_txt, const void* V_txt, const void* dO, void* dQ, void* dK, void* dV,
                         void* dG, void* dK_txt, void* dV_txt, void* workspace, size_t workspace_bytes, void* stream,
                         bool from_forward) {
  size_t need = 0;
  vda_status s = vda_backward_workspace_size(p, &need);
  if (s != VDA_OK) return s;
  if ((s = check_backward_pointers(*p, Q, K, V, G, K_txt, V_txt, dO, dQ, dK, dV, dG, dK_txt, dV_txt)) != VDA_OK) return s;
  if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)workspace & 255u) return fail(VDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < need)
    return fail(VDA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  using bf = __nv_bfloat16;
  const char* where = "";
  cudaError_t e = vda::run_backward(*p, static_cast<const bf*>(Q), static_cast<const bf*>(K),
                                    static_cast<const bf*>(V), static_cast<const bf*>(G),
                                    static_cast<const bf*>(K_txt), static_cast<const bf*>(V_txt),
                                    static_cast<const bf*>(dO), static_cast<bf*>(dQ), static_cast<bf*>(dK),
                                    static_cast<bf*>(dV), static_cast<bf*>(dG), static_cast<bf*>(dK_txt),
                                    static_cast<bf*>(dV_txt), static_cast<char*>(workspace),
                                    static_cast<cudaStream_t>(stream), &where, from_forward);
  if (e != cudaSuccess) return cuda_fail(e, where);
  return VDA_OK;
}

}  // namespace

vda_status vda_backward(const vda_problem* p, const void* Q, const void* K, const void* V, const void* G,
                        const void* K_txt, const void* V_txt, const void* dO, void* dQ, void* dK, void* dV,
                        void* dG, void* dK_txt, void* dV_txt, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return backward_impl(p, Q, K, V, G, K_txt, V_txt, dO, dQ, dK, dV, dG, dK_txt, dV_txt, workspace, workspace_bytes,
                       stream, false);
}

vda_status vda_backward_from_forward(const vda_problem* p, const void* Q, const void* K, const void* V,
                                     const void* G, const void* K_txt, const void* V_txt, const void* dO, void* dQ,
                                     void* dK, void* dV, void* dG, void* dK_txt, void* dV_txt, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  return backward_impl(p, Q, K, V, G, K_txt, V_txt, dO, dQ, dK, dV, dG, dK_txt, dV_txt, workspace, workspace_bytes,
                       stream, true);
}

vda_status vda_local_softmax(const vda_problem* p, const void* Q, const void* K, const void* V, const void* G,
                             const void* K_txt, const void* V_txt, void* O, void* workspace, size_t workspace_bytes,
                             void* stream) {
  g_msg[0] = 0;
  if (!p) return fail(VDA_ERR_INVALID_ARG, "problem is NULL");
  vda_problem q = *p;
  q.lambda = 1.f;   // not read by this branch
  vda_status s = check_problem(&q);
  if (s != VDA_OK) return s;
  if (q.dtype != VDA_DTYPE_BF16)
    return fail(VDA_ERR_UNSUPPORTED, "the local softmax branch supports bfloat16 inputs only");
  if ((s = check_pointers(q, Q, K, V, G, K_txt, V_txt, O)) != VDA_OK) return s;
  if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)workspace & 255u) return fail(VDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < 256) return fail(VDA_ERR_WORKSPACE, "workspace has %zu bytes, needs 256", workspace_bytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(workspace, 0, 256, st);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the error word");
  using bf = __nv_bfloat16;
  e = vda::launch_local_softmax_tc(q, static_cast<const bf*>(Q), static_cast<const bf*>(K), static_cast<const bf*>(V),
                                   static_cast<const bf*>(G), static_cast<const bf*>(K_txt),
                                   static_cast<const bf*>(V_txt), static_cast<bf*>(O),
                                   static_cast<unsigned*>(workspace), st);
  if (e != cudaSuccess) return cuda_fail(e, "local softmax launch");
  return VDA_OK;
}

vda_status vda_merge_project(const vda_merge_problem* p, const void* O_lin, const void* W_lin, const void* O_sm,
                             const void* W_sm, void* Y, void* workspace, size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  if (!p) return fail(VDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->tokens < 1 || p->tokens > (1LL << 31) - 256)
    return fail(VDA_ERR_INVALID_ARG, "tokens must be in [1, 2^31 - 256] (got %lld)", (long long)p->tokens);
  if (p->K < 64 || p->K % 64) return fail(VDA_ERR_UNSUPPORTED, "K must be a positive multiple of 64 (got %d)", p->K);
  if (p->D < 8 || p->D % 8) return fail(VDA_ERR_UNSUPPORTED, "D must be a positive multiple of 8 (got %d)", p->D);
  if (p->test_stall < 0 || p->test_stall > VDA_TEST_STALL_MAX)
    return fail(VDA_ERR_INVALID_ARG, "unknown test_stall site %d", p->test_stall);
  if (p->reserved != 0) return fail(VDA_ERR_INVALID_ARG, "reserved must be 0 (got %d)", p->reserved);
  const void* req[3] = {O_lin, W_lin, Y};
  const char* names[3] = {"O_lin", "W_lin", "Y"};
  for (int i = 0; i < 3; ++i) {
    if (!req[i]) return fail(VDA_ERR_INVALID_ARG, "%s is NULL", names[i]);
    if (!aligned16(req[i])) return fail(VDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  if ((O_sm == nullptr) != (W_sm == nullptr))
    return fail(VDA_ERR_INVALID_ARG, "O_sm and W_sm must both be given or both be NULL");
  if (O_sm && (!aligned16(O_sm) || !aligned16(W_sm)))
    return fail(VDA_ERR_INVALID_ARG, "O_sm / W_sm not 16-byte aligned");
  if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)workspace & 255u) return fail(VDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < 256) return fail(VDA_ERR_WORKSPACE, "workspace has %zu bytes, needs 256", workspace_bytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(workspace, 0, 256, st);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the error word");
  using bf = __nv_bfloat16;
  e = vda::launch_merge_tc(p->tokens, p->K, p->D, static_cast<const bf*>(O_lin), static_cast<const bf*>(W_lin),
                           static_cast<const bf*>(O_sm), static_cast<const bf*>(W_sm), static_cast<bf*>(Y),
                           static_cast<unsigned*>(workspace), st, p->test_stall);
  if (e != cudaSuccess) return cuda_fail(e, "merge launch");
  return VDA_OK;
}

// ------------------------------------------------------------------ token operators
namespace {

bool float_type(int dt) { return dt == VDA_DTYPE_F32 || dt == VDA_DTYPE_BF16; }
bool aligned_elem(const void* x, int dt) { return ((uintptr_t)x & (dt == VDA_DTYPE_BF16 ? 1u : 3u)) == 0; }
constexpr int64_t kMaxStride = (1LL << 31) - 1;

// A tensor that the call reads or writes: not NULL, aligned to its elements.
vda_status check_tensor(const void* x, int dt, const char* name) {
  if (!x) return fail(VDA_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned_elem(x, dt)) return fail(VDA_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  return VDA_OK;
}
vda_status check_optional(const void* x, int dt, const char* name) {
  return x ? check_tensor(x, dt, name) : VDA_OK;
}
vda_status check_stride(int64_t ld, int64_t least, const char* name) {
  if (ld != 0 && (ld < least || ld > kMaxStride))
    return fail(VDA_ERR_INVALID_ARG, "%s must be 0 or in [%lld, 2^31) (got %lld)", name, (long long)least, (long long)ld);
  return VDA_OK;
}

#define VDA_CHECK(expr)                  \
  do {                                   \
    const vda_status s_ = (expr);        \
    if (s_ != VDA_OK) return s_;         \
  } while (0)

vda_status check_norm(const vda_norm_problem* p) {
  if (!p) return fail(VDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->tokens < 0 || p->tokens > kMaxStride)
    return fail(VDA_ERR_INVALID_ARG, "tokens must be in [0, 2^31) (got %lld)", (long long)p->tokens);
  if (p->heads < 1 || p->D < 1)
    return fail(VDA_ERR_INVALID_ARG, "heads and D must be >= 1 (got %d, %d)", p->heads, p->D);
  if (p->heads > 65536 || p->D > 8192)
    return fail(VDA_ERR_UNSUPPORTED, "heads up to 65536 and D up to 8192 are supported (got %d, %d)", p->heads, p->D);
  if (!float_type(p->dtype) || !float_type(p->w_dtype))
    return fail(VDA_ERR_INVALID_ARG, "dtype and w_dtype must be float32 or bfloat16 (got %d, %d)", p->dtype, p->w_dtype);
  if (!(p->eps > 0.f) || !isfinite(p->eps))
    return fail(VDA_ERR_INVALID_ARG, "eps must be finite and > 0 (got %g)", (double)p->eps);
  if (p->reserved != 0) return fail(VDA_ERR_INVALID_ARG, "reserved must be 0 (got %d)", p->reserved);
  VDA_CHECK(check_stride(p->ld_x, (int64_t)p->heads * p->D, "ld_x"));
  return check_stride(p->ld_y, (int64_t)p->heads * p->D, "ld_y");
}

vda_status norm_backward_impl(const vda_norm_problem* p, const void* dY, const void* X, const float* mean,
                              const float* rstd, const void* codes, const void* scales, const void* W, void* dX,
                              float* dW, float* dbias, void* workspace, size_t workspace_bytes, void* stream,
                              bool from_checkpoint) {
  g_msg[0] = 0;
  VDA_CHECK(check_norm(p));
  VDA_CHECK(check_optional(W, p->w_dtype, "W"));
  VDA_CHECK(check_optional(dW, VDA_DTYPE_F32, "dW"));
  VDA_CHECK(check_optional(dbias, VDA_DTYPE_F32, "dbias"));
  if (p->tokens > 0) {
    VDA_CHECK(check_tensor(dY, p->dtype, "dY"));
    VDA_CHECK(check_tensor(dX, p->dtype, "dX"));
    VDA_CHECK(check_tensor(rstd, VDA_DTYPE_F32, "rstd"));
    if (from_checkpoint) {
      if (!codes || !scales) return fail(VDA_ERR_INVALID_ARG, "codes / scales is NULL");
    } else {
      VDA_CHECK(check_tensor(X, p->dtype, "X"));
      VDA_CHECK(check_tensor(mean, VDA_DTYPE_F32, "mean"));
    }
    if (dW || dbias) {
      const size_t need = vda::norm_backward_workspace_bytes(*p);
      if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
      if ((uintptr_t)workspace & 255u) return fail(VDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
      if (workspace_bytes < need)
        return fail(VDA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    }
  }
  float* partial = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e =
      from_checkpoint
          ? vda::launch_layer_norm_backward_from_checkpoint(*p, dY, static_cast<const uint8_t*>(codes),
                                                            static_cast<const uint8_t*>(scales), rstd, W, dX, dW,
                                                            dbias, partial, st)
          : vda::launch_layer_norm_backward(*p, dY, X, mean, rstd, W, dX, dW, dbias, partial, st);
  if (e != cudaSuccess) return cuda_fail(e, "layer norm backward launch");
  return VDA_OK;
}

vda_status check_rope(const vda_rope_problem* p) {
  if (!p) return fail(VDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->B < 0 || p->T < 0 || p->height < 0 || p->width < 0)
    return fail(VDA_ERR_INVALID_ARG, "B, T, height, width must be >= 0 (got %d, %d, %d, %d)", p->B, p->T, p->height,
                p->width);
  if (p->H_q < 0 || p->H_k < 0 || (int64_t)p->H_q + p->H_k > 65535)
    return fail(VDA_ERR_INVALID_ARG, "H_q, H_k must be >= 0 and H_q + H_k <= 65535 (got %d, %d)", p->H_q, p->H_k);
  if (p->d < 1) return fail(VDA_ERR_INVALID_ARG, "d must be >= 1 (got %d)", p->d);
  if (p->d > 256) return fail(VDA_ERR_UNSUPPORTED, "d up to 256 is supported (got %d)", p->d);
  if (p->d_t < 0 || p->d_y < 0 || p->d_x < 0 || (p->d_t | p->d_y | p->d_x) & 1 ||
      (int64_t)p->d_t + p->d_y + p->d_x > p->d)
    return fail(VDA_ERR_INVALID_ARG, "d_t, d_y, d_x must be even, >= 0 and at most d = %d together (got %d, %d, %d)",
                p->d, p->d_t, p->d_y, p->d_x);
  if (!float_type(p->dtype)) return fail(VDA_ERR_INVALID_ARG, "dtype must be float32 or bfloat16 (got %d)", p->dtype);
  if (p->layout != VDA_LAYOUT_BHTND && p->layout != VDA_LAYOUT_BTNHD)
    return fail(VDA_ERR_INVALID_ARG, "unknown layout %d", p->layout);
  if (p->pairing != VDA_ROPE_INTERLEAVED && p->pairing != VDA_ROPE_HALVES)
    return fail(VDA_ERR_INVALID_ARG, "unknown pairing %d", p->pairing);
  if (!(p->theta > 0.0) || !isfinite(p->theta))
    return fail(VDA_ERR_INVALID_ARG, "theta must be finite and > 0 (got %g)", p->theta);
  for (int i = 0; i < 3; ++i)
    if (!isfinite(p->pos0[i]) || !isfinite(p->step[i]))
      return fail(VDA_ERR_INVALID_ARG, "pos0 and step must be finite (axis %d: %g, %g)", i, p->pos0[i], p->step[i]);
  if (p->reserved != 0) return fail(VDA_ERR_INVALID_ARG, "reserved must be 0 (got %d)", p->reserved);
  // B * T * height * width below 2^31, without overflowing on the way.
  int64_t tokens = p->B;
  for (int f : {p->T, p->height, p->width}) {
    if (f == 0) tokens = 0;
    if (tokens > kMaxStride) break;
    tokens *= f;
  }
  if (tokens > kMaxStride && p->T && p->height && p->width)
    return fail(VDA_ERR_UNSUPPORTED, "B * T * height * width must be below 2^31");
  const int64_t ld[4] = {p->ld_q, p->ld_k, p->ld_qr, p->ld_kr};
  const char* names[4] = {"ld_q", "ld_k", "ld_qr", "ld_kr"};
  for (int i = 0; i < 4; ++i) {
    if (p->layout == VDA_LAYOUT_BHTND && ld[i] != 0)
      return fail(VDA_ERR_INVALID_ARG, "%s must be 0 in the [B, H, N, d] layout (got %lld)", names[i], (long long)ld[i]);
    VDA_CHECK(check_stride(ld[i], (int64_t)(i % 2 ? p->H_k : p->H_q) * p->d, names[i]));
  }
  return VDA_OK;
}

vda_status rope_impl(const vda_rope_problem* p, const void* Q, const void* K, const float* positions, void* Qo,
                     void* Ko, void* stream, bool backward) {
  g_msg[0] = 0;
  VDA_CHECK(check_rope(p));
  VDA_CHECK(check_optional(positions, VDA_DTYPE_F32, "positions"));
  if (p->B && p->T && p->height && p->width) {
    if (p->H_q) {
      VDA_CHECK(check_tensor(Q, p->dtype, backward ? "dQ_rot" : "Q"));
      VDA_CHECK(check_tensor(Qo, p->dtype, backward ? "dQ" : "Q_rot"));
    }
    if (p->H_k) {
      VDA_CHECK(check_tensor(K, p->dtype, backward ? "dK_rot" : "K"));
      VDA_CHECK(check_tensor(Ko, p->dtype, backward ? "dK" : "K_rot"));
    }
  }
  cudaError_t e = vda::launch_rope(*p, Q, K, positions, Qo, Ko, backward, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, backward ? "rope backward launch" : "rope launch");
  return VDA_OK;
}

vda_status check_checkpoint(const vda_checkpoint_problem* p, const void* X, const void* codes, const void* scales) {
  if (!p) return fail(VDA_ERR_INVALID_ARG, "problem is NULL");
  if (p->rows < 0 || p->rows > (1LL << 40))
    return fail(VDA_ERR_INVALID_ARG, "rows must be in [0, 2^40] (got %lld)", (long long)p->rows);
  if (p->D < 1) return fail(VDA_ERR_INVALID_ARG, "D must be >= 1 (got %d)", p->D);
  if (p->D > (1 << 24)) return fail(VDA_ERR_UNSUPPORTED, "D up to 2^24 is supported (got %d)", p->D);
  if (p->rows > ((1LL << 36) - 1) / ((p->D + 31) / 32))
    return fail(VDA_ERR_UNSUPPORTED, "rows * ceil(D / 32) must be below 2^36");
  if (!float_type(p->dtype)) return fail(VDA_ERR_INVALID_ARG, "dtype must be float32 or bfloat16 (got %d)", p->dtype);
  VDA_CHECK(check_stride(p->ld, p->D, "ld"));
  if (p->rows > 0) {
    VDA_CHECK(check_tensor(X, p->dtype, "X"));
    if (!codes || !scales) return fail(VDA_ERR_INVALID_ARG, "codes / scales is NULL");
  }
  return VDA_OK;
}

// Device copies of the backward's inputs behind its own workspace.
size_t checkpoint_backward_bytes(const vda_problem& p, size_t (&off)[6]) {
  const Sizes z = tensor_bytes(p);
  const size_t parts[6] = {z.q, z.k, z.v, z.g, z.kt, z.vt};
  size_t at = vda::backward_workspace_bytes(p);
  for (int i = 0; i < 6; ++i) {
    off[i] = at;
    at = vda::align_up(at + parts[i], 256);
  }
  return at;
}

}  // namespace

vda_status vda_layer_norm(const vda_norm_problem* p, const void* X, const void* W, const void* bias, void* Y,
                          float* mean, float* rstd, void* codes, void* scales, void* stream) {
  g_msg[0] = 0;
  VDA_CHECK(check_norm(p));
  VDA_CHECK(check_optional(W, p->w_dtype, "W"));
  VDA_CHECK(check_optional(bias, p->w_dtype, "bias"));
  VDA_CHECK(check_optional(mean, VDA_DTYPE_F32, "mean"));
  VDA_CHECK(check_optional(rstd, VDA_DTYPE_F32, "rstd"));
  if ((codes == nullptr) != (scales == nullptr))
    return fail(VDA_ERR_INVALID_ARG, "codes and scales must both be given or both be NULL");
  if (p->tokens > 0) {
    VDA_CHECK(check_tensor(X, p->dtype, "X"));
    VDA_CHECK(check_tensor(Y, p->dtype, "Y"));
  }
  cudaError_t e = vda::launch_layer_norm(*p, X, W, bias, Y, mean, rstd, static_cast<uint8_t*>(codes),
                                         static_cast<uint8_t*>(scales), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "layer norm launch");
  return VDA_OK;
}

vda_status vda_layer_norm_from_checkpoint(const vda_norm_problem* p, const void* codes, const void* scales,
                                          const void* W, const void* bias, void* Y, void* stream) {
  g_msg[0] = 0;
  VDA_CHECK(check_norm(p));
  VDA_CHECK(check_optional(W, p->w_dtype, "W"));
  VDA_CHECK(check_optional(bias, p->w_dtype, "bias"));
  if (p->tokens > 0) {
    if (!codes || !scales) return fail(VDA_ERR_INVALID_ARG, "codes / scales is NULL");
    VDA_CHECK(check_tensor(Y, p->dtype, "Y"));
  }
  cudaError_t e = vda::launch_layer_norm_from_checkpoint(*p, static_cast<const uint8_t*>(codes),
                                                         static_cast<const uint8_t*>(scales), W, bias, Y,
                                                         static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "layer norm from checkpoint launch");
  return VDA_OK;
}

vda_status vda_layer_norm_backward_workspace_size(const vda_norm_problem* p, size_t* bytes) {
  g_msg[0] = 0;
  VDA_CHECK(check_norm(p));
  if (!bytes) return fail(VDA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = vda::norm_backward_workspace_bytes(*p);
  return VDA_OK;
}

vda_status vda_layer_norm_backward(const vda_norm_problem* p, const void* dY, const void* X, const float* mean,
                                   const float* rstd, const void* W, void* dX, float* dW, float* dbias,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return norm_backward_impl(p, dY, X, mean, rstd, nullptr, nullptr, W, dX, dW, dbias, workspace, workspace_bytes,
                            stream, false);
}

vda_status vda_layer_norm_backward_from_checkpoint(const vda_norm_problem* p, const void* dY, const void* codes,
                                                   const void* scales, const float* rstd, const void* W, void* dX,
                                                   float* dW, float* dbias, void* workspace, size_t workspace_bytes,
                                                   void* stream) {
  return norm_backward_impl(p, dY, nullptr, nullptr, rstd, codes, scales, W, dX, dW, dbias, workspace,
                            workspace_bytes, stream, true);
}

vda_status vda_rope(const vda_rope_problem* p, const void* Q, const void* K, const float* positions, void* Q_rot,
                    void* K_rot, void* stream) {
  return rope_impl(p, Q, K, positions, Q_rot, K_rot, stream, false);
}

vda_status vda_rope_backward(const vda_rope_problem* p, const void* dQ_rot, const void* dK_rot,
                             const float* positions, void* dQ, void* dK, void* stream) {
  return rope_impl(p, dQ_rot, dK_rot, positions, dQ, dK, stream, true);
}

vda_status vda_checkpoint_pack(const vda_checkpoint_problem* p, const void* X, void* codes, void* scales,
                               void* stream) {
  g_msg[0] = 0;
  VDA_CHECK(check_checkpoint(p, X, codes, scales));
  cudaError_t e = vda::launch_checkpoint_pack(*p, X, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                              static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "checkpoint pack launch");
  return VDA_OK;
}

vda_status vda_checkpoint_unpack(const vda_checkpoint_problem* p, const void* codes, const void* scales, void* X,
                                 void* stream) {
  g_msg[0] = 0;
  VDA_CHECK(check_checkpoint(p, X, codes, scales));
  cudaError_t e = vda::launch_checkpoint_unpack(*p, static_cast<const uint8_t*>(codes),
                                                static_cast<const uint8_t*>(scales), X,
                                                static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "checkpoint unpack launch");
  return VDA_OK;
}

vda_status vda_backward_from_checkpoint_workspace_size(const vda_problem* p, size_t* bytes) {
  size_t need = 0, off[6];
  VDA_CHECK(vda_backward_workspace_size(p, &need));
  if (!bytes) return fail(VDA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = checkpoint_backward_bytes(*p, off);
  return VDA_OK;
}

vda_status vda_backward_from_checkpoint(const vda_problem* p, const vda_checkpoint* in, const void* dO, void* dQ,
                                        void* dK, void* dV, void* dG, void* dK_txt, void* dV_txt, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  size_t need = 0, off[6];
  VDA_CHECK(vda_backward_workspace_size(p, &need));
  if (!in) return fail(VDA_ERR_INVALID_ARG, "in is NULL");
  const int count = p->n_txt > 0 ? 6 : 4;
  static const char* const names[6] = {"Q", "K", "V", "G", "K_txt", "V_txt"};
  for (int i = 0; i < count; ++i)
    if (!in[i].codes || !in[i].scales) return fail(VDA_ERR_INVALID_ARG, "%s's codes / scales is NULL", names[i]);
  const size_t total = checkpoint_backward_bytes(*p, off);
  if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)workspace & 255u) return fail(VDA_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (workspace_bytes < total)
    return fail(VDA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, total);
  // The remaining pointers are checked before anything is enqueued, too.
  char* ws = static_cast<char*>(workspace);
  void* x[6];
  for (int i = 0; i < 6; ++i) x[i] = i < count ? ws + off[i] : nullptr;
  VDA_CHECK(check_backward_pointers(*p, x[0], x[1], x[2], x[3], x[4], x[5], dO, dQ, dK, dV, dG, dK_txt, dV_txt));
  const int64_t tokens = (int64_t)p->B * p->H * p->T * p->n, text = (int64_t)p->B * p->H * p->n_txt;
  for (int i = 0; i < count; ++i) {
    const vda_checkpoint_problem q = {i < 4 ? tokens : text, 0, 128, VDA_DTYPE_BF16};
    cudaError_t e = vda::launch_checkpoint_unpack(q, static_cast<const uint8_t*>(in[i].codes),
                                                  static_cast<const uint8_t*>(in[i].scales), x[i],
                                                  static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "checkpoint unpack launch");
  }
  return backward_impl(p, x[0], x[1], x[2], x[3], x[4], x[5], dO, dQ, dK, dV, dG, dK_txt, dV_txt, workspace,
                       need, stream, false);
}

vda_status vda_sync_status(void* workspace, void* stream) {
  g_msg[0] = 0;
  if (!workspace) return fail(VDA_ERR_WORKSPACE, "workspace is NULL");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  unsigned word = 0;
  e = cudaMemcpy(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "reading the error word");
  if (word) {
    e = cudaMemset(workspace, 0, sizeof(word));
    if (e != cudaSuccess) return cuda_fail(e, "clearing the error word");
  }
  if (word & vda::kDevErrNotSpd) return fail(VDA_ERR_NOT_SPD, "a Cholesky pivot was not positive");
  if (word & vda::kDevErrTimeout) return fail(VDA_ERR_TIMEOUT, "a bounded device wait gave up");
  return VDA_OK;
}

const char* vda_status_string(vda_status s) {
  switch (s) {
    case VDA_OK: return "VDA_OK";
    case VDA_ERR_INVALID_ARG: return "VDA_ERR_INVALID_ARG";
    case VDA_ERR_UNSUPPORTED: return "VDA_ERR_UNSUPPORTED";
    case VDA_ERR_WORKSPACE: return "VDA_ERR_WORKSPACE";
    case VDA_ERR_CUDA: return "VDA_ERR_CUDA";
    case VDA_ERR_NOT_SPD: return "VDA_ERR_NOT_SPD";
    case VDA_ERR_TIMEOUT: return "VDA_ERR_TIMEOUT";
  }
  return "VDA_ERR_UNKNOWN";
}

const char* vda_last_error(void) { return g_msg; }

}  // extern "C"
