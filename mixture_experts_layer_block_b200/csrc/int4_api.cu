// int4_api.cu -- the C entry points of 4-bit weights (moe_*_int4): argument checks and launches.
#include <algorithm>
#include <cmath>

#include "handle.h"
#include "matvec.cuh"

using namespace moe;

namespace moe {
// api.cu: the forward's router projection and gating into the handle's workspace
int run_router_and_gate(moe_handle* h, const void* x, int32_t T, const void* w_router, const float* router_bias,
                        int32_t top_k, cudaStream_t st);
int forward_capacity(const moe_handle* h, int T, int k);
}  // namespace moe

namespace {

int check_format(int64_t rows, int64_t cols, int32_t group) {
  if (rows < 1 || cols < 8 || cols % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  // row tiles, column indices and the blocks of a CTA's share stay within 28 bits
  if (cols > (1 << 24) || rows > ((int64_t)1 << 42) / cols) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool has(const moe_int4_mat& m) { return m.codes && m.scales; }
bool aligned(const moe_int4_mat& m) { return aligned16(m.codes) && aligned16(m.scales); }

int cuda_rc(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();  // a refused launch is reported here, not by a later call
  return check_cuda(e);
}

// The experts' arguments, checked without a CUDA call.
int check_experts(const moe_handle* h, int32_t T, int32_t top_k, const moe_int4_experts* w) {
  const moe_config& c = h->cfg;
  if (T < 0 || T > c.max_tokens || top_k < 1 || top_k > c.top_k) return MOE_ERR_INVALID_ARG;
  if (!w || !has(w->up) || !has(w->gate) || !has(w->down)) return MOE_ERR_INVALID_ARG;
  if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_ERR_INVALID_ARG;
  const bool shared = c.inter_shared > 0;
  if (shared && (!has(w->shared_up) || !has(w->shared_gate) || !has(w->shared_down))) return MOE_ERR_INVALID_ARG;
  // an expert's rows are whole 16-row tiles of the stacked matrices
  if (T > kMvTokens || c.hidden % kMvRows != 0 || c.inter % kMvRows != 0) return MOE_ERR_UNSUPPORTED;
  if (!aligned(w->up) || !aligned(w->gate) || !aligned(w->down)) return MOE_ERR_MISALIGNED;
  if (shared && (!aligned(w->shared_up) || !aligned(w->shared_gate) || !aligned(w->shared_down)))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

// Whether a call's result overlaps its experts' matrices: the down projection's CTAs store while others still
// copy weights.
bool overlaps_experts(const moe_config& c, const Span& out, const moe_int4_experts& w) {
  auto in = [&](const moe_int4_mat& m, int64_t rows, int64_t cols) {
    return overlap(out, {m.codes, int4_code_bytes(rows, cols)}) ||
           overlap(out, {m.scales, int4_scale_bytes(rows, cols, w.group, w.zeros != 0)});
  };
  const int64_t E = c.num_experts, H = c.hidden, D = c.inter, Ds = c.inter_shared;
  if (in(w.up, E * D, H) || in(w.gate, E * D, H) || in(w.down, E * H, D)) return true;
  return Ds > 0 && (in(w.shared_up, Ds, H) || in(w.shared_gate, Ds, H) || in(w.shared_down, H, Ds));
}

// Up projections with SwiGLU into the workspace's h, then the down projections' weighted sum.
int run_experts(moe_handle* h, const void* x, int32_t T, const int32_t* ids, const float* topk_w, int32_t k,
                const moe_int4_experts* w, int capacity, void* out, bool out_bf16, cudaStream_t st) {
  const moe_config& c = h->cfg;
  MvArgs a{};
  a.m = MvMatrix{{w->up.codes, w->gate.codes}, {w->up.scales, w->gate.scales}, c.inter, c.hidden};
  if (c.inter_shared > 0)
    a.shared = MvMatrix{{w->shared_up.codes, w->shared_gate.codes}, {w->shared_up.scales, w->shared_gate.scales},
                        c.inter_shared, c.hidden};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = c.hidden;
  a.T = T;
  a.group = w->group;
  a.ids = ids;
  a.topk_w = topk_w;
  a.E = c.num_experts;
  a.k = k;
  a.capacity = capacity;
  a.out = h->ws.h;
  a.ldo = h->ws.ldh;
  a.out_bf16 = 1;
  int rc;
  if ((rc = cuda_rc(launch_mv_int4(a, kMvUp, w->zeros != 0, h->num_sms, st)))) return rc;
  a.m = MvMatrix{{w->down.codes, nullptr}, {w->down.scales, nullptr}, c.hidden, c.inter};
  a.shared = MvMatrix{};
  if (c.inter_shared > 0)
    a.shared = MvMatrix{{w->shared_down.codes, nullptr}, {w->shared_down.scales, nullptr}, c.hidden, c.inter_shared};
  a.x = h->ws.h;
  a.ldx = h->ws.ldh;
  a.early = 1;
  a.out = out;
  a.ldo = c.hidden;
  a.out_bf16 = out_bf16;
  return cuda_rc(launch_mv_int4(a, kMvDown, w->zeros != 0, h->num_sms, st));
}

}  // namespace

extern "C" {

int64_t moe_int4_code_bytes(int64_t rows, int64_t cols) {
  return check_format(rows, cols, 32) == MOE_OK ? int4_code_bytes(rows, cols) : -1;
}

int64_t moe_int4_scale_bytes(int64_t rows, int64_t cols, int32_t group, int32_t zeros) {
  return check_format(rows, cols, group) == MOE_OK ? int4_scale_bytes(rows, cols, group, zeros != 0) : -1;
}

int moe_quantize_int4(moe_handle* h, const void* src, int64_t rows, int64_t cols, int32_t group, int32_t zeros,
                      void* codes, void* scales, void* stream) {
  int rc;
  if ((rc = check_format(rows, cols, group))) return rc;
  if (!src || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned16(src) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_MISALIGNED;
  if (clobbers({{codes, int4_code_bytes(rows, cols)}, {scales, int4_scale_bytes(rows, cols, group, zeros != 0)}},
               {{src, rows * cols * 2}}))
    return MOE_ERR_INVALID_ARG;
  if (!h) return MOE_ERR_INVALID_ARG;
  DeviceScope dev(h->device);
  if ((rc = dev.rc())) return rc;
  return cuda_rc(launch_int4_quantize(static_cast<const uint16_t*>(src), rows, cols, group, zeros != 0, codes, scales,
                                      h->num_sms, static_cast<cudaStream_t>(stream)));
}

int moe_pack_int4(moe_handle* h, const uint8_t* q, const void* s, const uint8_t* z, int64_t rows, int64_t cols,
                  int32_t group, void* codes, void* scales, void* stream) {
  int rc;
  if ((rc = check_format(rows, cols, group))) return rc;
  if (!q || !s || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(s) || !aligned16(z) || !aligned16(codes) || !aligned16(scales))
    return MOE_ERR_MISALIGNED;
  const int64_t entries = rows * ((cols + group - 1) / group);
  if (clobbers({{codes, int4_code_bytes(rows, cols)}, {scales, int4_scale_bytes(rows, cols, group, z != nullptr)}},
               {{q, rows * cols / 2}, {s, entries * 2}, {z, entries}}))
    return MOE_ERR_INVALID_ARG;
  if (!h) return MOE_ERR_INVALID_ARG;
  DeviceScope dev(h->device);
  if ((rc = dev.rc())) return rc;
  return cuda_rc(launch_int4_pack(q, static_cast<const uint16_t*>(s), z, rows, cols, group, codes, scales, h->num_sms,
                                  static_cast<cudaStream_t>(stream)));
}

int moe_matvec_int4(moe_handle* h, const void* x, int64_t T, const moe_int4_mat* w, int64_t rows, int64_t cols,
                    int32_t group, int32_t zeros, void* out, int32_t out_bf16, void* stream) {
  int rc;
  if ((rc = check_format(rows, cols, group))) return rc;
  if (T < 0 || !w || !has(*w)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !out)) return MOE_ERR_INVALID_ARG;
  // the kernel rounds rows up to whole tiles in 32 bits
  if (rows > INT32_MAX - (kMvRows - 1) || T > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned(*w) || (reinterpret_cast<uintptr_t>(out) & (out_bf16 ? 1u : 3u)) != 0)
    return MOE_ERR_MISALIGNED;
  if (clobbers({{out, T * rows * (out_bf16 ? 2 : 4)}},
               {{x, T * cols * 2},
                {w->codes, int4_code_bytes(rows, cols)},
                {w->scales, int4_scale_bytes(rows, cols, group, zeros != 0)}}))
    return MOE_ERR_INVALID_ARG;
  if (!h) return MOE_ERR_INVALID_ARG;
  DeviceScope dev(h->device);
  if ((rc = dev.rc())) return rc;
  MvArgs a{};
  a.m = MvMatrix{{w->codes, nullptr}, {w->scales, nullptr}, (int32_t)rows, (int32_t)cols};
  a.ldx = cols;
  a.group = group;
  a.ldo = rows;
  a.out_bf16 = out_bf16 != 0;
  for (int64_t t = 0; t < T; t += kMvTokens) {  // 16 tokens a launch, each reading the weights
    a.x = static_cast<const uint16_t*>(x) + t * cols;
    a.T = (int32_t)std::min<int64_t>(kMvTokens, T - t);
    a.out = static_cast<char*>(out) + t * rows * (out_bf16 ? 2 : 4);
    if ((rc = cuda_rc(launch_mv_int4(a, kMvOne, zeros != 0, h->num_sms, static_cast<cudaStream_t>(stream))))) return rc;
  }
  return MOE_OK;
}

int moe_experts_int4(moe_handle* h, const void* x, int32_t T, const int32_t* topk_ids, const float* topk_w,
                     int32_t top_k, const moe_int4_experts* w, void* out, int32_t out_bf16, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  int rc;
  if ((rc = check_experts(h, T, top_k, w))) return rc;
  if (T > 0 && (!x || !topk_ids || !topk_w || !out)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(topk_ids) || !aligned16(topk_w) || !aligned16(out)) return MOE_ERR_MISALIGNED;
  const int64_t n = (int64_t)T * h->cfg.hidden, slots = (int64_t)T * top_k;
  const Span result{out, n * (out_bf16 ? 2 : 4)};
  if (clobbers({result}, {{x, n * 2}, {topk_ids, slots * 4}, {topk_w, slots * 4}}) || overlaps_experts(h->cfg, result, *w))
    return MOE_ERR_INVALID_ARG;
  DeviceScope dev(h->device);
  if ((rc = dev.rc())) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  h->last_stream = st;
  h->have_forward = false;  // h goes where the layer's intermediates were
  if (T == 0) return MOE_OK;
  return run_experts(h, x, T, topk_ids, topk_w, top_k, w, 0, out, out_bf16 != 0, st);
}

int moe_forward_int4(moe_handle* h, const void* x, int32_t T, const void* w_router, const float* router_bias,
                     const moe_int4_experts* w, int32_t top_k, void* out, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  int rc;
  if ((rc = check_experts(h, T, top_k, w))) return rc;
  if (!w_router || (T > 0 && (!x || !out))) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(out) || !aligned16(router_bias)) return MOE_ERR_MISALIGNED;
  const int64_t n = (int64_t)T * h->cfg.hidden;
  const Span result{out, n * ((h->cfg.flags & MOE_FLAG_OUT_BF16) ? 2 : 4)};
  const int64_t E = h->cfg.num_experts;
  if (clobbers({result}, {{x, n * 2}, {w_router, E * h->cfg.hidden * 2}, {router_bias, E * 4}}) ||
      overlaps_experts(h->cfg, result, *w))
    return MOE_ERR_INVALID_ARG;
  DeviceScope dev(h->device);
  if ((rc = dev.rc())) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  h->last_stream = st;
  h->have_forward = false;
  if (T == 0) return MOE_OK;
  if ((rc = run_router_and_gate(h, x, T, w_router, router_bias, top_k, st))) return rc;
  return run_experts(h, x, T, h->ws.topk_ids, h->ws.topk_w, top_k, w, forward_capacity(h, T, top_k), out,
                     (h->cfg.flags & MOE_FLAG_OUT_BF16) != 0, st);
}

}  // extern "C"
