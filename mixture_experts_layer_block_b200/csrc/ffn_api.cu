// ffn_api.cu -- the C entry points of the gated feed-forward block (moe_ffn_*): argument checks,
// the plan of each launch (tile width, K splits, workspace) and the launches.
#include <algorithm>

#include "ffn.cuh"
#include "handle.h"
#include "matvec.cuh"

using namespace moe;

namespace {

// The plan is made for a full B200 (148 SMs), so that the workspace's size needs no handle; a
// device with fewer free pairs runs the same units over more rounds.
constexpr int kPlanPairs = 74;

struct Product {
  int64_t M, N;  // of the output (dual: of one of the two halves)
  int nkb;       // 64-wide K blocks in all
  bool dual;     // u and g side by side
  bool b_mn;     // B has n contiguous
  bool a_mn;     // A has m contiguous
  // the plan
  int bn, mrows, mt, nt, splits;
  int64_t part_ld, part_bytes;  // fp32 partials: row stride in elements, bytes over all splits
};

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

void shape_product(Product& p, int bn, int splits) {
  p.bn = bn;
  p.mt = (int)((p.M + kFfnTileM - 1) / kFfnTileM);
  // The rows are spread evenly over the tiles and their two CTAs: an SM's share of the operands' bytes is
  // what bounds small batches (333 tokens of 2048 x 2048: tiles of 176 rows instead of 256 and 77). Where A has
  // m contiguous its boxes are 64 wide.
  p.mrows = p.a_mn ? kFfnTileM / 2 : (int)round_up((p.M + 2 * p.mt - 1) / (2 * p.mt), 8);
  const int cols = p.dual ? bn / 2 : bn;
  p.nt = (int)((p.N + cols - 1) / cols);
  p.splits = splits;
  // a stored chunk is 32 columns wide and may start at any multiple of 8 below N: g's part starts
  // past the end of u's last chunk
  p.part_ld = p.dual ? 2 * (round_up(p.N, 16) + 32) : p.N;
  p.part_bytes = splits > 1 ? (int64_t)splits * p.mt * 2 * p.mrows * p.part_ld * 4 : 0;
}

// Picks the tile width and the K splits of one launch's products by an estimate in SM clocks:
//  - a 64-wide K block of a 256 x bn tile takes 2 * bn clocks of the pair's tensor cores (4096 MACs
//    an SM and clock), but no less than an SM's share of A (mrows rows) and B takes (72 bytes a clock;
//    40 where few SMs read weights with n contiguous, whose boxes are 64 short rows: 4 tiles of dh for 128 tokens
//    took 430 clocks a block), nor than the issuing threads take (230, with two blocks to a stage). The backward in us
//    with 72 everywhere, 40 everywhere and the step at a quarter of the pairs: 128 tokens of 2048 x 512 19.1, 16.3,
//    16.3; 257 tokens 19.3, 21.3, 17.9; 1000 tokens 30.1, 30.0, 26.8; 200 tokens of 4096 x 1536 44.0, 47.9, 44.0; but 300
//    tokens of 7168 x 1024 54.8, 49.0, 54.8 and 128 tokens of 4096 x 4096 86.8, 78.3, 86.9;
//  - a unit's fill and drain that nothing overlaps takes about 2500;
//  - with more than one unit a pair, the last round is as long as a full one;
//  - partial sums cost a second launch (about 6000) and their bytes, written and read once.
// Narrow tiles fill the last round better and wide ones feed the tensor cores better. Where B has n
// contiguous, both CTAs' boxes have to start on a 128-byte line, so the width is 128 or 256: a
// box of 64 columns across two lines costs two requests a row (dh at 4096 tokens, hidden 7168, inner
// 2048: 650 clocks a K block at 240 columns, 530 at 256).
void plan(Product* p, int n) {
  int best_bn = 256, best_L = 1 << 30;
  double best = 1e30;
  bool dual = false, b_mn = false;
  int most = 1;
  for (int i = 0; i < n; ++i) {
    dual = dual || p[i].dual;
    b_mn = b_mn || p[i].b_mn;
    most = std::max(most, p[i].nkb);
  }
  for (int bn = b_mn ? 128 : 64; bn <= 256; bn += b_mn ? 128 : 16) {
    for (int L = most; L >= 4 || L == most; L = L / 2) {
      double total = 0, longest = 0, parts = 0;
      int64_t units = 0;
      for (int i = 0; i < n; ++i) {
        shape_product(p[i], bn, std::min(16, (p[i].nkb + L - 1) / L));
        units += (int64_t)p[i].mt * p[i].nt * p[i].splits;
      }
      const double rate = b_mn && units < kPlanPairs / 4 ? 40 : 72;
      for (int i = 0; i < n; ++i) {
        const int64_t u = (int64_t)p[i].mt * p[i].nt * p[i].splits;
        const double kb = (double)((p[i].nkb + p[i].splits - 1) / p[i].splits) *
                              std::max({2.0 * bn, (128 * p[i].mrows + 64 * bn) / rate, 230.0}) + 4.0 * bn;
        total += kb * u;
        longest = std::max(longest, kb);
        parts += p[i].part_bytes;
      }
      const int64_t rounds = (units + kPlanPairs - 1) / kPlanPairs;
      const double mean = total / units;
      const double cost = (n == 1 ? rounds * mean : std::max(longest, total / kPlanPairs + longest / 2)) + 2500 +
                          (parts > 0 ? 6000 + parts * 2 / 3000.0 : 0);
      if (cost < best) {
        best = cost;
        best_bn = bn;
        best_L = L;
      }
      if (L <= 4) break;
    }
  }
  for (int i = 0; i < n; ++i) shape_product(p[i], best_bn, std::min(16, (p[i].nkb + best_L - 1) / best_L));
}

int blocks_of(int64_t k) { return (int)((k + kBK - 1) / kBK); }

// Workspace pieces, each on a 256-byte boundary.
struct Layout {
  int64_t at = 0;
  int64_t take(int64_t bytes) {
    const int64_t o = at;
    at += round_up(bytes, 256);
    return o;
  }
};

struct ForwardPlan {
  Product up, down;
  int64_t h, up_parts, down_parts, bytes;
};

ForwardPlan plan_forward(int64_t T, int64_t H, int64_t D) {
  ForwardPlan f{};
  if (T <= kMvTokens) {  // only h: the small-batch products keep their partial sums on the chip
    Layout l;
    f.h = l.take(T * D * 2);
    f.bytes = l.at;
    return f;
  }
  f.up = Product{T, D, blocks_of(H), true, false, false};
  f.down = Product{T, H, blocks_of(D), false, false, false};
  plan(&f.up, 1);
  plan(&f.down, 1);
  Layout l;
  f.h = l.take(T * D * 2);
  f.up_parts = l.take(f.up.part_bytes);
  f.down_parts = l.take(f.down.part_bytes);
  f.bytes = l.at;
  return f;
}

struct BackwardPlan {
  Product dh, rest[4];  // dx, dW_up, dW_gate, dW_down
  int64_t du, dg, h, dh_parts, parts[4], bytes;
};

// Planned as if every gradient is asked for: a call that leaves some out runs the others' plan.
BackwardPlan plan_backward(int64_t T, int64_t H, int64_t D) {
  BackwardPlan b{};
  b.dh = Product{T, D, blocks_of(H), false, true, false};
  plan(&b.dh, 1);
  b.rest[0] = Product{T, H, 2 * blocks_of(D), false, true, false};
  b.rest[1] = Product{D, H, blocks_of(T), false, true, true};
  b.rest[2] = b.rest[1];
  b.rest[3] = Product{H, D, blocks_of(T), false, true, true};
  plan(b.rest, 4);
  Layout l;
  b.du = l.take(T * D * 2);
  b.dg = l.take(T * D * 2);
  b.h = l.take(T * D * 2);
  b.dh_parts = l.take(b.dh.part_bytes);
  for (int i = 0; i < 4; ++i) b.parts[i] = l.take(b.rest[i].part_bytes);
  b.bytes = l.at;
  return b;
}

// Sizes that a call may have: tensor-map coordinates and row counts stay within 31 bits.
int check_sizes(int64_t T, int64_t H, int64_t D) {
  if (T < 0 || H < 8 || D < 8 || H % 8 != 0 || D % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (T > (1 << 24) || H > (1 << 20) || D > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Activations and weights by 64-wide boxes: K-major {64 k, rows}, MN-major {64 m or n, 64 k}.
int operand(moe_handle* h, CUtensorMap* m, const void* p, int64_t inner, int64_t outer, int rows) {
  return encode_map(h, m, p, inner, outer, (uint64_t)inner * 2, kBK, rows);
}

// A result (or u, g on their way in) by chunks: 32 fp32 or, where `wide`, 64 bf16 columns (128 bytes a row), or 32 bf16
// columns (64 bytes).
int result(moe_handle* h, CUtensorMap* m, void* p, int64_t cols, int64_t rows, bool f32, int64_t ld, int box_rows,
           bool wide = false) {
  return encode_map(h, m, p, cols, rows, (uint64_t)ld * (f32 ? 4 : 2), wide && !f32 ? 64 : 32, box_rows,
                    f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    f32 || wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

void fill_problem(FfnProblem& f, const Product& p, int nseg, int unit0) {
  f.mt = p.mt;
  f.nt = p.nt;
  f.bn = p.bn;
  f.nrows = (int)p.M;
  f.ncols = (int)p.N;
  f.nseg = nseg;
  f.nkb = p.nkb / nseg;
  f.a_mn = p.a_mn;
  f.b_mn = p.b_mn;
  f.b_by_rank = p.dual;
  f.splits = p.splits;
  f.mrows = p.mrows;
  f.mpad = p.mt * 2 * p.mrows;
  f.unit0 = unit0;
  f.gcol = (int)(p.part_ld / 2);
  const uint64_t panel = (uint64_t)kFfnRaster * p.nt;
  f.panel_inv = (uint32_t)(((1ull << 32) + panel - 1) / panel);
}

int units_of(const Product& p) { return p.mt * p.nt * p.splits; }

// Where a product's tiles go: its result (`wide`: the only one, by 128-byte rows), or the splits' partials.
int set_result(moe_handle* h, FfnProblem& f, const Product& p, void* out, int kind, void* parts, bool wide) {
  if (p.splits > 1) {
    f.out_kind = 1;
    return result(h, &f.out, parts, p.part_ld, (int64_t)p.splits * f.mpad, true, p.part_ld, p.mrows);
  }
  f.out_kind = kind;
  return result(h, &f.out, out, p.N, p.M, kind != 0, p.N, p.mrows, wide);
}

FfnReduce reduce_of(const Product& p, const void* parts, void* out, int kind) {
  FfnReduce r{};
  r.parts = static_cast<const float*>(parts);
  r.ld = p.part_ld;
  r.split_stride = (int64_t)p.mt * 2 * p.mrows * p.part_ld;
  r.splits = p.splits;
  r.rows = (int)p.M;
  r.cols = (int)p.N;
  r.gcol = (int)(p.part_ld / 2);
  r.out_kind = kind;
  r.out = out;
  return r;
}

bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}

int cuda_rc(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();  // a refused launch is reported here, not by a later call
  return check_cuda(e);
}

}  // namespace

extern "C" {

int64_t moe_ffn_workspace_bytes(int64_t T, int32_t hidden, int32_t inter, int32_t backward) {
  if (check_sizes(T, hidden, inter) != MOE_OK) return -1;
  if (T == 0) return 0;
  return backward ? plan_backward(T, hidden, inter).bytes : plan_forward(T, hidden, inter).bytes;
}

int moe_ffn_forward(moe_handle* h, const void* x, int64_t T, int32_t hidden, int32_t inter, const moe_shared_w* w,
                    void* out, int32_t out_bf16, void* u, void* g, void* workspace, int64_t workspace_bytes,
                    void* stream) {
  int rc;
  if ((rc = check_sizes(T, hidden, inter))) return rc;
  if (!w || !w->up || !w->gate || !w->down || (u == nullptr) != (g == nullptr)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !out || !workspace)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned({x, w->up, w->gate, w->down, out, u, g, workspace})) return MOE_ERR_MISALIGNED;
  const int64_t H = hidden, D = inter;
  const ForwardPlan f = T > 0 ? plan_forward(T, H, D) : ForwardPlan{};
  const int64_t act = T * H * 2, pre = T * D * 2, wb = H * D * 2;
  if (clobbers({{out, out_bf16 ? act : 2 * act}, {u, pre}, {g, pre}, {workspace, f.bytes}},
               {{x, act}, {w->up, wb}, {w->gate, wb}, {w->down, wb}}))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < f.bytes || !h) return MOE_ERR_INVALID_ARG;
  if (h->ffn_pairs < 1) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  DeviceScope dev(h->device);
  if ((rc = dev.rc())) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  h->ffn_used.store(true, std::memory_order_relaxed);
  char* ws = static_cast<char*>(workspace);
  void* hb = ws + f.h;

  if (T <= kMvTokens) {
    // at most 16 tokens: the weights' bytes are the cost, and the tensor-core tiles would be empty
    MvArgs a{};
    a.m = MvMatrix{{w->up, w->gate}, {nullptr, nullptr}, (int32_t)D, (int32_t)H};
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = H;
    a.T = (int32_t)T;
    a.out = hb;
    a.ldo = D;
    a.out_bf16 = 1;
    a.u = static_cast<uint16_t*>(u);
    a.g = static_cast<uint16_t*>(g);
    if ((rc = cuda_rc(launch_mv_bf16(a, true, h->num_sms, st)))) return rc;
    a.m = MvMatrix{{w->down, nullptr}, {nullptr, nullptr}, (int32_t)H, (int32_t)D};
    a.x = static_cast<const uint16_t*>(hb);
    a.ldx = D;
    a.early = 1;
    a.out = out;
    a.ldo = H;
    a.out_bf16 = out_bf16 != 0;
    a.u = a.g = nullptr;
    return cuda_rc(launch_mv_bf16(a, false, h->num_sms, st));
  }
  FfnParams P{};
  P.meta = h->ffn_meta;
  P.timeout_ns = h->timeout_ns;
  P.nprob = 1;
  // u and g side by side, h from the epilogue
  fill_problem(P.p[0], f.up, 1, 0);
  P.units = units_of(f.up);
  P.save = u != nullptr;
  if ((rc = operand(h, &P.p[0].a[0], x, H, T, f.up.mrows))) return rc;
  if ((rc = operand(h, &P.p[0].b[0], w->up, H, D, f.up.bn / 2))) return rc;
  if ((rc = operand(h, &P.p[0].b[1], w->gate, H, D, f.up.bn / 2))) return rc;
  if ((rc = set_result(h, P.p[0], f.up, hb, 0, ws + f.up_parts, false))) return rc;
  if (u) {
    if ((rc = result(h, &P.out2, u, D, T, false, D, f.up.mrows))) return rc;
    if ((rc = result(h, &P.out3, g, D, T, false, D, f.up.mrows))) return rc;
  }
  if ((rc = cuda_rc(launch_ffn_gemm(P, kFfnSwiglu, h->ffn_pairs, st)))) return rc;
  if (f.up.splits > 1) {
    FfnReduce r = reduce_of(f.up, ws + f.up_parts, hb, 0);
    r.out2 = static_cast<uint16_t*>(u);
    r.out3 = static_cast<uint16_t*>(g);
    if ((rc = cuda_rc(launch_ffn_reduce(r, kFfnSwiglu, h->num_sms, st)))) return rc;
  }
  // out = h W_down^T
  const int kind = out_bf16 ? 0 : 1;
  fill_problem(P.p[0], f.down, 1, 0);
  P.units = units_of(f.down);
  if ((rc = operand(h, &P.p[0].a[0], hb, D, T, f.down.mrows))) return rc;
  if ((rc = operand(h, &P.p[0].b[0], w->down, D, H, f.down.bn / 2))) return rc;
  if ((rc = set_result(h, P.p[0], f.down, out, kind, ws + f.down_parts, true))) return rc;
  if ((rc = cuda_rc(launch_ffn_gemm(P, kFfnStore, h->ffn_pairs, st)))) return rc;
  if (f.down.splits > 1)
    return cuda_rc(launch_ffn_reduce(reduce_of(f.down, ws + f.down_parts, out, kind), kFfnStore, h->num_sms, st));
  return MOE_OK;
}

int moe_ffn_backward(moe_handle* h, const void* dout, const void* x, const void* u, const void* g, int64_t T,
                     int32_t hidden, int32_t inter, const moe_shared_w* w, void* dx, const moe_ffn_grads* grads,
                     uint32_t flags, void* workspace, int64_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_sizes(T, hidden, inter))) return rc;
  if (flags & ~(MOE_FFN_GRAD_F32 | MOE_FFN_GRAD_ADD)) return MOE_ERR_INVALID_ARG;
  if ((flags & MOE_FFN_GRAD_ADD) && !(flags & MOE_FFN_GRAD_F32)) return MOE_ERR_INVALID_ARG;
  if (!w || !w->up || !w->gate || !w->down) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dout || !x || !u || !g || !workspace)) return MOE_ERR_INVALID_ARG;
  const moe_ffn_grads none{};
  const moe_ffn_grads gr = grads ? *grads : none;
  if (!all_aligned({dout, x, u, g, w->up, w->gate, w->down, dx, gr.up, gr.gate, gr.down, workspace}))
    return MOE_ERR_MISALIGNED;
  const int64_t H = hidden, D = inter;
  const BackwardPlan b = T > 0 ? plan_backward(T, H, D) : BackwardPlan{};
  const int64_t act = T * H * 2, pre = T * D * 2, wb = H * D * 2, gb = (flags & MOE_FFN_GRAD_F32) ? 2 * wb : wb;
  if (clobbers({{dx, act}, {gr.up, gb}, {gr.gate, gb}, {gr.down, gb}, {workspace, b.bytes}},
               {{dout, act}, {x, act}, {u, pre}, {g, pre}, {w->up, wb}, {w->gate, wb}, {w->down, wb}}))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < b.bytes || !h) return MOE_ERR_INVALID_ARG;
  if (h->ffn_pairs < 1) return MOE_ERR_UNSUPPORTED;
  DeviceScope dev(h->device);
  if ((rc = dev.rc())) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  h->ffn_used.store(true, std::memory_order_relaxed);
  void* dw[3] = {gr.up, gr.gate, gr.down};
  const int wkind = (flags & MOE_FFN_GRAD_ADD) ? 2 : ((flags & MOE_FFN_GRAD_F32) ? 1 : 0);
  if (T == 0) {  // sums over no tokens
    for (void* p : dw)
      if (p && wkind != 2 && (rc = cuda_rc(cudaMemsetAsync(p, 0, (size_t)H * D * (wkind ? 4 : 2), st)))) return rc;
    return MOE_OK;
  }
  if (!dx && !dw[0] && !dw[1] && !dw[2]) return MOE_OK;
  char* ws = static_cast<char*>(workspace);
  void *du = ws + b.du, *dg = ws + b.dg, *hb = ws + b.h;

  FfnParams P{};
  P.meta = h->ffn_meta;
  P.timeout_ns = h->timeout_ns;
  // dh = dout W_down, and du, dg and h from the epilogue
  P.nprob = 1;
  fill_problem(P.p[0], b.dh, 1, 0);
  P.units = units_of(b.dh);
  if ((rc = result(h, &P.in_u, const_cast<void*>(u), D, T, false, D, b.dh.mrows))) return rc;
  if ((rc = result(h, &P.in_g, const_cast<void*>(g), D, T, false, D, b.dh.mrows))) return rc;
  if ((rc = operand(h, &P.p[0].a[0], dout, H, T, b.dh.mrows))) return rc;
  if ((rc = operand(h, &P.p[0].b[0], w->down, D, H, 64))) return rc;
  if ((rc = set_result(h, P.p[0], b.dh, du, 0, ws + b.dh_parts, false))) return rc;
  if ((rc = result(h, &P.out2, dg, D, T, false, D, b.dh.mrows))) return rc;
  if ((rc = result(h, &P.out3, hb, D, T, false, D, b.dh.mrows))) return rc;
  if ((rc = cuda_rc(launch_ffn_gemm(P, kFfnDSwiglu, h->ffn_pairs, st)))) return rc;
  if (b.dh.splits > 1) {
    FfnReduce r = reduce_of(b.dh, ws + b.dh_parts, du, 0);
    r.out2 = static_cast<uint16_t*>(dg);
    r.out3 = static_cast<uint16_t*>(hb);
    r.u = static_cast<const uint16_t*>(u);
    r.g = static_cast<const uint16_t*>(g);
    if ((rc = cuda_rc(launch_ffn_reduce(r, kFfnDSwiglu, h->num_sms, st)))) return rc;
  }
  // the four gradients in one launch
  struct Grad {
    void* out;
    const void* a[2];
    const void* b[2];
    int64_t am, bn;  // inner extents of A and B
  };
  const Grad want[4] = {{dx, {du, dg}, {w->up, w->gate}, D, H},
                        {dw[0], {du, nullptr}, {x, nullptr}, D, H},
                        {dw[1], {dg, nullptr}, {x, nullptr}, D, H},
                        {dw[2], {dout, nullptr}, {hb, nullptr}, H, D}};
  int n = 0, units = 0;
  for (int i = 0; i < 4; ++i) {
    if (!want[i].out) continue;
    FfnProblem& f = P.p[n++];
    fill_problem(f, b.rest[i], i == 0 ? 2 : 1, units);
    units += units_of(b.rest[i]);
    for (int s = 0; s < (i == 0 ? 2 : 1); ++s) {
      if ((rc = operand(h, &f.a[s], want[i].a[s], want[i].am, T, i == 0 ? b.rest[0].mrows : 64))) return rc;
      if ((rc = operand(h, &f.b[s], want[i].b[s], want[i].bn, i == 0 ? D : T, 64))) return rc;
    }
    if ((rc = set_result(h, f, b.rest[i], want[i].out, i == 0 ? 0 : wkind, ws + b.parts[i], true))) return rc;
  }
  P.nprob = n;
  P.units = units;
  if ((rc = cuda_rc(launch_ffn_gemm(P, kFfnStore, h->ffn_pairs, st)))) return rc;
  for (int i = 0; i < 4; ++i)
    if (want[i].out && b.rest[i].splits > 1 &&
        (rc = cuda_rc(launch_ffn_reduce(reduce_of(b.rest[i], ws + b.parts[i], want[i].out, i == 0 ? 0 : wkind),
                                        kFfnStore, h->num_sms, st))))
      return rc;
  return MOE_OK;
}

}  // extern "C"
