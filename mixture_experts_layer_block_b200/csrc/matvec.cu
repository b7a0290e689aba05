// matvec.cu -- products of at most 16 tokens with bf16 or 4-bit weights (matvec.cuh).
//
// What bounds them: the weights' bytes, each read once from HBM, and at the smallest sizes the
// latency of one trip there. So the design is about bytes in flight and short dependent chains:
//  - a unit is 16 output rows (for the experts: of one expert, or, in the down projection, of the sum
//    over all experts that were hit); the CTA's 8 warps split its K blocks evenly, and the down
//    projection's K runs over every expert hit, so that warps are even there too;
//  - each lane copies its own 16-byte pieces of weights to shared memory with cp.async, a fixed number
//    of blocks ahead and across unit boundaries, and reads only its own: no barrier in the K loop;
//  - the products run on mma.sync m16n8k16 (fp32 accumulation): weights come out of a register
//    unpacking as the A fragment, tokens are the N columns. tcgen05 would need the unpacked weights
//    written back to shared memory, for products that take a fraction of the copy's time anyway;
//  - 4-bit codes become bf16 exactly: (code | 0x4300) is 128 + code, less bf16(128 + zero). A group's
//    sum is scaled in fp32, so nothing is rounded before the result;
//  - a kernel behind another of the same call starts copying weights before that one is done.
// The warps' partial sums meet in shared memory and are added in warp order: equal inputs give equal
// bits.
#include <algorithm>

#include "ffn.cuh"
#include "launch.h"
#include "matvec.cuh"

namespace moe {

namespace {

constexpr int kMvWarps = 8;
constexpr int kMvThreads = kMvWarps * 32;
constexpr int kMvSmem = 227 * 1024;      // shared memory of an SM that CTAs can use
constexpr int kMvMaxDepth = 12;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  const uint32_t n = in ? 16u : 0u;  // 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool in) {
  const uint32_t n = in ? (uint32_t)kBytes : 0u;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The experts of a batch: which were hit, in rising order, and by which tokens.
struct Hits {
  int32_t n;
  uint16_t expert[kMvMaxSlots];
  uint16_t mask[kMvMaxSlots];
  int16_t id[kMvMaxSlots];   // the caller's ids, -1 where they are out of range
  float w[kMvMaxSlots];
};

template <bool kW4, bool kDual, int kKind, int kNT, bool kG32, bool kZeros>
struct Mv {
  static constexpr int kMats = kDual ? 2 : 1;
  static constexpr int kScaleBytes = kZeros ? 8 : 4;             // a lane's entries of a group: rows q and q + 8
  static constexpr int kGroups = kG32 ? 2 : 1;                   // groups of a K block
  static constexpr int kLane = kW4 ? 16 : 64;                    // weight bytes of a lane and block
  static constexpr int kMetaLane = kW4 ? kScaleBytes * kGroups : 0;
  static constexpr int kStage = kMats * 32 * (kLane + kMetaLane);  // bytes of a warp's block
  static constexpr int kCols = kNT * 8;
  static constexpr int kRedLd = kMvRows + 1;
  static constexpr int kRed = kMats * kCols * kRedLd;            // floats of a warp's partial sums
  static constexpr int kRest = 2 * kMvWarps * kRed * (int)sizeof(float) + (kKind != kMvOne ? (int)sizeof(Hits) : 0);
  // two CTAs to an SM where each still gets 4 blocks a warp, else one
  static constexpr int depth_of(int ctas) {
    return std::min(kMvMaxDepth, (kMvSmem / ctas - 1024 - kRest) / (kMvWarps * kStage));
  }
  static constexpr int kPerSm = depth_of(2) >= 4 ? 2 : 1;
  static constexpr int kDepth = depth_of(kPerSm);
  static constexpr int kRingTotal = kMvWarps * kStage * kDepth;
  static constexpr int kSmem = kRingTotal + kRest;
  static_assert(kDepth >= 3, "enough blocks in flight");
};

// A position in a warp's sequence of K blocks: its units, and in each the warp's share of blocks.
struct Cursor {
  int u;        // unit
  int b, hi;    // block of the unit's K (all its experts), end of this warp's share
  int ent;      // entry of the hit list (n: the shared expert)
  int kb, nb;   // block of the entry's matrix, blocks it has
  int tile;     // 16-row tile of the entry's matrix
};

}  // namespace

template <bool kW4, bool kDual, int kKind, int kNT, bool kG32, bool kZeros>
__global__ void __launch_bounds__(kMvThreads, Mv<kW4, kDual, kKind, kNT, kG32, kZeros>::kPerSm)
    mv_kernel(const __grid_constant__ MvArgs a) {
  using C = Mv<kW4, kDual, kKind, kNT, kG32, kZeros>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane >> 2, c = lane & 3;
  float* red = reinterpret_cast<float*>(smem + C::kRingTotal);
  Hits* hits = reinterpret_cast<Hits*>(smem + C::kRingTotal + 2 * kMvWarps * C::kRed * sizeof(float));
  uint8_t* ring = smem + (size_t)warp * C::kStage * C::kDepth;

  if (!a.early) griddep_wait();
  int nhit = 1;
  if constexpr (kKind != kMvOne) {
    // the partial sums' buffer is free until the first unit: token masks by expert
    uint32_t* emask = reinterpret_cast<uint32_t*>(red);
    static_assert(2 * kMvWarps * C::kRed * 4 >= kMaxExperts * 4, "the masks fit");
    for (int e = threadIdx.x; e < a.E; e += kMvThreads) emask[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < a.T * a.k; s += kMvThreads) {
      const int e = __ldcg(a.ids + s);
      const bool in = e >= 0 && e < a.E;
      hits->id[s] = in ? (int16_t)e : (int16_t)-1;
      hits->w[s] = __ldcg(a.topk_w + s);
      if (in) atomicOr(&emask[e], 1u << (s / a.k));
    }
    __syncthreads();
    if (warp == 0) {
      int n = 0;
      for (int e0 = 0; e0 < a.E; e0 += 32) {
        uint32_t m = e0 + lane < a.E ? emask[e0 + lane] : 0;
        if (a.capacity > 0)
          while (__popc(m) > a.capacity) m &= ~(0x80000000u >> __clz(m));  // the highest token is dropped
        const uint32_t any = __ballot_sync(0xffffffffu, m != 0);
        if (m) {
          const int at = n + __popc(any & ((1u << lane) - 1));
          hits->expert[at] = (uint16_t)(e0 + lane);
          hits->mask[at] = (uint16_t)m;
        }
        n += __popc(any);
      }
      if (lane == 0) hits->n = n;
    }
    __syncthreads();
    nhit = hits->n;
  }

  const int tiles = ceil_div(a.m.R, kMvRows), nb = ceil_div(a.m.K, kMvBK);
  const int stiles = ceil_div(a.shared.R, kMvRows), snb = ceil_div(a.shared.K, kMvBK);
  const int units = kKind == kMvOne ? tiles : (kKind == kMvUp ? nhit * tiles + stiles : tiles);

  auto start_entry = [&](Cursor& p) {  // kMvDown: the entry that block p.b belongs to
    p.ent = min(p.b / max(nb, 1), nhit);
    p.kb = p.b - p.ent * nb;
    p.nb = p.ent == nhit ? snb : nb;
  };
  auto start_unit = [&](Cursor& p) {
    while (p.u < units) {
      int total;
      if constexpr (kKind == kMvDown) {
        p.tile = p.u;
        total = nhit * nb + snb;
      } else if constexpr (kKind == kMvUp) {
        const bool sh = p.u >= nhit * tiles;
        p.ent = sh ? nhit : p.u / tiles;
        p.tile = sh ? p.u - nhit * tiles : p.u % tiles;
        total = p.nb = sh ? snb : nb;
      } else {
        p.ent = 0;
        p.tile = p.u;
        total = p.nb = nb;
      }
      p.b = (int)((int64_t)warp * total / kMvWarps);
      p.hi = (int)((int64_t)(warp + 1) * total / kMvWarps);
      if (p.b < p.hi) {
        if constexpr (kKind == kMvDown) start_entry(p);
        else p.kb = p.b;
        return;
      }
      p.u += gridDim.x;  // fewer blocks than warps: nothing of this unit is this warp's
    }
  };
  auto advance = [&](Cursor& p) {
    ++p.b;
    ++p.kb;
    if (p.b >= p.hi) {
      p.u += gridDim.x;
      start_unit(p);
    } else if (kKind == kMvDown && p.kb == p.nb) {
      start_entry(p);
    }
  };

  // ---- weights: block `p` into ring slot `slot`, this lane's pieces only ----
  auto copy = [&](const Cursor& p, int slot) {
    const bool sh = kKind != kMvOne && p.ent == nhit;
    const MvMatrix& m = sh ? a.shared : a.m;
    const int e = kKind == kMvOne || sh ? 0 : hits->expert[p.ent];
    const uint32_t dst = smem_u32(ring) + slot * C::kStage + lane * C::kLane;
#pragma unroll
    for (int i = 0; i < C::kMats; ++i) {
      if constexpr (kW4) {
        const int64_t tile = (int64_t)e * int4_row_tiles(m.R) + p.tile;
        const uint8_t* w = static_cast<const uint8_t*>(m.w[i]) + (tile * p.nb + p.kb) * 512 + lane * 16;
        cp_async16(dst + i * 32 * C::kLane, w, true);
        const int G = (m.K + a.group - 1) / a.group;
        const uint32_t md = smem_u32(ring) + slot * C::kStage + C::kMats * 32 * C::kLane + i * 32 * C::kMetaLane +
                            lane * C::kMetaLane;
#pragma unroll
        for (int g2 = 0; g2 < C::kGroups; ++g2) {
          const int g = kG32 ? 2 * p.kb + g2 : (a.group == 64 ? p.kb : p.kb >> 1);
          const bool in = g < G;
          const uint8_t* s = static_cast<const uint8_t*>(m.scales[i]) +
                             (tile * G + (in ? g : 0)) * (kMvRows * (kZeros ? 4 : 2)) + q * C::kScaleBytes;
          cp_async_small<C::kScaleBytes>(md + g2 * C::kScaleBytes, s, in);
        }
      } else {
        const uint16_t* w = static_cast<const uint16_t*>(m.w[i]);
#pragma unroll
        for (int r2 = 0; r2 < 2; ++r2) {
          const int row = p.tile * kMvRows + q + 8 * r2;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = p.kb * kMvBK + 32 * h + 8 * c;  // K is a multiple of 8
            const bool in = row < m.R && k < m.K;
            // the four pieces of a lane are 16 lanes' widths apart: conflict-free writes and reads
            cp_async16(smem_u32(ring) + slot * C::kStage + (i * 4 + r2 * 2 + h) * 512 + lane * 16,
                       in ? w + (int64_t)row * m.K + k : w, in);
          }
        }
      }
    }
  };

  // ---- activations: this lane's columns of block `p` for tokens q and q + 8 ----
  auto load_x = [&](const Cursor& p, uint4 (&x)[kNT][2]) {
    const bool sh = kKind != kMvOne && p.ent == nhit;
    const int K = sh ? a.shared.K : a.m.K;
    const uint32_t members = kKind == kMvOne || sh ? 0xffffu : hits->mask[p.ent];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const int t = q + 8 * n;
      const bool in = t < a.T && (members >> t & 1);
      int64_t row = t;
      if constexpr (kKind == kMvDown) {
        if (sh) {
          row = (int64_t)a.T * a.k + t;
        } else if (in) {
          const int e = hits->expert[p.ent];
          int j = 0;
          while (j < a.k - 1 && hits->id[t * a.k + j] != e) ++j;
          row = (int64_t)t * a.k + j;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = p.kb * kMvBK + 32 * h + 8 * c;
        // plain loads: the CTAs of an SM share the rows through L1
        x[n][h] = in && k < K ? *reinterpret_cast<const uint4*>(a.x + row * a.ldx + k) : make_uint4(0, 0, 0, 0);
      }
    }
  };

  Cursor prod{};
  prod.u = blockIdx.x;
  start_unit(prod);
  Cursor cur = prod, nxt = prod;
  int slot_in = 0, slot = 0;
#pragma unroll 1
  for (int i = 0; i < C::kDepth - 1; ++i) {
    if (prod.u < units) {
      copy(prod, slot_in);
      advance(prod);
    }
    cp_async_commit();
    if (++slot_in == C::kDepth) slot_in = 0;
  }
  if (a.early) griddep_wait();
  griddep_launch_dependents();

  uint4 xn[kNT][2];
  if (nxt.u < units) load_x(nxt, xn);
  int parity = 0;
#pragma unroll 1
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    float acc[C::kMats][kNT][4] = {};   // of the current expert
    float tot[kNT][4] = {};             // kMvDown: router-weighted, over the experts so far
    auto close_entry = [&](int ent) {
      if constexpr (kKind == kMvDown) {
        const bool sh = ent == nhit;
        const uint32_t members = sh ? 0xffffu : hits->mask[ent];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2) {
            const int t = 8 * n + 2 * c + t2;
            if (t < a.T && (members >> t & 1)) {
              float w = sh ? 1.f : 0.f;
              if (!sh) {  // an expert named twice counts twice
                const int e = hits->expert[ent];
                for (int j = 0; j < a.k; ++j)
                  if (hits->id[t * a.k + j] == e) w += hits->w[t * a.k + j];
              }
              tot[n][t2] += w * acc[0][n][t2];
              tot[n][2 + t2] += w * acc[0][n][2 + t2];
            }
            acc[0][n][t2] = acc[0][n][2 + t2] = 0.f;
          }
      }
    };
    while (cur.u == u) {
      if (prod.u < units) {
        copy(prod, slot_in);
        advance(prod);
      }
      cp_async_commit();
      if (++slot_in == C::kDepth) slot_in = 0;
      uint4 x[kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        x[n][0] = xn[n][0];
        x[n][1] = xn[n][1];
      }
      advance(nxt);
      if (nxt.u < units) load_x(nxt, xn);
      cp_async_wait<C::kDepth - 1>();
      const uint8_t* st = ring + (size_t)slot * C::kStage;
      if (++slot == C::kDepth) slot = 0;
#pragma unroll
      for (int i = 0; i < C::kMats; ++i) {
        if constexpr (kW4) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(st + i * 32 * C::kLane + lane * 16);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          const uint8_t* meta = st + C::kMats * 32 * C::kLane + (i * 32 + lane) * C::kMetaLane;
#pragma unroll
          for (int g2 = 0; g2 < C::kGroups; ++g2) {
            float s0, s1;                            // rows q and q + 8
            uint32_t z0 = 0x43084308u, z1 = z0;      // bf16x2 of 128 + zero
            if constexpr (kZeros) {
              const uint2 v = *reinterpret_cast<const uint2*>(meta + g2 * 8);
              s0 = __uint_as_float(v.x << 16);
              s1 = __uint_as_float(v.y << 16);
              z0 = __byte_perm(v.x, 0, 0x3232);
              z1 = __byte_perm(v.y, 0, 0x3232);
            } else {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(meta + g2 * 4);
              s0 = __uint_as_float(v << 16);
              s1 = __uint_as_float(v & 0xffff0000u);
            }
            float part[kNT][4] = {};
#pragma unroll
            for (int jj = 0; jj < 4 / C::kGroups; ++jj) {
              const int j = g2 * 2 * (C::kGroups - 1) + jj;
              uint32_t f[4];
#pragma unroll
              for (int n = 0; n < 4; ++n)
                f[n] = sub_bf16x2(((w[j] >> (4 * n)) & 0x000f000fu) | 0x43004300u, (n & 1) ? z1 : z0);
#pragma unroll
              for (int n = 0; n < kNT; ++n) {
                const uint4 v = x[n][j >> 1];
                if (j & 1) mma_bf16(part[n], f, v.z, v.w);
                else mma_bf16(part[n], f, v.x, v.y);
              }
            }
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
              acc[i][n][0] += s0 * part[n][0];
              acc[i][n][1] += s0 * part[n][1];
              acc[i][n][2] += s1 * part[n][2];
              acc[i][n][3] += s1 * part[n][3];
            }
          }
        } else {
          uint4 w[2][2];  // rows q, q + 8; halves of the block
#pragma unroll
          for (int r2 = 0; r2 < 2; ++r2)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[r2][h] = *reinterpret_cast<const uint4*>(st + (i * 4 + r2 * 2 + h) * 512 + lane * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 lo = w[0][j >> 1], hi = w[1][j >> 1];
            const uint32_t f[4] = {(j & 1) ? lo.z : lo.x, (j & 1) ? hi.z : hi.x, (j & 1) ? lo.w : lo.y,
                                   (j & 1) ? hi.w : hi.y};
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
              const uint4 v = x[n][j >> 1];
              if (j & 1) mma_bf16(acc[i][n], f, v.z, v.w);
              else mma_bf16(acc[i][n], f, v.x, v.y);
            }
          }
        }
      }
      const int ent = cur.ent;
      advance(cur);
      if (kKind == kMvDown && (cur.u != u || cur.ent != ent)) close_entry(ent);
    }

    // ---- the warps' sums meet ----
    float* mine = red + (parity * kMvWarps + warp) * C::kRed;
#pragma unroll
    for (int i = 0; i < C::kMats; ++i)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          mine[(i * C::kCols + 8 * n + 2 * c + (v & 1)) * C::kRedLd + q + 8 * (v >> 1)] =
              kKind == kMvDown ? tot[n][v] : acc[i][n][v];
    __syncthreads();
    const int o = threadIdx.x;
    if (o < kMvRows * C::kCols) {
      const int r = o % kMvRows, t = o / kMvRows;
      float s[C::kMats];
#pragma unroll
      for (int i = 0; i < C::kMats; ++i) {
        s[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kMvWarps; ++w)
          s[i] += red[(parity * kMvWarps + w) * C::kRed + (i * C::kCols + t) * C::kRedLd + r];
      }
      int tile = u, R = a.m.R;
      int64_t row = t;
      bool in = t < a.T;
      if constexpr (kKind == kMvUp) {
        const bool sh = u >= nhit * tiles;
        tile = sh ? u - nhit * tiles : u % tiles;
        if (sh) {
          R = a.shared.R;
          row = (int64_t)a.T * a.k + t;
        } else {
          const int ent = u / tiles, e = hits->expert[ent];
          in = in && (hits->mask[ent] >> t & 1);
          int j = 0;
          if (in)
            while (j < a.k - 1 && hits->id[t * a.k + j] != e) ++j;
          row = (int64_t)t * a.k + j;
        }
      }
      const int col = tile * kMvRows + r;
      if (in && col < R) {
        const int64_t at = row * a.ldo + col;
        float v = s[0];
        if constexpr (kDual) {
          v = swiglu(s[0], s[1]);
          if (kKind == kMvOne && a.u) {
            a.u[at] = (uint16_t)(pack_bf16x2(s[0], 0.f) & 0xffffu);
            a.g[at] = (uint16_t)(pack_bf16x2(s[1], 0.f) & 0xffffu);
          }
        }
        if (a.out_bf16) static_cast<uint16_t*>(a.out)[at] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
        else static_cast<float*>(a.out)[at] = v;
      }
    }
    parity ^= 1;  // the next unit writes the other buffer: one barrier a unit is enough
  }
  cp_async_wait<0>();
}

namespace {

template <bool kW4, bool kDual, int kKind, int kNT, bool kG32, bool kZeros>
cudaError_t launch_mv(const MvArgs& a, int64_t units, int num_sms, cudaStream_t stream) {
  using C = Mv<kW4, kDual, kKind, kNT, kG32, kZeros>;
  auto* k = mv_kernel<kW4, kDual, kKind, kNT, kG32, kZeros>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(units, C::kPerSm * num_sms));
  return launch_k(k, dim3(grid), dim3(kMvThreads), C::kSmem, stream, a);
}

template <bool kDual, int kKind, bool kG32, bool kZeros>
cudaError_t pick_nt(const MvArgs& a, int64_t units, int num_sms, cudaStream_t stream) {
  return a.T <= 8 ? launch_mv<true, kDual, kKind, 1, kG32, kZeros>(a, units, num_sms, stream)
                  : launch_mv<true, kDual, kKind, 2, kG32, kZeros>(a, units, num_sms, stream);
}

template <bool kDual, int kKind>
cudaError_t pick_int4(const MvArgs& a, bool zeros, int64_t units, int num_sms, cudaStream_t stream) {
  if (a.group == 32)
    return zeros ? pick_nt<kDual, kKind, true, true>(a, units, num_sms, stream)
                 : pick_nt<kDual, kKind, true, false>(a, units, num_sms, stream);
  return zeros ? pick_nt<kDual, kKind, false, true>(a, units, num_sms, stream)
               : pick_nt<kDual, kKind, false, false>(a, units, num_sms, stream);
}

// ---- laying out 4-bit matrices ----------------------------------------------------------------
// One warp per 16 rows x 128 columns (two K blocks): lane 4 q + c holds its pieces of both blocks,
// 64 values of rows q and q + 8 as v[block][half][row][column]. Writes the codes' words.
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t tile, int nb, int kb0, const uint8_t (&v)[2][2][2][8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (kb0 + b >= nb) break;
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t x = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n)  // (row q | q + 8, columns + 0, + 2) low, (+ 1, + 3) high half word
          x |= (uint32_t)v[b][h][n & 1][4 * i + 2 * ((n >> 1) & 1) + (n >> 2)] << (4 * n);
        w[2 * h + i] = x;
      }
    *reinterpret_cast<uint4*>(codes + (tile * nb + kb0 + b) * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ void store_scale(uint8_t* scales, int64_t tile, int G, int g, int row, bool zeros, uint32_t s,
                                            uint32_t zero) {
  const int at = 2 * (row & 7) + (row >> 3);
  const int64_t o = (tile * G + g) * kMvRows + at;
  if (zeros)
    reinterpret_cast<uint32_t*>(scales)[o] = s | (pack_bf16x2(128.f + (float)zero, 0.f) << 16);
  else
    reinterpret_cast<uint16_t*>(scales)[o] = (uint16_t)s;
}

// Scale and zero point of a group from its extremes (both counting 0), in IEEE fp32: symmetric
// s = bf16(max|v| / 7), zero 8; or s = bf16((max - min) / 15), zero = round(-min / s) in 0..15.
// A scale of 0 (a group of zeros, or of values whose scale underflows) leaves every code at zero 8.
template <bool kZeros>
__global__ void __launch_bounds__(256) int4_quantize_kernel(const uint16_t* __restrict__ src, int64_t R, int K, int group,
                                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, q = lane >> 2, c = lane & 3;
  const int nb = (int)int4_col_blocks(K), np = (nb + 1) / 2, G = (int)int4_groups(K, group);
  const int64_t tiles = int4_row_tiles(R), items = tiles * np;
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * 8) {
    const int64_t tile = it / np;
    const int kb0 = (int)(it % np) * 2;
    float f[2][2][2][8];
    float lo[4][2], hi[4][2];  // per 32 columns and row
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = tile * kMvRows + q + 8 * r;
        const int k = kb0 * kMvBK + 32 * p + 8 * c;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < R && k < K) x = __ldg(reinterpret_cast<const uint4*>(src + row * K + k));
        float(&v)[8] = f[p >> 1][p & 1][r];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        add_bf16x8(v, x);
        lo[p][r] = hi[p][r] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[p][r] = fminf(lo[p][r], v[i]);
          hi[p][r] = fmaxf(hi[p][r], v[i]);
        }
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {  // the four lanes of a row
          lo[p][r] = fminf(lo[p][r], __shfl_xor_sync(0xffffffffu, lo[p][r], o));
          hi[p][r] = fmaxf(hi[p][r], __shfl_xor_sync(0xffffffffu, hi[p][r], o));
        }
      }
    uint8_t v[2][2][2][8];
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int first = group == 32 ? p : (group == 64 ? p & ~1 : 0), n = group / 32;
        float mn = 0.f, mx = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i >= first && i < first + n) {
            mn = fminf(mn, lo[i][r]);
            mx = fmaxf(mx, hi[i][r]);
          }
        const float raw = kZeros ? __fdiv_rn(mx - mn, 15.f) : __fdiv_rn(fmaxf(mx, -mn), 7.f);
        const uint32_t sb = pack_bf16x2(raw, 0.f) & 0xffffu;
        const float s = __uint_as_float(sb << 16);
        const float zero = kZeros && s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-mn, s)), 0.f), 15.f) : 8.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[p >> 1][p & 1][r][i] =
              s > 0.f ? (uint8_t)fminf(fmaxf(rintf(__fdiv_rn(f[p >> 1][p & 1][r][i], s)) + zero, 0.f), 15.f) : (uint8_t)8;
        const int g = (kb0 * kMvBK + 32 * p) / group;
        if (p == first && c == 0 && g < G) store_scale(scales, tile, G, g, q + 8 * r, kZeros, sb, (uint32_t)zero);
      }
    store_codes(codes, tile, nb, kb0, v);
  }
}

__global__ void __launch_bounds__(256) int4_pack_kernel(const uint8_t* __restrict__ src, const uint16_t* __restrict__ s,
                                                        const uint8_t* __restrict__ z, int64_t R, int K, int group,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, q = lane >> 2, c = lane & 3;
  const int nb = (int)int4_col_blocks(K), np = (nb + 1) / 2, G = (int)int4_groups(K, group);
  const int64_t tiles = int4_row_tiles(R), items = tiles * np;
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * 8) {
    const int64_t tile = it / np;
    const int kb0 = (int)(it % np) * 2;
    uint8_t v[2][2][2][8];
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = tile * kMvRows + q + 8 * r;
        const int k = kb0 * kMvBK + 32 * p + 8 * c;
        uint32_t x = 0;
        if (row < R && k < K) x = __ldg(reinterpret_cast<const uint32_t*>(src + row * (K / 2) + k / 2));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p >> 1][p & 1][r][i] = (uint8_t)(x >> (4 * i) & 15u);
        const int g = (kb0 * kMvBK + 32 * p) / group;
        if ((kb0 * kMvBK + 32 * p) % group == 0 && c == 0 && g < G) {
          const bool in = row < R;
          store_scale(scales, tile, G, g, q + 8 * r, z != nullptr, in ? __ldg(s + row * G + g) : 0u,
                      in && z ? __ldg(z + row * G + g) : 8u);
        }
      }
    store_codes(codes, tile, nb, kb0, v);
  }
}

int layout_grid(int64_t R, int64_t K, int num_sms) {
  const int64_t items = int4_row_tiles(R) * ((int4_col_blocks(K) + 1) / 2);
  return (int)std::max<int64_t>(1, std::min<int64_t>((items + 7) / 8, (int64_t)num_sms * 16));
}

}  // namespace

cudaError_t launch_int4_quantize(const uint16_t* src, int64_t R, int64_t K, int group, bool zeros, void* codes,
                                 void* scales, int num_sms, cudaStream_t stream) {
  auto* k = zeros ? int4_quantize_kernel<true> : int4_quantize_kernel<false>;
  return launch_k(k, dim3(layout_grid(R, K, num_sms)), dim3(256), 0, stream, src, R, (int)K, group,
                  static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

cudaError_t launch_int4_pack(const uint8_t* q, const uint16_t* s, const uint8_t* z, int64_t R, int64_t K, int group,
                             void* codes, void* scales, int num_sms, cudaStream_t stream) {
  return launch_k(int4_pack_kernel, dim3(layout_grid(R, K, num_sms)), dim3(256), 0, stream, q, s, z, R, (int)K, group,
                  static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

cudaError_t launch_mv_bf16(const MvArgs& a, bool dual, int num_sms, cudaStream_t stream) {
  const int64_t units = ceil_div(a.m.R, kMvRows);
  if (dual)
    return a.T <= 8 ? launch_mv<false, true, kMvOne, 1, false, false>(a, units, num_sms, stream)
                    : launch_mv<false, true, kMvOne, 2, false, false>(a, units, num_sms, stream);
  return a.T <= 8 ? launch_mv<false, false, kMvOne, 1, false, false>(a, units, num_sms, stream)
                  : launch_mv<false, false, kMvOne, 2, false, false>(a, units, num_sms, stream);
}

cudaError_t launch_mv_int4(const MvArgs& a, int kind, bool zeros, int num_sms, cudaStream_t stream) {
  const int64_t tiles = ceil_div(a.m.R, kMvRows);
  if (kind == kMvOne) return pick_int4<false, kMvOne>(a, zeros, tiles, num_sms, stream);
  if (kind == kMvDown) return pick_int4<false, kMvDown>(a, zeros, tiles, num_sms, stream);
  // at most one expert per slot
  const int64_t units = tiles * std::min(a.E, a.T * a.k) + ceil_div(a.shared.R, kMvRows);
  return pick_int4<true, kMvUp>(a, zeros, units, num_sms, stream);
}

}  // namespace moe
