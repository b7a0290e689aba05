// matvec.cu -- products of at most 16 tokens with bf16 or 4-bit weights (matvec.cuh).
//
// What bounds them: the weights' bytes, each read once from HBM, and at the smallest sizes the
// latency of one trip there. So the design is about bytes in flight and short dependent chains:
//  - a unit is 16 output rows (for the experts: of one expert, or, in the down projection, of the sum
//    over all experts that were hit, whose K blocks then follow one another). A CTA (one to an SM) has
//    a run of units, and its 16 warps split the run's K blocks evenly, whatever the units' number and
//    length;
//  - each warp copies its weights to a ring of its own in shared memory with cp.async, a fixed number of
//    blocks ahead and across unit boundaries: no barrier of the CTA in the K loop;
//  - the products run on mma.sync m16n8k16 (fp32 accumulation): weights come out of a register
//    unpacking as the A fragment, tokens are the N columns. tcgen05 would need the unpacked weights
//    written back to shared memory, for products that take a fraction of the copy's time anyway;
//  - 4-bit codes become bf16 exactly: (code | 0x4300) is 128 + code, less bf16(128 + zero). A group's
//    sum is scaled in fp32, so nothing of one product is rounded before its result. Of two, h is: to bf16, the
//    operand type of the down product's MMA, as everywhere in the layer;
//  - a kernel behind another of the same call may copy weights before that one is done.
// The sums of a unit that several warps share meet in shared memory and are added in warp order: equal
// inputs give equal bits.
// Measured (one B200, calls back to back on three sets of weights): W of 151552 x 4096 in 4 bits times one
// token 77 us, 4.1 TB/s, bound by the integer pipe (unpacking 8 codes takes 7 of its half-rate operations:
// with the shifts left out, and wrong numbers, 12 % less time); 2048 x 7168 times one token 4.5 us, which is
// latency: about 1.2 us to set up, 1 us to the first data, 0.3 us for the sums, and the change of kernels.
#include <algorithm>
#include <atomic>
#include <climits>

#include "ffn.cuh"
#include "launch.h"
#include "matvec.cuh"

namespace moe {

namespace {

// Shared memory of a CTA, but for rings of fewer than two blocks. What it leaves of an SM's 256 KB is L1, where the
// activations are found again, and one or two blocks in flight a warp (16 to 64 KB an SM) are enough: with 227 KB the
// experts took 42.4 us for 16 tokens where they now take 37.9, the block 23.1 us for 16 tokens instead of 21.5, and
// one token times 37888 x 4096 in 4 bits 25.7 us instead of 22.6.
constexpr int kMvSmem = 63 * 1024;
constexpr int kMvMaxDepth = 12;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zeros(uint32_t dst, const void* src, bool in) {
  const uint32_t n = in ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same onto zeros.
__device__ __forceinline__ void mma_bf16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The experts of a batch: which were hit, in rising order, by which tokens, and for every (expert,
// token) pair, in that order, the token's router weight for that expert. An entry has at most 8 tokens
// (the MMA's columns): an expert with more has two, and its weights are read twice, in turn.
struct Hits {
  int32_t n;
  uint16_t expert[kMvMaxSlots];
  uint16_t mask[kMvMaxSlots];
  uint16_t first[kMvMaxSlots];  // the entry's first pair
  float weight[kMvMaxSlots];    // by pair: an expert that a token names twice counts twice
  uint8_t token[kMvMaxSlots];   // by pair
};

constexpr int kMvWarps = 16;  // one CTA to an SM (20 warps, with fewer registers each, were within 5 % either way)
constexpr int kMvThreads = kMvWarps * 32;

// kGroup: columns to a scale, 0 for bf16 weights.
template <bool kDual, int kKind, int kNT, int kGroup, bool kZeros>
struct Mv {
  static constexpr bool kW4 = kGroup != 0;
  static constexpr int kMats = kDual ? 2 : 1;
  static constexpr int kCols = kW4 ? kInt4Cols : 64;     // columns of a K block
  static constexpr int kVecs = kCols / 64;               // 16-byte vectors of a lane's activations in half a block
  static constexpr int kParts = kW4 ? kInt4Cols / kGroup : 1;        // groups of a block
  static constexpr int kMeta = kW4 ? (kZeros ? 8 : 4) * kParts : 0;  // scale bytes of a lane and block
  static constexpr int kCodes = kW4 ? 1024 : 2048;                   // weight bytes of a warp's block
  static constexpr int kMat = kCodes + 8 * kMeta;                    // with its scales
  static constexpr int kStage = kMats * kMat;
  static constexpr int kXT = kKind == kMvOne ? kNT : 1;              // token tiles of a product
  static constexpr int kTok = kKind == kMvUp ? 8 : kNT * 8;          // columns of a unit's sums
  static constexpr int kRed = kMats * kTok * kMvRows;                // floats of a warp's partial sums
  static constexpr int kRest = kMvWarps * kRed * (int)sizeof(float) + (kKind != kMvOne ? (int)sizeof(Hits) : 0);
  static constexpr int kDepth = std::max(2, std::min(kMvMaxDepth, (kMvSmem - 1024 - kRest) / (kMvWarps * kStage)));
  static constexpr int kRingTotal = kMvWarps * kStage * kDepth;
  static constexpr int kSmem = kRingTotal + kRest;
  static_assert(kSmem <= 227 * 1024, "what a CTA can have");
  // percent of an SM's shared memory (228 KB, 1 KB of each CTA for the system) that the kernel asks for
  static constexpr int kCarveout = std::min(100, ((kSmem + 2047) / 1024 * 100 + 227) / 228);
};

// Where a warp is in its share of the CTA's K blocks. A segment is a run of blocks of one matrix within
// one unit.
struct Walk {
  int u;      // unit
  int rest;   // blocks of the share behind this segment
  int n;      // blocks of the segment from here on (0 past the share's end)
  int ent;    // the matrix: entry of the hit list (from its length on: of the shared expert)
  int tile;   // the unit's 16-row tile of the matrix
  int kb;     // block of the matrix where the segment begins
};

// Scratch bytes of build_hits: a word per expert, the chunks' totals, the batch's ids and weights.
constexpr int hit_scratch(int slots) { return (kMaxExperts + 32 + 2 * slots) * 4; }

// Every thread of the CTA: the hit list of the batch. Integers only, and weights added in slot order.
__device__ __forceinline__ void build_hits(const MvArgs& a, Hits* hits, uint32_t* scratch) {
  uint32_t* emask = scratch;  // tokens by expert; later | index of the expert's first entry << 16
  int* chunk = reinterpret_cast<int*>(scratch + kMaxExperts);  // entries | pairs << 16, of 32 experts
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.T * a.k, s = threadIdx.x;
  int* ids = chunk + 32;
  float* w = reinterpret_cast<float*>(ids + S);
  static_assert(kMvThreads >= kMvMaxSlots && kMvWarps * 64 >= kMaxExperts, "a thread per slot, two chunks a warp");
  int e = -1;
  if (s < S) {
    e = __ldcg(a.ids + s);
    w[s] = __ldcg(a.topk_w + s);
    ids[s] = e;
  }
  for (int i = threadIdx.x; i < a.E; i += kMvThreads) emask[i] = 0;
  __syncthreads();
  const bool in = e >= 0 && e < a.E;
  const int t = s / a.k;
  if (in) atomicOr(&emask[e], 1u << t);
  __syncthreads();
  // chunks of 32 experts: warp w's are w and w + 16
  const int chunks = (a.E + 31) >> 5;
  uint32_t m[2];
  int sum[2], own[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = (warp + kMvWarps * i) * 32 + lane;
    m[i] = x < a.E ? emask[x] : 0;
    if (a.capacity > 0)
      while (__popc(m[i]) > a.capacity) m[i] &= ~(0x80000000u >> __clz(m[i]));  // the highest token is dropped
    const int n = __popc(m[i]);
    own[i] = (n + 7) / 8 | n << 16;
    sum[i] = own[i];  // inclusive scan
    if (__ballot_sync(0xffffffffu, n > 0)) {
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, sum[i], o);
        if (lane >= o) sum[i] += v;
      }
    }
    if (lane == 31) chunk[warp + kMvWarps * i] = sum[i];
  }
  __syncthreads();
  int before = lane < chunks ? chunk[lane] : 0;  // both counts at once: neither reaches 2^15
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (threadIdx.x == 31) hits->n = before & 0xffff;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int ch = warp + kMvWarps * i, x = ch * 32 + lane;
    const int base = __shfl_sync(0xffffffffu, before, ch == 0 ? 0 : ch - 1);
    const int at = (ch ? base : 0) + sum[i] - own[i];  // entries and pairs before this expert's
    if (m[i]) {
      uint32_t rest = m[i];
      for (int n = 0; n < (own[i] & 0xffff); ++n) {
        uint32_t part = rest;  // its lowest 8 tokens
        while (__popc(part) > 8) part &= ~(0x80000000u >> __clz(part));
        rest &= ~part;
        hits->expert[(at & 0xffff) + n] = (uint16_t)x;
        hits->mask[(at & 0xffff) + n] = (uint16_t)part;
        hits->first[(at & 0xffff) + n] = (uint16_t)((at >> 16) + 8 * n);
      }
    }
    if (x < a.E) emask[x] = m[i] ? m[i] | (uint32_t)(at & 0xffff) << 16 : 0;
  }
  __syncthreads();
  if (in) {
    const uint32_t v = emask[e], mask = v & 0xffffu;
    float weight = 0.f;
    bool first = mask >> t & 1;
    for (int j = t * a.k; j < (t + 1) * a.k; ++j)
      if (ids[j] == e) {
        if (j < s) first = false;
        weight += w[j];
      }
    if (first) {
      const int pair = hits->first[v >> 16] + __popc(mask & ((1u << t) - 1));
      hits->weight[pair] = weight;
      hits->token[pair] = (uint8_t)t;
    }
  }
  __syncthreads();
}

// What lanes without a token read in place of its activations.
__device__ const uint4 kMvZeros[16] = {};

// A sum's place in a warp's partial sums: 16 rows to a token, rotated so that the four tokens that a
// quarter warp writes at once fall into different banks.
__device__ __forceinline__ int red_at(int col, int row) { return col * kMvRows + ((row + 4 * (col >> 1)) & 15); }

}  // namespace

template <bool kDual, int kKind, int kNT, int kGroup, bool kZeros>
__global__ void __launch_bounds__(kMvThreads, 1) mv_kernel(const __grid_constant__ MvArgs a) {
  using C = Mv<kDual, kKind, kNT, kGroup, kZeros>;
  constexpr bool kW4 = C::kW4;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = lane >> 2, c = lane & 3;
  float* red = reinterpret_cast<float*>(smem + C::kRingTotal);
  Hits* hits = reinterpret_cast<Hits*>(smem + C::kRingTotal + kMvWarps * C::kRed * sizeof(float));
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * C::kStage * C::kDepth) + (uint32_t)lane * 16;
  const uint8_t* ring_p = smem + (size_t)warp * C::kStage * C::kDepth;

  if (kKind != kMvOne && !a.early) griddep_wait();  // the ids; one matrix: before its first copy
  int nhit = 1;
  if constexpr (kKind != kMvOne) {
    build_hits(a, hits, reinterpret_cast<uint32_t*>(red));  // the sums' buffer is free until the first unit
    constexpr int kSlots = kKind == kMvUp ? kMvMaxSlots : kNT * 8 * kMaxTopK;
    static_assert(kMvWarps * C::kRed * 4 >= hit_scratch(kSlots), "its scratch memory fits");
    nhit = hits->n;
  }

  const int tiles = ceil_div(a.m.R, kMvRows), nb = ceil_div(a.m.K, C::kCols);
  const int stiles = ceil_div(a.shared.R, kMvRows), snb = ceil_div(a.shared.K, C::kCols);
  const int shared = kKind != kMvOne && a.shared.R > 0 ? (a.T + 7) / 8 : 0;  // entries of the shared expert: nhit ...
  const int routed = kKind == kMvUp ? nhit * tiles : tiles;                  // units of the routed experts
  const int units = kKind == kMvUp ? routed + shared * stiles : tiles;

  // This CTA's units, its K blocks one after another (each unit has as many), and this warp's even
  // share of them: whole units, but for the first and the last.
  const int each = units / (int)gridDim.x, more = units - each * (int)gridDim.x;
  const int u0 = blockIdx.x * each + min((int)blockIdx.x, more);
  const int mine = each + ((int)blockIdx.x < more ? 1 : 0);
  const int len = kKind == kMvDown ? nhit * nb + shared * snb : nb;
  const int total = mine * len;
  auto share = [&](int w) { return (int)((uint32_t)(w * total) / kMvWarps); };  // where warp w's begins

  auto locate = [&](int u, int& ent, int& tile) {  // a unit's matrix (kMvDown: the first) and tile
    ent = 0;
    tile = u;
    if constexpr (kKind == kMvUp) {
      const bool sh = u >= routed;
      const int v = sh ? u - routed : u, n = v / (sh ? stiles : tiles);
      ent = sh ? nhit + n : n;
      tile = v - n * (sh ? stiles : tiles);
    }
  };
  auto set_segment = [&](Walk& p, int left) {  // p.u, p.ent and p.kb are set; `left` blocks of the share
    const int seg = (kKind != kMvOne && p.ent >= nhit ? snb : nb) - p.kb;
    p.n = min(left, seg);
    p.rest = left - p.n;
  };
  auto next_segment = [&](Walk& p) {
    if (p.rest == 0) {
      p.n = 0;
      return;
    }
    p.kb = 0;
    if (kKind == kMvDown && p.ent + 1 < nhit + shared) {
      ++p.ent;
    } else {
      ++p.u;
      ++p.tile;
      if constexpr (kKind == kMvDown) p.ent = 0;
      if (kKind == kMvUp && p.tile == (p.ent >= nhit ? stiles : tiles)) {
        ++p.ent;
        p.tile = 0;
      }
    }
    set_segment(p, p.rest);
  };

  // ---- weights: this lane's pieces of a block, from running addresses ----
  Walk prod{};
  const int first = share(warp);
  if (first < share(warp + 1)) {
    const int i = first / len, b = first - i * len;
    prod.u = u0 + i;
    locate(prod.u, prod.ent, prod.tile);
    prod.kb = b;
    if constexpr (kKind == kMvDown) {
      const bool sh = b >= nhit * nb;
      const int v = sh ? b - nhit * nb : b, n = v / (sh ? snb : nb);
      prod.ent = sh ? nhit + n : n;
      prod.kb = v - n * (sh ? snb : nb);
    }
    set_segment(prod, share(warp + 1) - first);
  }
  const uint8_t* wp[C::kMats];   // 4-bit: codes; bf16: row q
  const uint8_t* sp[C::kMats];   // 4-bit: scales; bf16: row q + 8
  bool in0 = true, in1 = true;   // bf16: rows q and q + 8 exist
  int wcols = 0;                 // bf16: columns from this lane's first one to the end of the matrix
  auto aim_weights = [&]() {
    if (prod.n == 0) return;
    const bool sh = kKind != kMvOne && prod.ent >= nhit;
    const MvMatrix& m = sh ? a.shared : a.m;
    const int e = kKind == kMvOne || sh ? 0 : hits->expert[prod.ent];
    const int tile = prod.tile;
#pragma unroll
    for (int i = 0; i < C::kMats; ++i) {
      if constexpr (kW4) {
        const int64_t at = ((int64_t)e * (sh ? stiles : tiles) + tile) * (sh ? snb : nb) + prod.kb;
        wp[i] = static_cast<const uint8_t*>(m.w[i]) + at * C::kCodes + lane * 16;
        sp[i] = static_cast<const uint8_t*>(m.scales[i]) + at * (8 * C::kMeta) + lane * 16;
      } else {
        const int row = tile * kMvRows + q;
        in0 = row < m.R;
        in1 = row + 8 < m.R;
        const uint16_t* w = static_cast<const uint16_t*>(m.w[i]);
        const int64_t col = prod.kb * C::kCols + 8 * c;
        wp[i] = reinterpret_cast<const uint8_t*>(w + (in0 ? (int64_t)row * m.K : 0) + col);
        sp[i] = reinterpret_cast<const uint8_t*>(w + (in1 ? (int64_t)(row + 8) * m.K : 0) + col);
        wcols = m.K - (int)col;
      }
    }
  };
  auto copy_block = [&](uint32_t slot_off) {
    const uint32_t dst = ring + slot_off;
#pragma unroll
    for (int i = 0; i < C::kMats; ++i) {
      if constexpr (kW4) {
        cp_async16(dst + i * C::kMat, wp[i]);
        cp_async16(dst + i * C::kMat + 512, wp[i] + 512);
        if (lane < C::kMeta / 2) cp_async16(dst + i * C::kMat + 1024, sp[i]);  // 8 * kMeta bytes
        wp[i] += C::kCodes;
        sp[i] += 8 * C::kMeta;
      } else {
        // a piece outside the matrix is zeros; K is a multiple of 8, so that pieces are whole
        const bool k0 = wcols > 0, k1 = wcols > 32;
        const void* any = a.m.w[i];
        cp_async16_or_zeros(dst + (i * 4 + 0) * 512, k0 ? wp[i] : any, in0 && k0);
        cp_async16_or_zeros(dst + (i * 4 + 1) * 512, k1 ? wp[i] + 64 : any, in0 && k1);
        cp_async16_or_zeros(dst + (i * 4 + 2) * 512, k0 ? sp[i] : any, in1 && k0);
        cp_async16_or_zeros(dst + (i * 4 + 3) * 512, k1 ? sp[i] + 64 : any, in1 && k1);
        wp[i] += 2 * C::kCols;
        sp[i] += 2 * C::kCols;
      }
    }
    if constexpr (!kW4) wcols -= C::kCols;
  };
  auto copy = [&](uint32_t slot_off) {
    copy_block(slot_off);
    if (--prod.n == 0) {
      next_segment(prod);
      aim_weights();
    }
  };

  // ---- activations: this lane's columns of a block for its tokens ----
  // An entry's tokens, one after another, are the MMA's columns.
  Walk nxt{};
  const uint16_t* xp[C::kXT];    // zeros where the lane has no token of this expert
  int xstep[C::kXT];              // elements to the next block (0: zeros)
  int xk = 0;                    // columns from this lane's first one to the end
  int whole = 0;                 // blocks of the matrix from here on with all their columns
  auto tokens_of = [&](int ent) -> uint32_t {
    const uint32_t all = (1u << a.T) - 1;
    if (kKind == kMvOne) return all;
    return ent >= nhit ? all & 0xffu << 8 * (ent - nhit) : hits->mask[ent];
  };
  auto aim_x = [&]() {
    if (nxt.n == 0) return;
    const bool sh = kKind != kMvOne && nxt.ent >= nhit;
    const int K = sh ? a.shared.K : a.m.K;
    const int count = __popc(tokens_of(nxt.ent));
    // the entry's first token (the one matrix, the shared expert) or pair
    const int first = kKind == kMvOne ? 0 : (sh ? 8 * (nxt.ent - nhit) : hits->first[nxt.ent]);
    const int col = nxt.kb * C::kCols + 8 * c;
    xk = K - col;
    whole = K / C::kCols - nxt.kb;
#pragma unroll
    for (int n = 0; n < C::kXT; ++n) {
      const int i = q + 8 * n;
      const bool in = i < count;
      int64_t row = first + i;
      if constexpr (kKind == kMvDown) row += sh ? a.T * a.k : 0;  // h's rows
      else if (kKind == kMvUp && !sh) row = in ? hits->token[first + i] : 0;
      xp[n] = in ? a.x + row * a.ldx + col : reinterpret_cast<const uint16_t*>(kMvZeros);
      xstep[n] = in ? C::kCols : 0;
    }
  };
  auto load_x = [&](uint4 (&x)[C::kXT][C::kVecs], int h) {  // half h of the block that nxt is at
    if (nxt.n == 0) return;
    // plain loads: the warps of an SM share the rows through L1
    if (whole > 0) {
#pragma unroll
      for (int n = 0; n < C::kXT; ++n) {
#pragma unroll
        for (int v = 0; v < C::kVecs; ++v)
          x[n][v] = *reinterpret_cast<const uint4*>(xp[n] + 32 * (C::kVecs * h + v));
      }
    } else {
#pragma unroll
      for (int n = 0; n < C::kXT; ++n)
#pragma unroll
        for (int v = 0; v < C::kVecs; ++v)
          x[n][v] = xk > 32 * (C::kVecs * h + v) ? *reinterpret_cast<const uint4*>(xp[n] + 32 * (C::kVecs * h + v))
                                                 : make_uint4(0, 0, 0, 0);
    }
  };
  auto advance_x = [&]() {
    if (nxt.n == 0) return;
#pragma unroll
    for (int n = 0; n < C::kXT; ++n) xp[n] += xstep[n];
    xk -= C::kCols;
    --whole;
    if (--nxt.n == 0) {
      next_segment(nxt);
      aim_x();
    }
  };

  Walk cur = prod;
  nxt = prod;
  aim_weights();
  if (kKind == kMvOne && !a.early) griddep_wait();
  uint32_t slot = 0, vacant = 0;  // byte offsets in the ring: the block in use, the one used before it
#pragma unroll 1
  for (int i = 0; i < C::kDepth - 1; ++i) {
    if (prod.n) copy(vacant);
    cp_async_commit();
    vacant += C::kStage;
  }
  if (a.early) griddep_wait();
  griddep_launch_dependents();

  float acc[C::kMats][C::kXT][4];   // of the current matrix
  float tot[kNT][4];             // kMvDown: router-weighted, over the experts so far
  uint4 xa[C::kXT][C::kVecs], xb[C::kXT][C::kVecs];  // halves of a block: first, second
  // Half h of a block's products; 4-bit: one half holds kParts / 2 groups, or half of the one. Calls
  // reload(n, v) behind the last use of x[n][v] (4-bit).
  float part[C::kMats][C::kXT][4];  // 4-bit: sums of the current group, not scaled
  auto products = [&](const uint8_t* st, uint4 (&x)[C::kXT][C::kVecs], int h, auto&& reload) {
#pragma unroll
    for (int i = 0; i < C::kMats; ++i) {
      if constexpr (kW4) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(st + i * C::kMat + h * 512 + lane * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        constexpr int kHere = C::kParts >= 2 ? C::kParts / 2 : 1;  // groups of this half
        constexpr int kWords = 4 / kHere;
        const uint8_t* meta = st + i * C::kMat + 1024 + q * C::kMeta + (C::kParts >= 2 ? h * (C::kMeta / 2) : 0);
        constexpr int kMetaWords = kHere * (kZeros ? 2 : 1);
        uint32_t mv[kMetaWords];
        if constexpr (kMetaWords == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(meta);
          mv[0] = v.x; mv[1] = v.y; mv[2] = v.z; mv[3] = v.w;
        } else if constexpr (kMetaWords == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(meta);
          mv[0] = v.x; mv[1] = v.y;
        } else {
          mv[0] = *reinterpret_cast<const uint32_t*>(meta);
        }
#pragma unroll
        for (int g = 0; g < kHere; ++g) {
          float s0, s1;                            // rows q and q + 8
          uint32_t z0 = 0x43084308u, z1 = z0;      // bf16x2 of 128 + zero
          if constexpr (kZeros) {
            s0 = __uint_as_float(mv[2 * g] << 16);
            s1 = __uint_as_float(mv[2 * g + 1] << 16);
            z0 = __byte_perm(mv[2 * g], 0, 0x3232);
            z1 = __byte_perm(mv[2 * g + 1], 0, 0x3232);
          } else {
            s0 = __uint_as_float(mv[g] << 16);
            s1 = __uint_as_float(mv[g] & 0xffff0000u);
          }
          uint32_t f[kWords][4];
#pragma unroll
          for (int jj = 0; jj < kWords; ++jj)
#pragma unroll
            for (int n = 0; n < 4; ++n)
              f[jj][n] = sub_bf16x2(((w[g * kWords + jj] >> (4 * n)) & 0x000f000fu) | 0x43004300u, (n & 1) ? z1 : z0);
#pragma unroll
          for (int n = 0; n < C::kXT; ++n) {
            float(&p)[4] = part[i][n];
#pragma unroll
            for (int jj = 0; jj < kWords; ++jj) {
              const int j = g * kWords + jj;
              const uint4 v = x[n][j >> 1];
              if (jj == 0 && (C::kParts >= 2 || h == 0)) mma_bf16_zero(p, f[jj], v.x, v.y);
              else if (j & 1) mma_bf16(p, f[jj], v.z, v.w);
              else mma_bf16(p, f[jj], v.x, v.y);
            }
            if (i == C::kMats - 1) {
#pragma unroll
              for (int j = g * kWords + 1; j < (g + 1) * kWords; j += 2) reload(n, j >> 1);
            }
            if (C::kParts >= 2 || h == 1) {
              acc[i][n][0] += s0 * p[0];
              acc[i][n][1] += s0 * p[1];
              acc[i][n][2] += s1 * p[2];
              acc[i][n][3] += s1 * p[3];
            }
          }
        }
      } else {
        // rows q and q + 8 of this half
        const uint4 lo = *reinterpret_cast<const uint4*>(st + (i * 4 + h) * 512 + lane * 16);
        const uint4 hi = *reinterpret_cast<const uint4*>(st + (i * 4 + 2 + h) * 512 + lane * 16);
        const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
        for (int n = 0; n < C::kXT; ++n) {
          mma_bf16(acc[i][n], f0, x[n][0].x, x[n][0].y);
          mma_bf16(acc[i][n], f1, x[n][0].z, x[n][0].w);
        }
      }
    }
  };
  // One block: the copy of a later one, activations ahead, and its products. The lanes
  // share a block's scales, so that the copy into the slot of the block before waits for them all.
  auto turn = [&]() {
    const uint32_t at = slot;
    vacant = slot;
    slot += C::kStage;
    if (slot == C::kStage * C::kDepth) slot = 0;
    return ring_p + at;
  };
  auto keep = [](int, int) {};
  auto block = [&]() {
    if constexpr (!kW4) load_x(xb, 1);
    cp_async_wait<C::kDepth - 2>();
    __syncwarp();
    if (prod.n) copy(vacant);
    cp_async_commit();
    const uint8_t* st = turn();
    products(st, xa, 0, keep);
    advance_x();
    load_x(xa, 0);
    products(st, xb, 1, keep);
    if constexpr (kW4) load_x(xb, 1);
  };
  // The same for `t` blocks at which no segment ends (neither this one nor that of the copies) and
  // whose following block is whole: nothing is asked in this loop.
  auto run = [&](int t) {
    prod.n -= t;
    nxt.n -= t;
    whole -= t;
    xk -= t * C::kCols;
#pragma unroll 1
    for (; t > 0; --t) {
      auto load_b = [&](int n, int v) { xb[n][v] = *reinterpret_cast<const uint4*>(xp[n] + 32 * (C::kVecs + v)); };
      auto load_a = [&](int n, int v) { xa[n][v] = *reinterpret_cast<const uint4*>(xp[n] + 32 * v); };
      if constexpr (kW4) {
#pragma unroll
        for (int n = 0; n < C::kXT; ++n) xp[n] += xstep[n];
      } else {
#pragma unroll
        for (int n = 0; n < C::kXT; ++n) load_b(n, 0);
      }
      cp_async_wait<C::kDepth - 2>();
      __syncwarp();
      copy_block(vacant);
      cp_async_commit();
      const uint8_t* st = turn();
      // 4-bit: every vector of activations is loaded again as soon as it is used, three quarters of a block ahead
      // (experts, 8 tokens of 7168 x 2048: 183 -> 179 us, since h comes from L2). bf16, whose block is one
      // vector a half, is faster with the loads in two bunches (16 tokens: 21.5 us instead of 22.2).
      if constexpr (kW4) {
        products(st, xa, 0, load_a);
        products(st, xb, 1, load_b);
      } else {
        products(st, xa, 0, keep);
#pragma unroll
        for (int n = 0; n < C::kXT; ++n) {
          xp[n] += xstep[n];
          load_a(n, 0);
        }
        products(st, xb, 1, keep);
      }
    }
  };

  aim_x();
  load_x(xa, 0);
  if constexpr (kW4) load_x(xb, 1);
  // Where a unit's results go: column or token t's row is row0 + t, for t < count; output rows below R.
  struct Place {
    int64_t row0;
    int count, col0, R;
  };
  auto place = [&](int ent, int tile) {
    Place p{0, a.T, tile * kMvRows, a.m.R};
    if constexpr (kKind == kMvUp) {
      if (ent >= nhit) {
        p.R = a.shared.R;
        p.row0 = a.T * a.k + 8 * (ent - nhit);
        p.count = a.T - 8 * (ent - nhit);
      } else {
        p.row0 = hits->first[ent];
        p.count = __popc((uint32_t)hits->mask[ent]);
      }
    }
    return p;
  };
  auto emit = [&](const Place& p, int t, int r, float s0, float s1) {
    const int col = p.col0 + r;
    if (t >= p.count || col >= p.R) return;
    const int64_t at = (p.row0 + t) * a.ldo + col;
    float v = s0;
    if constexpr (kDual) {
      v = swiglu(s0, s1);
      if (kKind == kMvOne && a.u) {
        a.u[at] = (uint16_t)(pack_bf16x2(s0, 0.f) & 0xffffu);
        a.g[at] = (uint16_t)(pack_bf16x2(s1, 0.f) & 0xffffu);
      }
    }
    if (a.out_bf16) static_cast<uint16_t*>(a.out)[at] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
    else static_cast<float*>(a.out)[at] = v;
  };
  auto clear = [&]() {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
#pragma unroll
      for (int n = 0; n < C::kXT; ++n)
#pragma unroll
        for (int i = 0; i < C::kMats; ++i) acc[i][n][v] = 0.f;
#pragma unroll
      for (int n = 0; n < kNT; ++n) tot[n][v] = 0.f;
    }
  };
  // Calls f(token or column, row, sum, second matrix's sum) for this lane's sums of the unit.
  auto each_sum = [&](auto&& f) {
#pragma unroll
    for (int n = 0; n < C::kTok / 8; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if constexpr (kKind == kMvDown) f(8 * n + 2 * c + (v & 1), q + 8 * (v >> 1), tot[n][v], 0.f);
        else f(8 * n + 2 * c + (v & 1), q + 8 * (v >> 1), acc[0][n][v], acc[C::kMats - 1][n][v]);
      }
  };
  auto put = [&](float* dst) {
    each_sum([&](int t, int r, float s0, float s1) {
      dst[red_at(t, r)] = s0;
      if constexpr (kDual) dst[C::kTok * kMvRows + red_at(t, r)] = s1;
    });
  };

  // Units that this warp computes whole go straight to memory. Of a unit that begins in another
  // warp's share the sums go to `red`; those of one that ends in another's stay in registers until
  // every warp is done with the ring, and go there.
  const bool one = mine == 1;  // a single unit: every warp's sums go to `red`, zeros too
  bool open = false;           // the registers hold the beginning of a unit that another warp ends
  bool mid = one || first % max(len, 1) != 0;
  clear();
  if (one && cur.n == 0) put(red + warp * C::kRed);
#pragma unroll 1
  while (cur.n) {
    const uint32_t members = tokens_of(cur.ent);
#pragma unroll 1
    for (int n = cur.n; n > 0;) {
      const int t = min(min(n, whole), prod.n) - 1;
      if (t > 0) {
        run(t);
        n -= t;
      }
      block();
      --n;
    }
    const int ent = cur.ent, tile = cur.tile, u = cur.u;
    next_segment(cur);
    if constexpr (kKind == kMvDown) {
      // the router weights of the matrix that ends here; its columns go to their tokens' places
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          const int t = 8 * n + 2 * c + t2, i = __popc(members & ((1u << t) - 1));
          const int from = (lane & ~3) | ((i & 7) >> 1);
          float y[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float v0 = __shfl_sync(0xffffffffu, acc[0][0][2 * r], from);
            const float v1 = __shfl_sync(0xffffffffu, acc[0][0][2 * r + 1], from);
            y[r] = i & 1 ? v1 : v0;
          }
          if (members >> t & 1) {
            const float w = ent >= nhit ? 1.f : hits->weight[hits->first[ent] + i];
            tot[n][t2] += w * y[0];
            tot[n][2 + t2] += w * y[1];
          }
        }
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[0][0][v] = 0.f;
    }
    if (cur.n && cur.u == u) continue;
    const bool ended = cur.n || share(warp + 1) == (u - u0 + 1) * len;
    if (mid) {
      put(red + warp * C::kRed);
      clear();
    } else if (ended) {
      const Place p = place(ent, tile);
      each_sum([&](int t, int r, float s0, float s1) { emit(p, t, r, s0, s1); });
      clear();
    } else {
      open = true;
    }
    mid = false;
  }
  cp_async_wait<0>();
  if (kKind == kMvDown && len == 0) {  // no expert was hit: zeros
    const int n = mine * kMvRows * a.T;
    for (int o = threadIdx.x; o < n; o += kMvThreads)
      emit(place(0, u0 + o / (kMvRows * a.T)), o / kMvRows % a.T, o % kMvRows, 0.f, 0.f);
    return;
  }
  __syncthreads();
  constexpr int kOuts = kMvRows * C::kTok;
  if (one) {
    const int o = threadIdx.x, r = o % kMvRows, t = o / kMvRows;
    if (o < kOuts) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
      for (int w = 0; w < kMvWarps; ++w) {
        const float* src = red + w * C::kRed + red_at(t, r);
        s0 += src[0];
        if constexpr (kDual) s1 += src[C::kTok * kMvRows];
      }
      int ent, tile;
      locate(u0, ent, tile);
      emit(place(ent, tile), t, r, s0, s1);
    }
    return;
  }
  float* red1 = reinterpret_cast<float*>(smem);
  static_assert(C::kRingTotal >= kMvWarps * C::kRed * 4, "the ring is large enough");
  if (open) put(red1 + warp * C::kRed);
  __syncthreads();
  // Units that are spread over warps, a thread to an output. Lane w looks at share w: a unit is spread
  // where a share is the first to begin inside it. Its sums are in `red1` of the warp before and in `red`
  // of each warp until its end, and are added in warp order.
  const int mark = lane <= kMvWarps ? share(lane) : INT_MAX;  // where share `lane` begins
  const int before = __shfl_up_sync(0xffffffffu, mark, 1), after = __shfl_down_sync(0xffffffffu, mark, 1);
  const int at = lane > 0 && lane < kMvWarps && mark < total ? mark / len : -1;
  const uint32_t firsts = __ballot_sync(0xffffffffu, at >= 0 && mark > at * len && before <= at * len);
  for (int item = threadIdx.x; item < __popc(firsts) * kOuts; item += kMvThreads) {  // whole warps
    uint32_t m = firsts;
    for (int j = item / kOuts; j > 0; --j) m &= m - 1;
    const int w = __ffs(m) - 1, i = __shfl_sync(0xffffffffu, at, w);
    uint32_t spread = __ballot_sync(0xffffffffu, lane >= w && lane < kMvWarps && mark < (i + 1) * len && mark != after);
    const int o = item % kOuts, r = o % kMvRows, t = o / kMvRows;
    const float* src = red1 + (w - 1) * C::kRed + red_at(t, r);
    float s0 = src[0], s1 = 0.f;
    if constexpr (kDual) s1 = src[C::kTok * kMvRows];
    src = red + red_at(t, r);
    for (; spread; spread &= spread - 1) {
      const float* k = src + (__ffs(spread) - 1) * C::kRed;
      s0 += k[0];
      if constexpr (kDual) s1 += k[C::kTok * kMvRows];
    }
    int ent, tile;
    locate(u0 + i, ent, tile);
    emit(place(ent, tile), t, r, s0, s1);
  }
}

namespace {

template <bool kDual, int kKind, int kNT, int kGroup, bool kZeros>
cudaError_t launch_mv(const MvArgs& a, int64_t units, int num_sms, cudaStream_t stream) {
  using C = Mv<kDual, kKind, kNT, kGroup, kZeros>;
  auto* k = mv_kernel<kDual, kKind, kNT, kGroup, kZeros>;
  // the kernel's shared-memory limit and share are set at its first launch on a device; should the device
  // have been reset since, the launch is refused once and repeated
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(units, num_sms));
  for (int attempt = 0;; ++attempt) {
    if (attempt > 0 || !(raised.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, C::kCarveout);
      if (e != cudaSuccess) return e;
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
    e = launch_k(k, dim3(grid), dim3(kMvThreads), C::kSmem, stream, a);
    if (e != cudaErrorInvalidValue || attempt > 0) return e;
    cudaGetLastError();
  }
}

template <bool kDual, int kKind, int kGroup, bool kZeros>
cudaError_t pick_nt(const MvArgs& a, int64_t units, int num_sms, cudaStream_t stream) {
  if constexpr (kKind != kMvUp)
    if (a.T > 8) return launch_mv<kDual, kKind, 2, kGroup, kZeros>(a, units, num_sms, stream);
  return launch_mv<kDual, kKind, 1, kGroup, kZeros>(a, units, num_sms, stream);
}

template <bool kDual, int kKind, bool kZeros>
cudaError_t pick_group(const MvArgs& a, int64_t units, int num_sms, cudaStream_t stream) {
  if (a.group == 32) return pick_nt<kDual, kKind, 32, kZeros>(a, units, num_sms, stream);
  if (a.group == 64) return pick_nt<kDual, kKind, 64, kZeros>(a, units, num_sms, stream);
  return pick_nt<kDual, kKind, 128, kZeros>(a, units, num_sms, stream);
}

template <bool kDual, int kKind>
cudaError_t pick_int4(const MvArgs& a, bool zeros, int64_t units, int num_sms, cudaStream_t stream) {
  return zeros ? pick_group<kDual, kKind, true>(a, units, num_sms, stream)
               : pick_group<kDual, kKind, false>(a, units, num_sms, stream);
}

// ---- laying out 4-bit matrices ----------------------------------------------------------------
// One warp per block of 16 rows x 128 columns: lane 4 q + c holds its pieces of both halves, 64 values
// of rows q and q + 8 as v[half][h][row][column]. Writes the codes' words.
__device__ __forceinline__ void store_codes(uint8_t* codes, int64_t block, const uint8_t (&v)[2][2][2][8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
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
    *reinterpret_cast<uint4*>(codes + block * 1024 + b * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ void store_scale(uint8_t* scales, int64_t tile, int blocks, int group, int g, int row, bool zeros,
                                            uint32_t s, uint32_t zero) {
  const int64_t o = tile * blocks * (kInt4Cols / group) * kMvRows + int4_scale_at(row, g, group);
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
  const int nb = (int)int4_blocks(K);
  const int64_t items = int4_row_tiles(R) * nb;
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * 8) {
    const int64_t tile = it / nb;
    const int k0 = (int)(it % nb) * kInt4Cols;
    float f[2][2][2][8];
    float lo[4][2], hi[4][2];  // per 32 columns and row
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = tile * kMvRows + q + 8 * r;
        const int k = k0 + 32 * p + 8 * c;
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
        const int g = (k0 + 32 * p) / group;
        if (p == first && c == 0) store_scale(scales, tile, nb, group, g, q + 8 * r, kZeros, sb, (uint32_t)zero);
      }
    store_codes(codes, it, v);
  }
}

__global__ void __launch_bounds__(256) int4_pack_kernel(const uint8_t* __restrict__ src, const uint16_t* __restrict__ s,
                                                        const uint8_t* __restrict__ z, int64_t R, int K, int group,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, q = lane >> 2, c = lane & 3;
  const int nb = (int)int4_blocks(K), G = (K + group - 1) / group;
  const int64_t items = int4_row_tiles(R) * nb;
  for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < items; it += (int64_t)gridDim.x * 8) {
    const int64_t tile = it / nb;
    const int k0 = (int)(it % nb) * kInt4Cols;
    uint8_t v[2][2][2][8];
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = tile * kMvRows + q + 8 * r;
        const int k = k0 + 32 * p + 8 * c;
        uint32_t x = 0;
        if (row < R && k < K) x = __ldg(reinterpret_cast<const uint32_t*>(src + row * (K / 2) + k / 2));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p >> 1][p & 1][r][i] = (uint8_t)(x >> (4 * i) & 15u);
        const int g = (k0 + 32 * p) / group;
        if ((k0 + 32 * p) % group == 0 && c == 0) {
          const bool in = row < R && g < G;
          store_scale(scales, tile, nb, group, g, q + 8 * r, z != nullptr, in ? __ldg(s + row * G + g) : 0u,
                      in && z ? __ldg(z + row * G + g) : 8u);
        }
      }
    store_codes(codes, it, v);
  }
}

int layout_grid(int64_t R, int64_t K, int num_sms) {
  const int64_t items = int4_row_tiles(R) * int4_blocks(K);
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
  return dual ? pick_nt<true, kMvOne, 0, false>(a, units, num_sms, stream)
              : pick_nt<false, kMvOne, 0, false>(a, units, num_sms, stream);
}

cudaError_t launch_mv_int4(const MvArgs& a, int kind, bool zeros, int num_sms, cudaStream_t stream) {
  const int64_t tiles = ceil_div(a.m.R, kMvRows);
  if (kind == kMvOne) return pick_int4<false, kMvOne>(a, zeros, tiles, num_sms, stream);
  if (kind == kMvDown) return pick_int4<false, kMvDown>(a, zeros, tiles, num_sms, stream);
  // at most an entry per slot
  const int64_t units = tiles * a.T * a.k + 2 * ceil_div(a.shared.R, kMvRows);
  return pick_int4<true, kMvUp>(a, zeros, units, num_sms, stream);
}

}  // namespace moe
