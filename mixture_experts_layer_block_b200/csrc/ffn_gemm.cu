// ffn_gemm.cu -- the matrix products of the gated feed-forward block and of its backward pass
// (ffn.cuh gives the formulas) as one persistent GEMM on pairs of SMs.
//
// What bounds it: at training sizes the tensor cores; at a few hundred tokens the start and end of its
// launches and the pace of the threads that issue TMA and MMA.
// Each output tile of up to 256 x bn (bn <= 256) belongs to a cluster of two CTAs: one
// tcgen05.mma.cta_group::2 (M = 256) per 16-wide K step, issued by CTA 0, with up to 128 rows of A
// and bn / 2 rows of B staged by each CTA. A pair moves 32 KB per SM and 64-wide K step where a
// 128 x 256 tile on one SM needs 48 KB for the same work. Two accumulators fill the tensor memory,
// so that the epilogue of one tile runs under the products of the next.
//
// Operands come as they lie in memory. A K-major operand is one TMA box of {64 k, rows}; an
// MN-major one (the weights of the backward products, and both operands of the weight gradients)
// is boxes of {64 m or n, 64 k}, which the MMA reads through an MN-major descriptor: no transposed
// copy is ever made. Everything past an edge is filled with zeros by TMA on both operands (the MMA's rows past
// a tile's own hold leftovers of the ring, each of which makes a row of its own), and clipped on the way out.
//
// The units (tile, K split) of up to four products form one list (the four gradients that depend
// on du, dg and h run as one launch), dealt round robin to the pairs: with equal units per
// product this is as even as a shared counter and needs no state in memory. With fewer tiles than pairs
// K is split; the partial sums go to a workspace in fp32 and ffn_reduce_kernel adds them in split
// order, so that results do not depend on timing.
//
// Warp roles per CTA: warps 0 and 6 TMA producers (A and B), warp 1 MMA issuer (CTA 0), warps 2-5
// epilogue, warp 7 (dh only) the epilogue's loads of u and g and its stores: with 16-byte loads by
// the epilogue's own threads, each of another row, a tile's epilogue took 25,000 clocks and slowed
// the products beside it by a third.
// Every TMA and MMA loop runs in one elected lane: under a test of the lane's number the compiler
// looped over the active lanes around each of these instructions (135 clocks a TMA instruction, 400 for
// four MMAs and a commit; now 50 and 100).
//
// Measured (one B200, T = 4096, H = 7168, D = 2048): u | g 177 us (1360 TFLOP/s), the four gradients 410 us
// (1465 TFLOP/s), dh 100 us alone (1200 TFLOP/s; 128 tiles are 1.7 rounds of 74 pairs); cuBLAS does one of
// these products at 1320-1480 TFLOP/s. Back to back, power holds both near 1300-1380. A pair's 32 KB per SM and
// K block need 64 bytes a clock from L2 at full rate, which is about all that an SM takes. 333 tokens of 2048 x
// 2048: 20.8 us for both launches, 32 K blocks each at 250-330 clocks.
#include <algorithm>

#include "ffn.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int kFThreads = 256;
constexpr int kFMaxStages = 20;
constexpr int kFBoxBytes = 64 * 64 * 2;  // an MN-major box of 64 x 64
constexpr int kFChunk = 32;              // columns per epilogue step
constexpr int kFBarBytes = 512;
constexpr int kFSmem = 227 * 1024 - 1024;  // less the alignment slack
// Epilogue buffers: two chunks of one result (16 KB each, fp32), of three (h, u, g: 24 KB), or (dh)
// two chunks of u and g (16 KB) and one of du, dg and h (24 KB).
__host__ __device__ constexpr int staging_bytes(int epi) {
  return (epi == kFfnStore ? 32 : (epi == kFfnSwiglu ? 48 : 56)) * 1024;
}
constexpr int kFInBytes = 16384;               // u and g of a chunk (of 128 rows)
constexpr int kFOutOff = 2 * kFInBytes;        // du, dg and h of a chunk
__host__ __device__ constexpr int ring_bytes(int epi) { return kFSmem - staging_bytes(epi) - kFBarBytes; }

// A's bytes per CTA and stage: mrows rows of 128 bytes (a multiple of 8 rows, so that B begins on a 1024-byte
// line), or two 64-wide boxes. The MMA reads 128 rows all the same: what lies past the box makes rows that are
// not stored.
__host__ __device__ inline int a_bytes(const FfnProblem& p) { return p.a_mn ? 2 * kFBoxBytes : p.mrows * kBK * 2; }
// B's bytes per CTA and stage: bn / 2 rows of 128 bytes, or whole 64-wide boxes
__host__ __device__ inline int b_bytes(int bn, int b_mn) {
  return b_mn ? ((bn / 2 + 63) / 64) * kFBoxBytes : (bn / 2) * 128;
}

// Descriptor of an MN-major bf16 operand with the 128-byte swizzle: 64-element rows of 128 bytes
// (m or n contiguous), 8 k to a 1024-byte atom, atoms along k 1024 bytes apart (stride byte
// offset) and along m or n one 64 x 64 box apart (leading byte offset).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(kFBoxBytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// fp32 tile added to global memory by the TMA unit (each element once: the order is fixed).
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, uint32_t src, int32_t c0, int32_t c1) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}

// One lane of a converged warp, chosen by the hardware. Unlike a test of the lane's number this
// tells the compiler that what follows runs in one lane, so that the TMA and MMA instructions,
// whose operands live in the warp's uniform registers, need no loop over the active lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// wait_bar with the first probe inline: most waits find their phase complete.
__device__ __forceinline__ bool wait_bar_fast(uint64_t* bar, uint32_t parity, DeviceMeta* meta, volatile int* s_abort,
                                              int64_t limit, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_bar(bar, parity, meta, s_abort, limit, site);
}

__host__ __device__ inline int most_block_bytes(const FfnParams& P) {
  int most = 0;
  for (int i = 0; i < P.nprob; ++i) {
    const int b = a_bytes(P.p[i]) + b_bytes(P.p[i].bn, P.p[i].b_mn);
    most = most > b ? most : b;
  }
  return (most + 1023) & ~1023;
}

struct Unit {
  int prob, m, n, split;
};

// Unit `id` of the launch: its product, and within it the K split (fastest, so that the splits of a
// tile share its operands' L2 lines in time) and the tile, walked in panels of kFfnRaster m-tiles.
__device__ __forceinline__ Unit find_unit_ffn(const FfnParams& P, int id) {
  Unit t;
  t.prob = 0;
#pragma unroll
  for (int i = 1; i < kFfnMaxProblems; ++i)
    if (i < P.nprob && id >= P.p[i].unit0) t.prob = i;
  const FfnProblem& p = P.p[t.prob];
  id -= p.unit0;
  t.split = 0;
  int tile = id;
  if (p.splits > 1) {
    t.split = id % p.splits;
    tile = id / p.splits;
  }
  // tile / per by the reciprocal rounded up, which is one too many at most (four divisions took 500 clocks of every
  // unit's epilogue, and of every role's start)
  const int per = kFfnRaster * p.nt;
  int panel = (int)__umulhi((uint32_t)tile, p.panel_inv);
  if (panel * per > tile) --panel;
  const int first = panel * kFfnRaster, r = tile - panel * per;
  if (p.mt - first >= kFfnRaster) {
    t.m = first + r % kFfnRaster;
    t.n = r / kFfnRaster;
  } else {
    const int gm = p.mt - first;
    t.m = first + r % gm;
    t.n = r / gm;
  }
  return t;
}

// First column of a tile's chunk `cc`. A width that is no multiple of the chunk's ends in a chunk that
// overlaps the one before it: those columns are stored twice, with the same values.
__device__ __forceinline__ int chunk_col(int cc, int width, int chunk = kFChunk) {
  return min(cc * chunk, width - chunk);
}

__device__ __forceinline__ void split_range(const FfnProblem& p, int split, int& k0, int& k1) {
  const int total = p.nkb * p.nseg;
  k0 = (int)((int64_t)split * total / p.splits);
  k1 = (int)((int64_t)(split + 1) * total / p.splits);
}

}  // namespace

// kPer: 64-wide K blocks of a stage, 1 or 2. A stage's barriers, its commit and the loops around them take about 330
// clocks of the threads that issue, where four MMAs of 128 columns take 256: with two blocks to a stage narrow
// tiles are no longer bound by that (333 tokens of 2048 x 2048: 23.0 -> 21.4 us).
template <int kEpi, int kPer>
__global__ void __launch_bounds__(kFThreads, 1) ffn_gemm_kernel(const __grid_constant__ FfnParams P) {
  constexpr int kStagingTotal = staging_bytes(kEpi);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = smem + (ring_bytes(kEpi) & ~1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStagingTotal);
  uint64_t* empty = full + kFMaxStages;
  uint64_t* acc_full = empty + kFMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* ug_full = acc_empty + 2;   // dh: u and g of a chunk are in its buffer
  uint64_t* ug_free = ug_full + 2;     // dh: every thread has read its row of them
  uint64_t* ready = ug_free + 2;       // dh: du, dg and h of a chunk are in the out buffer
  uint64_t* out_free = ready + 1;      // dh: they have been read
  uint64_t* drain = out_free + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  volatile int* s_go = reinterpret_cast<volatile int*>(s_tmem + 2);           // [2]
  volatile uint32_t* s_nfill = reinterpret_cast<volatile uint32_t*>(s_tmem + 4);  // [4] fills per producer
  volatile uint32_t* s_left = reinterpret_cast<volatile uint32_t*>(s_tmem + 8);   // a role of the pair gave up

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  DeviceMeta* meta = P.meta;
  const int64_t limit = P.timeout_ns;
  // one ring for the whole launch: a block holds the largest product's operands of 64 k
  const int block_bytes = most_block_bytes(P), stage_bytes = kPer * block_bytes;
  const int nst = min(kFMaxStages, (ring_bytes(kEpi) & ~1023) / stage_bytes);

  if (threadIdx.x == 0) {
    for (int i = 0; i < nst; ++i) {
      mbar_init(&full[i], 4);  // one arrival per producer (CTA 0's barrier is the one used)
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);  // 4 epilogue warps x 2 CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ug_full[i], 1);
      mbar_init(&ug_free[i], 128);
    }
    mbar_init(ready, 128);
    mbar_init(out_free, 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    for (int i = 0; i < 4; ++i) s_nfill[i] = 0;
    *s_left = 0;
    fence_mbar_init();
    for (int i = 0; i < P.nprob; ++i) {
      tma_prefetch_desc(&P.p[i].a[0]);
      tma_prefetch_desc(&P.p[i].b[P.p[i].b_by_rank ? rank : 0]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(s_tmem), 2 * kAccCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  // each role waits for the kernel in front (griddep_wait) where it first touches memory: finding its first
  // unit, and fetching the code that does, goes before
  const uint32_t full_c0 = mapa_shared(smem_u32(full), 0);
  const uint32_t acc_empty_c0 = mapa_shared(smem_u32(acc_empty), 0);
  auto give_up = [&]() {  // known to both CTAs behind the teardown's barrier
    for (uint32_t r = 0; r < 2; ++r) st_cluster_u32(mapa_shared(smem_u32((const void*)s_left), r), 1);
  };
  uint32_t nfill = 0;
  bool mma_issued = false;

  if (warp == 0 || warp == 6) {
    // ---------------------------------- producers ----------------------------------
    // Warp 0 loads this CTA's rows of A, warp 6 its rows of B: a stage has up to four TMA
    // instructions, and one thread that issued them all fell behind the tensor cores.
    const bool is_a = warp == 0;
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int id = pair; ok && id < P.units; id += npairs) {
        const Unit t = find_unit_ffn(P, id);
        const FfnProblem& p = P.p[t.prob];
        int k0, k1;
        split_range(p, t.split, k0, k1);
        const int half = p.bn / 2;
        const bool mn = is_a ? p.a_mn : p.b_mn;
        const int row = is_a ? t.m * 2 * p.mrows + (int)rank * p.mrows
                             : (p.b_by_rank ? t.n * half : t.n * p.bn + (int)rank * half);
        const bool two = mn && (is_a || half > 64);
        const uint32_t ring = smem_u32(smem) + (is_a ? 0 : a_bytes(p));
        const uint32_t bytes = is_a ? a_bytes(p) : b_bytes(p.bn, p.b_mn);
        const CUtensorMap* maps = is_a ? p.a : p.b;
        int seg = k0 >= p.nkb ? 1 : 0;
        int left = p.nkb * (seg + 1) - k0;
        int k = (k0 - seg * p.nkb) * kBK;
        const CUtensorMap* map = &maps[!is_a && p.b_by_rank ? (int)rank : seg];
        if (nfill == 0) griddep_wait();
        for (int n = k1 - k0; n > 0; n -= kPer) {
          if (!wait_bar_fast(&empty[stage], phase ^ 1, meta, s_abort, limit, kSiteProducerEmpty)) { ok = false; break; }
          const uint32_t fb = full_c0 + 8u * stage;
          auto block = [&](uint32_t dst) {
            if (mn) {
              tma_load_2d_pair(dst, map, fb, row, k);
              if (two) tma_load_2d_pair(dst + kFBoxBytes, map, fb, row + 64, k);
            } else {
              tma_load_2d_pair(dst, map, fb, k, row);
            }
            k += kBK;
            if (--left == 0) {  // the second segment's operands
              k = 0;
              map = &maps[!is_a && p.b_by_rank ? (int)rank : 1];
            }
          };
          const uint32_t dst = ring + stage * stage_bytes;
          const bool both = kPer == 2 && n > 1;
          mbar_arrive_expect_tx_cluster(fb, both ? 2 * bytes : bytes);
          block(dst);
          if (both) block(dst + block_bytes);
          ++nfill;
          if (++stage == (uint32_t)nst) { stage = 0; phase ^= 1; }
        }
      }
      // the arrivals of CTA 0's commits on this CTA's `empty` barriers: the last of them are here before
      // this CTA may end
      for (int i = 0; is_a && ok && i < nst; ++i) {
        ok = wait_bar_fast(&empty[stage], phase ^ 1, meta, s_abort, limit, kSiteProducerEmpty);
        if (++stage == (uint32_t)nst) { stage = 0; phase ^= 1; }
      }
    }
    __syncwarp();
    nfill = __reduce_max_sync(0xffffffffu, nfill);  // every lane: what the elected one counted
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (CTA 0) ------------------------------
    if (rank == 0 && elect_one()) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      griddep_wait();  // the kernel in front is not on this one's clock
      for (int id = pair; ok && id < P.units; id += npairs) {
        const Unit t = find_unit_ffn(P, id);
        const FfnProblem& p = P.p[t.prob];
        int k0, k1;
        split_range(p, t.split, k0, k1);
        const uint32_t idesc = idesc_bf16_f32(kFfnTileM, p.bn) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16);
        // a 16-wide K step: 32 bytes further along a K-major row, two atoms along MN-major k
        const uint64_t astep = p.a_mn ? (2048 >> 4) : (32 >> 4), bstep = p.b_mn ? (2048 >> 4) : (32 >> 4);
        if (!wait_bar_fast(&acc_empty[acc], acc_phase ^ 1, meta, s_abort, limit, kSiteMmaAcc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kAccCols;
        for (int kb = k0; kb < k1; kb += kPer) {
          if (!wait_bar_fast(&full[stage], phase, meta, s_abort, limit, kSiteMmaFull)) { ok = false; break; }
          tc_fence_after();
          auto block = [&](uint32_t a, bool onto) {
            const uint32_t b = a + a_bytes(p);
            const uint64_t ad = p.a_mn ? sdesc_mnmajor_sw128(a) : sdesc_kmajor_sw128(a);
            const uint64_t bd = p.b_mn ? sdesc_mnmajor_sw128(b) : sdesc_kmajor_sw128(b);
#pragma unroll
            for (int kk = 0; kk < kBK / kUK; ++kk)
              umma_bf16_pair(d, ad + kk * astep, bd + kk * bstep, idesc, onto || kk != 0);
          };
          const uint32_t a = smem_u32(smem + stage * stage_bytes);
          block(a, kb != k0);
          if (kPer == 2 && kb + 1 < k1) block(a + block_bytes, true);
          mma_issued = true;
          umma_commit_pair_mc(&empty[stage], 3);
          if (++stage == (uint32_t)nst) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        umma_commit_pair_mc(&acc_full[acc], 3);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok) give_up();
    }
    __syncwarp();
  } else if (warp == 7) {
    // ------------- dh: u and g into the staging buffers, du, dg and h out of them -------------
    if (kEpi == kFfnDSwiglu && P.p[0].splits == 1 && elect_one()) {
      const FfnProblem& p = P.p[0];
      const int nchunk = (p.bn + kFChunk - 1) / kFChunk;
      struct Cursor {
        int id, cc, col, row;
      } in{pair, 0, 0, 0}, out{pair, 0, 0, 0};
      auto place = [&](Cursor& c) {
        const Unit t = find_unit_ffn(P, c.id);
        c.col = t.n * p.bn;
        c.row = t.m * 2 * p.mrows + (int)rank * p.mrows;
      };
      auto next = [&](Cursor& c) {
        if (++c.cc == nchunk) {
          c.cc = 0;
          c.id += npairs;
          if (c.id < P.units) place(c);
        }
      };
      place(in);
      place(out);
      griddep_wait();
      uint32_t loads = 0;
      auto load = [&]() {  // the next chunk's u and g into buffer loads % 2, which is free
        const uint32_t b = loads & 1;
        const uint32_t dst = smem_u32(staging) + b * kFInBytes;
        const int col = in.col + chunk_col(in.cc, p.bn);
        mbar_arrive_expect_tx(&ug_full[b], 2 * p.mrows * kFChunk * 2);
        tma_load_2d(dst, &P.in_u, &ug_full[b], col, in.row);
        tma_load_2d(dst + 8192, &P.in_g, &ug_full[b], col, in.row);
        ++loads;
        next(in);
      };
      for (int i = 0; i < 2 && in.id < P.units; ++i) load();
      const uint32_t src = smem_u32(staging) + kFOutOff;
      for (uint32_t n = 0; out.id < P.units; ++n) {
        if (in.id < P.units) {
          if (!wait_bar_fast(&ug_free[n & 1], (n >> 1) & 1, meta, s_abort, limit, kSiteEpiTask)) break;
          load();
        }
        if (!wait_bar_fast(ready, n & 1, meta, s_abort, limit, kSiteEpiTask)) break;
        const int col = out.col + chunk_col(out.cc, p.bn);
        if (out.row < p.nrows && col < p.ncols) {
          tma_store_2d(&p.out, src, col, out.row);
          tma_store_2d(&P.out2, src + 8192, col, out.row);
          tma_store_2d(&P.out3, src + 16384, col, out.row);
        }
        bulk_commit_group();
        bulk_wait_group_read<0>();
        mbar_arrive(out_free);
        next(out);
      }
      bulk_wait_group<0>();
      for (uint32_t b = 0; b < 2; ++b)  // after an abort, loads that nobody waited for
        if (loads > b) wait_bar_drain(&ug_full[b], ((loads - 1 - b) >> 1) & 1, meta, limit);
    }
    __syncwarp();
  } else {
    // ----------------------------------- epilogue -----------------------------------
    // Each thread owns one row of the MMA's 128 in this CTA, of which the first mrows are stored. A step
    // takes 32 columns, or 64 of a single bf16 result: rows of 128 bytes (128-byte swizzle) or, of several bf16 results, 64
    // (64-byte swizzle), stored by TMA.
    const int q = warp & 3;
    const int row = q * 32 + lane;
    auto leader = [&]() { return warp == 2 && elect_one(); };  // always the same lane
    uint32_t acc = 0, acc_phase = 0, sb = 0, ug_phase = 0, out_phase = 0;
    auto get_bf16 = [&](const uint8_t* buf, uint32_t (&w)[16]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(buf + row * 64 + ((j ^ ((row >> 1) & 3)) << 4));
        w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
      }
    };
    auto put_bf16 = [&](uint8_t* buf, const uint32_t (&w)[16]) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(buf + row * 64 + ((j ^ ((row >> 1) & 3)) << 4)) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    };
    auto put_128 = [&](uint8_t* buf, const uint32_t (&w)[32]) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(buf + row * 128 + ((j ^ (row & 7)) << 4)) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    };
    griddep_wait();
    uint32_t it = 0;
    for (int id = pair; id < P.units; id += npairs, ++it) {
      const Unit t = find_unit_ffn(P, id);
      const FfnProblem& p = P.p[t.prob];
      const int m0 = t.m * 2 * p.mrows + (int)rank * p.mrows;
      // one thread waits for the accumulator and tells the other 127, so that the warps always
      // leave the loop together
      if (leader()) s_go[it & 1] = wait_bar(&acc_full[acc], acc_phase, meta, s_abort, limit, kSiteEpiAcc) ? 1 : 0;
      named_bar_sync(1, 128);
      if (s_go[it & 1] == 0) {
        if (leader()) give_up();
        break;
      }
      tc_fence_after();
      const uint32_t tacc = tmem_base + acc * kAccCols + (static_cast<uint32_t>(q * 32) << 16);
      const int mstore = p.splits > 1 ? t.split * p.mpad + m0 : m0;
      const bool rows_in = p.splits > 1 || m0 < p.nrows;  // partials hold whole tiles of rows
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_c0 + 8u * acc);
      };
      if (kEpi == kFfnStore || p.splits > 1) {
        // partials of u | g: the tile's second half belongs to g's columns
        const int width = p.b_by_rank ? p.bn / 2 : p.bn;
        const int chunk = p.out_kind == 0 ? 2 * kFChunk : kFChunk, per = (width + chunk - 1) / chunk;
        const int nchunk = p.b_by_rank ? 2 * per : per;
#pragma unroll 1
        for (int cc = 0; cc < nchunk; ++cc) {
          const int part = cc >= per ? 1 : 0;
          const int c0 = chunk_col(cc - part * per, width, chunk);
          uint32_t v[32];
          tmem_ld_32x32b_x32(tacc + part * width + c0, v);
          uint8_t* buf = staging + sb * 16384;
          if (p.out_kind == 0) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(tacc + c0 + kFChunk, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              v[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
              x[j] = pack_bf16x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) v[16 + j] = x[j];
          } else {
            tmem_ld_wait();
          }
          if (cc == nchunk - 1) release();
          if (leader()) bulk_wait_group_read<1>();
          named_bar_sync(1, 128);
          if (p.out_kind == 2 && c0 < cc * kFChunk) {  // columns that the chunk before has added
#pragma unroll
            for (int j = 0; j < kFChunk; ++j)
              if (c0 + j < cc * kFChunk) v[j] = 0;
          }
          put_128(buf, v);
          fence_proxy_async_shared();
          named_bar_sync(1, 128);
          if (leader()) {
            const int c = t.n * width + c0, col = part * p.gcol + c;
            const bool in = rows_in && c < p.ncols;
            if (in) {
              if (p.out_kind == 2) tma_reduce_add_2d(&p.out, smem_u32(buf), col, mstore);
              else tma_store_2d(&p.out, smem_u32(buf), col, mstore);
            }
            bulk_commit_group();
          }
          sb ^= 1;
        }
      } else if constexpr (kEpi == kFfnSwiglu) {
        const int hn = p.bn / 2, nchunk = (hn + kFChunk - 1) / kFChunk;
#pragma unroll 1
        for (int cc = 0; cc < nchunk; ++cc) {
          const int c0 = chunk_col(cc, hn);
          uint32_t u[32], g[32], pk[16];
          tmem_ld_32x32b_x32(tacc + c0, u);
          tmem_ld_32x32b_x32(tacc + hn + c0, g);
          tmem_ld_wait();
          if (cc == nchunk - 1) release();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[j] = pack_bf16x2(swiglu(__uint_as_float(u[2 * j]), __uint_as_float(g[2 * j])),
                                swiglu(__uint_as_float(u[2 * j + 1]), __uint_as_float(g[2 * j + 1])));
          uint8_t* buf = staging + sb * 24576;
          if (leader()) bulk_wait_group_read<1>();
          named_bar_sync(1, 128);
          put_bf16(buf, pk);
          if (P.save) {
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
            put_bf16(buf + 8192, pk);
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(__uint_as_float(g[2 * j]), __uint_as_float(g[2 * j + 1]));
            put_bf16(buf + 16384, pk);
          }
          fence_proxy_async_shared();
          named_bar_sync(1, 128);
          if (leader()) {
            const int col = t.n * hn + c0;
            if (rows_in && col < p.ncols) {
              tma_store_2d(&p.out, smem_u32(buf), col, m0);
              if (P.save) {
                tma_store_2d(&P.out2, smem_u32(buf) + 8192, col, m0);
                tma_store_2d(&P.out3, smem_u32(buf) + 16384, col, m0);
              }
            }
            bulk_commit_group();
          }
          sb ^= 1;
        }
      } else if constexpr (kEpi == kFfnDSwiglu) {
        // warp 7 brings u and g of a chunk, two chunks ahead, and stores du, dg and h from the out
        // buffer. A wait that gives up only spoils results: the loop ends at the next tile.
        const int nchunk = (p.bn + kFChunk - 1) / kFChunk;
#pragma unroll 1
        for (int cc = 0; cc < nchunk; ++cc) {
          uint32_t v[32], uw[16], gw[16], hh[16];
          const uint8_t* inb = staging + sb * kFInBytes;
          uint8_t* buf = staging + kFOutOff;
          tmem_ld_32x32b_x32(tacc + chunk_col(cc, p.bn), v);
          wait_bar_fast(&ug_full[sb], ug_phase, meta, s_abort, limit, kSiteEpiTask);
          get_bf16(inb, uw);
          get_bf16(inb + 8192, gw);
          mbar_arrive(&ug_free[sb]);
          tmem_ld_wait();
          if (cc == nchunk - 1) release();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a0, a1, b0, b1, c0, c1;
            dswiglu(__uint_as_float(v[2 * j]), __uint_as_float(uw[j] << 16), __uint_as_float(gw[j] << 16), a0, b0, c0);
            dswiglu(__uint_as_float(v[2 * j + 1]), __uint_as_float(uw[j] & 0xffff0000u),
                    __uint_as_float(gw[j] & 0xffff0000u), a1, b1, c1);
            uw[j] = pack_bf16x2(a0, a1);
            gw[j] = pack_bf16x2(b0, b1);
            hh[j] = pack_bf16x2(c0, c1);
          }
          wait_bar_fast(out_free, out_phase ^ 1, meta, s_abort, limit, kSiteEpiTask);
          put_bf16(buf, uw);
          put_bf16(buf + 8192, gw);
          put_bf16(buf + 16384, hh);
          fence_proxy_async_shared();
          mbar_arrive(ready);
          out_phase ^= 1;
          sb ^= 1;
          if (sb == 0) ug_phase ^= 1;
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    if (leader()) bulk_wait_group<0>();
  }

  griddep_launch_dependents();
  // teardown. Where every unit was finished, every fill was consumed and every MMA waited for (by both
  // epilogues): nothing is in flight. After an abort CTA 0 drains both CTAs' fills, which complete on its
  // `full` barriers, and the MMAs, which write both CTAs' tensor memory, before either CTA moves on.
  // (Draining always took 3 us of every launch.)
  tc_fence_before();
  if (lane == 0 && (warp == 0 || warp == 6))
    st_cluster_u32(mapa_shared(smem_u32((const void*)&s_nfill[2 * rank + (warp == 6 ? 1 : 0)]), 0), nfill);
  cluster_sync_all();
  if (*s_left) {
    if (rank == 0 && threadIdx.x == 0) {
      // some producers may have issued up to a ring's worth of fills that others did not: arrive for
      // those so that the phases complete when the bytes land
      uint32_t hi = 0;
      for (int i = 0; i < 4; ++i) hi = max(hi, s_nfill[i]);
      for (int i = 0; i < 4; ++i)
        for (uint32_t j = s_nfill[i]; j < hi; ++j) mbar_arrive(&full[j % nst]);
      drain_fills(full, nst, hi, meta, limit);
    }
    if (mma_issued) {  // in the thread that issued the MMAs
      umma_commit_pair(drain);
      wait_bar_drain(drain, 0, meta, limit);
    }
    __syncwarp();
    cluster_sync_all();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, 2 * kAccCols);
}

namespace {

// 8 consecutive elements of the sum of the splits' partials, in split order.
__device__ __forceinline__ void sum_parts(const FfnReduce& r, int64_t off, float (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = 0.f;
  for (int s = 0; s < r.splits; ++s) {
    const float4* p = reinterpret_cast<const float4*>(r.parts + s * r.split_stride + off);
    const float4 x = __ldcg(p), y = __ldcg(p + 1);
    a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
    a[4] += y.x; a[5] += y.y; a[6] += y.z; a[7] += y.w;
  }
}

__device__ __forceinline__ void unpack8(const uint16_t* p, float (&a)[8]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = 0.f;
  add_bf16x8(a, v);
}

}  // namespace

// One thread per 8 columns (every N here is a multiple of 8).
template <int kEpi>
__global__ void __launch_bounds__(256) ffn_reduce_kernel(const FfnReduce r) {
  griddep_wait();
  griddep_launch_dependents();
  const int vec = r.cols / 8;
  const int64_t n = (int64_t)r.rows * vec;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / vec;
    const int col = (int)(i % vec) * 8;
    const int64_t o = row * r.cols + col;
    float a[8];
    sum_parts(r, row * r.ld + col, a);
    if constexpr (kEpi == kFfnStore) {
      if (r.out_kind == 0) {
        store8<true>(r.out, o, a);
      } else {
        if (r.out_kind == 2) {
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(r.out) + o);
          const float4 x = p[0], y = p[1];
          a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
          a[4] += y.x; a[5] += y.y; a[6] += y.z; a[7] += y.w;
        }
        store8<false>(r.out, o, a);
      }
    } else if constexpr (kEpi == kFfnSwiglu) {
      float g[8], h[8];
      sum_parts(r, row * r.ld + r.gcol + col, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = swiglu(a[j], g[j]);
      store8<true>(r.out, o, h);
      if (r.out2) {
        store8<true>(r.out2, o, a);
        store8<true>(r.out3, o, g);
      }
    } else {
      float u[8], g[8], du[8], dg[8], h[8];
      unpack8(r.u + o, u);
      unpack8(r.g + o, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) dswiglu(a[j], u[j], g[j], du[j], dg[j], h[j]);
      store8<true>(r.out, o, du);
      store8<true>(r.out2, o, dg);
      store8<true>(r.out3, o, h);
    }
  }
}

cudaError_t launch_ffn_reduce(const FfnReduce& r, int epilogue, int num_sms, cudaStream_t stream) {
  const int64_t n = (int64_t)r.rows * (r.cols / 8);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, (int64_t)num_sms * 8));
  auto* k = epilogue == kFfnStore ? ffn_reduce_kernel<kFfnStore>
                                  : (epilogue == kFfnSwiglu ? ffn_reduce_kernel<kFfnSwiglu> : ffn_reduce_kernel<kFfnDSwiglu>);
  return launch_k(k, dim3(grid), dim3(256), 0, stream, r);
}

namespace {

typedef void (*FfnKernel)(const FfnParams);

template <int kPer>
FfnKernel ffn_kernel_of(int epilogue) {
  return epilogue == kFfnStore
             ? ffn_gemm_kernel<kFfnStore, kPer>
             : (epilogue == kFfnSwiglu ? ffn_gemm_kernel<kFfnSwiglu, kPer> : ffn_gemm_kernel<kFfnDSwiglu, kPer>);
}

FfnKernel ffn_kernel(int epilogue, int per) { return per == 2 ? ffn_kernel_of<2>(epilogue) : ffn_kernel_of<1>(epilogue); }

// Blocks of a stage: two where four such stages fit (with fewer, 128 x 128 tiles of 2048 tokens were slower, 24.9
// us for 22.5) and no tile is so wide that its MMAs take longer than their issue.
int blocks_per_stage(const FfnParams& p, int epilogue) {
  int widest = 0;
  for (int i = 0; i < p.nprob; ++i) widest = std::max(widest, (int)p.p[i].bn);
  return widest <= 160 && ring_bytes(epilogue) >= 4 * 2 * most_block_bytes(p) ? 2 : 1;
}

}  // namespace

cudaError_t launch_ffn_gemm(const FfnParams& p, int epilogue, int pairs, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * std::min(pairs, p.units));
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = kFSmem + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ffn_kernel(epilogue, blocks_per_stage(p, epilogue)), p);
}

// Sets the kernels' shared-memory limits and returns how many 2-CTA clusters fit on the device at
// once (0 if none).
cudaError_t configure_ffn_kernels(int* max_pairs) {
  *max_pairs = 0;
  for (int e = 0; e < 6; ++e) {
    const cudaError_t rc =
        cudaFuncSetAttribute(ffn_kernel(e / 2, 1 + e % 2), cudaFuncAttributeMaxDynamicSharedMemorySize, kFSmem + 1024);
    if (rc != cudaSuccess) return rc;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = kFSmem + 1024;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(max_pairs, (void*)ffn_kernel(kFfnStore, 1), &cfg);
}

}  // namespace moe
