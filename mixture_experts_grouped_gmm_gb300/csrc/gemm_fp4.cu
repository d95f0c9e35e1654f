// mgemm_fwd_fp4 / mgemm_gmm_fp4: the grouped product of 4-bit block-scaled
// operands on the tensor cores,
//
//   out[r, n] = sum_k xv[r, k] wv[e(r), n, k]
//
// over the tile schedule of mgemm_fill_args.  The MMAs are block-scaled
// (kind::mxf4nvf4): D += sum over the 64 elements of a step of (a sfa)(b sfb),
// with one scale per 32 (MXFP4, e8m0) or 16 (NVFP4, e4m3) elements of each row
// read from tensor memory.  NVFP4's two row scales lie outside the sum: the
// epilogue multiplies by 1 / rx[r] and 1 / rw[e, n] (f4_far: the one may be far
// from 1 where the other brings the output back).  The casts' are powers of two,
// weights from elsewhere may have any.
//
// A tile is 128 token rows of one group by bn columns; a stage holds 256
// elements of the contraction (128 bytes of a row): the operands' codes,
// 128-byte swizzled by TMA, and their scale words, which the global layout
// keeps in the order tensor memory wants them, so the MMA thread only copies
// them there (tcgen05.cp, 512 bytes per 128 rows and word) ahead of the
// stage's four MMAs.
//
// CTA (persistent, one per SM, 384 threads; warps 4-11 take registers from the
// others, without which the accumulator's 128 columns spill):
//   warp 0     TMA producer: a ring of stages, as many as fit
//   warp 1     TMEM owner; issues the MMAs
//   warp 2     copies a stage's scales to tensor memory ahead of its MMAs (98304
//              x 1408 x 2048 takes 137 us with one warp for copies and MMAs, 126
//              with two)
//   warps 4-11 epilogue, two per TMEM lane quarter, each half of the columns:
//              the accumulator is read into registers and handed back, the next
//              tile's factors are fetched (16384 x 2048 x 256, NVFP4: 23.2 us,
//              27.8 with each tile's own fetched before its wait), and the
//              columns are scaled, rounded and stored, 32 at a time, through a
//              swizzled 2 KB buffer and TMA (stores of 32 rows from registers
//              hold up the load-store unit for some 3000 clocks a tile, and
//              with it every barrier of the pipeline); rows of a group's edge
//              and scattered rows are stored directly
// TMEM: one accumulator of 256 columns or two narrower ones, then as many slots
// of scales as fit (two to sixteen).  A slot is rewritten once the MMAs that read it
// have completed: the stage's empty barrier says so.
// PAIR (many groups of 256 rows and more, some of 128; see fp4_form): a cluster of two CTAs computes 256 rows by
// bn columns with cta_group::2 MMAs of the even CTA.  Each CTA copies its 128
// rows of A, half of B's columns and the scales of its rows and of all columns;
// the odd CTA's copies complete on the even CTA's barriers, and commits free a
// stage and publish the accumulator in both.  A CTA then fetches 38 KB per
// stage instead of 54.
// What bounds large products (pairs, 256 columns, at 1.8 GHz): a stage takes 0.35
// us, 0.28 (the 512 clocks of its MMAs) without its copies, 0.23 without its MMAs:
// shared memory takes in the 38 KB and gives 38 KB to the MMAs, 600 clocks at 128
// bytes each.  A tile adds about 1 us, most of it from the last MMA to the next
// tile's first, while the accumulator is read; two accumulators of 192 columns,
// which leave scales two slots, hide that and cost more (154 us for the above).
// Every wait is bounded; on expiry the kernel records MGEMM_STATUS_TIMEOUT,
// drains the copies and MMAs it issued, frees TMEM and returns.
#include <cmath>

#include "fp4.cuh"

namespace mgemm {
namespace {

struct Fp4Params {
  const uint8_t *args;
  const float *rx, *rw;
  __nv_bfloat16 *out;
  const int32_t *row_map;
  int64_t map_limit;
  const float *row_weight;
  int K, N, E;
  int bn, n_tiles;    // columns per tile: 64, 128, 192 or 256 (pairs: 128 or 256)
  int a_rows;         // rows of an A box: 128, or fewer when M is smaller (a multiple of 8)
  int stages, stage_bytes;
  int vec32;          // output rows and tiles start on 32-byte boundaries
  // Not NULL (mgemm_gmm_fp4): the group sizes, from which the kernel makes its own
  // schedule, so that it can start on the weights before the cast has ended (a
  // call of one token 14.6 -> 12.5 us, one of 16 at 16 experts 62.5 -> 59.8).
  const int64_t *sizes;
  int64_t M;
};

constexpr int kF4Threads = 384;
constexpr int kF4EpiWarps = 8;
// Registers a thread at launch, as ptxas gives them to kF4Threads threads (a build may say otherwise to test the
// refusal of any other count: see FEW_REGS).
#ifndef MGEMM_F4_REGS
#define MGEMM_F4_REGS 168
#endif
constexpr int kF4Regs = MGEMM_F4_REGS;
constexpr int kF4MaxStages = 20;
constexpr int kF4MaxSlots = 16;  // slots of scales in tensor memory
constexpr int kF4Groups = 128;  // active groups whose places are kept in shared memory
constexpr int kF4Stage = 32 * 64;  // bytes of an epilogue warp's staging buffer: 32 rows of 32 columns
constexpr size_t kF4Limit = (size_t)227 * 1024;

template <int FMT, bool kPair>
struct F4Cfg {
  static constexpr bool NV = FMT == MGEMM_NVFP4, PAIR = kPair;
  static constexpr int WPS = 256 / Fp4<FMT>::WORD;  // scale words of a row per stage: 4 or 2
  // Registers a thread after the launch, of the first four warps and of the epilogue's (where nothing spills). Were
  // they more than the launch's, the epilogue would wait for registers that nobody gives up.
  static constexpr int FEW_REGS = NV && PAIR ? 88 : 104, EPI_REGS = NV && PAIR ? 208 : 200;
  static_assert(128 * FEW_REGS + 32 * kF4EpiWarps * EPI_REGS <= kF4Threads * kF4Regs, "registers");
  // a CTA's codes and scales; nt = scale tiles (128 columns) of the B tile
  static int stage_bytes(int a_rows, int bn) {
    const int nt = (bn + 127) / 128;
    return (a_rows + (PAIR ? bn / 2 : bn)) * 128 + (1 + nt) * WPS * 512;
  }
};

struct F4Shared {
  uint64_t full[kF4MaxStages], empty[kF4MaxStages], tfull[2], tempty[2], drain, sf_ready[kF4MaxSlots], sf_drain;
  uint32_t tmem_slot;
  int abort_flag;
  float cinv[kF4EpiWarps][128];  // the warps' column factors
  GroupSums sums;
  int na;
  // the active groups' first tile, expert, rows and first scale tile
  int start[kF4Groups + 1], expert[kF4Groups], row[kF4Groups], end[kF4Groups], sf[kF4Groups];
};

struct F4Tile {
  int e, n0, rows, row0, sf_tile;
};

// The tile t: group by the row-tile prefix (of 256-row tiles for pairs), row
// tiles fastest inside it, so that CTAs running together share a weight tile
// through L2.  A pair's rank takes the tile's rows 128 rank ..; the odd one's may
// lie past the group (loaded, never stored).  Every role asks for rising tiles,
// so the group `g` is stepped on from the last one.  The groups' places come from
// shared memory: from the args block they are a chain of loads that mostly miss
// L1 (shared memory takes nearly all of it), 5000 clocks a tile and role.
template <bool PAIR>
__device__ __forceinline__ F4Tile f4_tile(int t, int &g, const Fp4Params &p, const F4Shared &S, const ArgsView &av,
                                          int na, int rank) {
  const int gm = t / p.n_tiles;
  F4Tile ti;
  int first, mts, end, sf;
  if (na <= kF4Groups) {
    while (S.start[g + 1] <= gm) ++g;
    first = S.start[g];
    mts = S.start[g + 1] - first;
    ti.e = S.expert[g];
    ti.row0 = S.row[g];
    end = S.end[g];
    sf = S.sf[g];
  } else {
    const int *start = PAIR ? av.ptile_start : av.mtile_start;
    while (__ldg(start + g + 1) <= gm) ++g;
    first = __ldg(start + g);
    mts = __ldg(start + g + 1) - first;
    ti.e = __ldg(av.active + g);
    ti.row0 = (int)__ldg(av.offsets + ti.e);
    end = (int)__ldg(av.offsets + ti.e + 1);
    sf = (int)(__ldg(av.poffsets + ti.e) >> 7);
  }
  const int local = t - first * p.n_tiles;
  const int mt = PAIR ? 2 * (local % mts) + rank : local % mts;
  ti.n0 = local / mts * p.bn;
  ti.row0 += mt * 128;
  ti.rows = max(0, min(end - ti.row0, p.a_rows));
  ti.sf_tile = sf + mt;
  return ti;
}

// The schedule of E <= 256 groups, at most kF4Groups of them with rows, from their
// sizes.  Sizes that do not fit leave no tile (the call's fill reports them).
__device__ __forceinline__ void f4_schedule(const Fp4Params &p, F4Shared &S) {
  const int i = threadIdx.x;
  const int64_t m = i < p.E ? __ldcg(p.sizes + i) : 0;
  int64_t rows;
  uint64_t tiles;
  const bool valid = scan_groups<kF4Threads>(m, p.M, S.sums, rows, tiles);
  if (valid && m > 0) {
    const int a = (int)(tiles >> 32) - 1;
    S.expert[a] = i;
    S.row[a] = (int)(rows - m);
    S.end[a] = (int)rows;
    S.start[a] = S.sf[a] = (int)tiles - (int)((m + 127) / 128);  // (row tiles are scale tiles)
  }
  if (i == kF4Threads - 1) {
    S.na = valid ? (int)(tiles >> 32) : 0;
    S.start[S.na] = valid ? (int)tiles : 0;
  }
  __syncthreads();
}

// One lane of a converged warp.  The instructions that take uniform registers
// (MMAs, scale copies, TMA, commits) are issued under it, with operands every
// lane has computed alike: behind a test of the lane number the compiler cannot
// know that, and moves each operand through a loop over the active lanes (an
// MMA then takes 170 to 220 clocks to issue; here a 128 x 256 x 64 one takes
// the 128 that it computes, scale copies hidden beneath).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// v, which every lane holds alike, as a result the compiler knows to be uniform
// (a warp reduction is written to a uniform register).
__device__ __forceinline__ int uniform(int v) { return (int)__reduce_or_sync(0xffffffffu, (unsigned)v); }

// Arrive on an mbarrier of the pair's other CTA.  The order that matters, of the
// accumulator's reads before it is written again, is the tcgen05 fence's; a
// release at cluster scope would also wait for the SM's output stores (3000
// clocks a tile).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_f4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
#define MGEMM_F4_MMA(GROUP, VEC)                                                                                      \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                     \
               "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                         \
               " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                                    \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                       \
               : "memory")
  if constexpr (PAIR) {
    if constexpr (FMT == MGEMM_NVFP4) MGEMM_F4_MMA("2", "4X");
    else MGEMM_F4_MMA("2", "2X");
  } else {
    if constexpr (FMT == MGEMM_NVFP4) MGEMM_F4_MMA("1", "4X");
    else MGEMM_F4_MMA("1", "2X");
  }
#undef MGEMM_F4_MMA
}

// 512 bytes of scales (32 rows of 16) to four columns of every lane quarter; a
// pair's copy does so in both CTAs, each from its own shared memory.
template <bool PAIR>
__device__ __forceinline__ void copy_scale_tile(uint32_t taddr, uint64_t sdesc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
  else
    tmem_cp_32x128b_warpx4(taddr, sdesc);
}

// Instruction descriptor of the block-scaled 4-bit MMA: e2m1 A and B (code 1),
// K-major, M = m, N = n, scales ue4m3 (0) or ue8m0 (1); the scale-factor ids
// (bits 4-5 and 29-30) are or-ed in per MMA.
__device__ __forceinline__ uint32_t f4_idesc(int m, int n, uint32_t ue8m0) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (ue8m0 << 23) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ uint64_t f32x2(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) { return f32x2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2_u64(uint64_t v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <int N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 1 / s within 2^-23 of it; exact where s is a power of two (2^-120 .. 2^120), as the casts' scales are
__device__ __forceinline__ float f4_recip(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// A row's factor f times a column's (2^-51 .. 2^117) has the range of a float, and that times the accumulator (0, or
// 2^-20 .. 2^23 K) leaves it only where the output does, for f in 2^-64 .. 2.  From any other f a power of two is taken
// out and returned: it multiplies the outputs once they are rounded, which is exact, and may take them out of range only
// where they are.  (Row times accumulator first, 1 / rx being up to 2^117, is past a float for rows of about 1e33 on
// whatever the column's factor.)
__device__ __forceinline__ float f4_far(float &f) {
  const int a = (int)((__float_as_uint(f) >> 23) & 0xFFu) - 127, h = a > 0 ? min(a, 126) : a < -64 ? a / 2 : 0;
  f *= __uint_as_float((uint32_t)(127 - h) << 23);
  return __uint_as_float((uint32_t)(127 + h) << 23);
}

__device__ __forceinline__ void store_32b(void *dst, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// NT: scale tiles (128 columns) of a column tile
template <int FMT, bool PAIR, int NT>
__global__ void __launch_bounds__(kF4Threads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ Fp4Params p) {
  using C = F4Cfg<FMT, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // [stages x (A codes | B codes)], then the stages' scales [A tile: WPS words][B tiles: WPS words each]
  const int nst = p.stages, bn = p.bn;
  const int b_rows = PAIR ? bn / 2 : bn;
  const int op_bytes = (p.a_rows + b_rows) * 128, sf_bytes = (1 + NT) * C::WPS * 512;
  uint8_t *sSF = smem + (size_t)nst * op_bytes;
  uint8_t *sOut = sSF + (size_t)nst * sf_bytes;  // the epilogue's staging buffers (512-byte aligned)
  F4Shared &S = *reinterpret_cast<F4Shared *>(sOut + kF4EpiWarps * kF4Stage);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  // accumulators, the columns from one to the next, and the slots of scales behind them
  const int nacc = bn == 256 ? 1 : 2, acc_cols = bn == 192 ? 192 : 128, sf_col0 = bn == 192 ? 384 : 256;
  constexpr int kSlotCols = C::WPS * (4 + 4 * NT);
  const int slots = (512 - sf_col0) / kSlotCols;
  const int rank = PAIR ? uniform((int)cluster_ctarank()) : 0;
  const int t_first = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int t_step = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const uint32_t op0 = (uint32_t)uniform((int)smem_u32(smem)), sf0 = op0 + (uint32_t)(nst * op_bytes);

  if (threadIdx.x == 0) {
    for (int i = 0; i < nst; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&S.tfull[a], 1);
      mbar_init(&S.tempty[a], PAIR ? 2 * kF4EpiWarps : kF4EpiWarps);
    }
    for (int i = 0; i < kF4MaxSlots; ++i) mbar_init(&S.sf_ready[i], 1);
    mbar_init(&S.drain, 1);
    mbar_init(&S.sf_drain, 1);
    S.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    tma_prefetch_desc(&tmOut);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&S.tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&S.tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers are initialised before either signals the other's
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = (uint32_t)uniform((int)S.tmem_slot);
  const ArgsView av(p.args, p.E);
  int na, total;
  const bool early = !PAIR && p.sizes != nullptr;
  if (early) {
    f4_schedule(p, S);
    na = uniform(S.na);
    total = uniform(S.start[na] * p.n_tiles);
  } else {
    pdl_wait();
    pdl_trigger();
    const int status0 = *av.status;
    na = uniform(*av.n_active);
    const int *start = PAIR ? av.ptile_start : av.mtile_start;
    total = uniform(status0 != 0 ? 0 : __ldg(start + na) * p.n_tiles);
    if (total > 0 && na <= kF4Groups) {
      for (int i = threadIdx.x; i < na; i += kF4Threads) {
        const int e = __ldg(av.active + i);
        S.start[i] = __ldg(start + i);
        S.expert[i] = e;
        S.row[i] = (int)__ldg(av.offsets + e);
        S.end[i] = (int)__ldg(av.offsets + e + 1);
        S.sf[i] = (int)(__ldg(av.poffsets + e) >> 7);
      }
      if (threadIdx.x == 0) S.start[na] = __ldg(start + na);
    }
    __syncthreads();
  }
  const int kb_count = (p.K + 255) / 256;
  int g = 0;  // the group of the last tile
  volatile int *vabort = &S.abort_flag;
  uint32_t issued = 0;  // stages armed, for the drain after an abort
  auto timeout = [&]() {
    set_status(av.status, MGEMM_STATUS_TIMEOUT);
    *vabort = 1;
    if constexpr (PAIR) st_cluster_u32(cluster_addr(&S.abort_flag, (uint32_t)rank ^ 1u), 1u);
  };
  // the MMA's columns of the tile at n0 (a pair's halves stay multiples of 32)
  auto tile_cols = [&](int n0) { return PAIR ? min(bn, (p.N - n0 + 63) & ~63) : min(bn, (p.N - n0 + 15) & ~15); };

  // (a schedule of its own: all but the producer wait here for the cast)
  if (early && warp != 0) {
    pdl_wait();
    pdl_trigger();
  }

  if (warp < 4) {
    reg_dealloc<C::FEW_REGS>();
    if (warp == 0) {
      bool ok = true;
      const uint32_t tx = (PAIR ? 2u : 1u) * (uint32_t)p.stage_bytes;
      const int wtiles = (p.N + 127) / 128;  // scale tiles of one expert's weights
      // body(step, stage, phase, kb, expert, columns, rows and their scale tiles), for every stage until it returns false
      auto for_stages = [&](auto &&body) {
        int step = 0, stage = 0;
        uint32_t phase = 0;
        g = 0;
        for (int t = t_first; t < total; t += t_step) {
          const F4Tile ti = f4_tile<PAIR>(t, g, p, S, av, na, rank);
          const int e = uniform(ti.e), n0 = uniform(ti.n0), row0 = uniform(ti.row0), sfa_tile = uniform(ti.sf_tile);
          const int sfb_tile = e * wtiles + n0 / 128, b_row = n0 + rank * (tile_cols(n0) / 2);
          for (int kb = 0; kb < kb_count; ++kb) {
            if (!body(step, stage, phase, kb, e, b_row, sfb_tile, row0, sfa_tile)) return;
            ++step;
            if (++stage == nst) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      };
      auto put = [&](bool w, bool x, int stage, int kb, int e, int b_row, int sfb_tile, int row0, int sfa_tile) {
        if (elect_one()) {
          uint8_t *a = smem + (size_t)stage * op_bytes, *sf = sSF + (size_t)stage * sf_bytes;
          if (!PAIR || rank == 0) {
            if (w) {
              mbar_arrive_expect_tx(&S.full[stage], tx);
              tma_load_3d(a + p.a_rows * 128, &tmB, &S.full[stage], kb * 128, b_row, e);
              tma_load_3d(sf + C::WPS * 512, &tmSB, &S.full[stage], 0, kb * C::WPS, sfb_tile);
            }
            if (x) {
              tma_load_2d(a, &tmA, &S.full[stage], kb * 128, row0);
              tma_load_3d(sf, &tmSA, &S.full[stage], 0, kb * C::WPS, sfa_tile);
            }
          } else {  // complete on the even CTA's barrier
            const uint32_t bar = cluster_addr(&S.full[stage], 0);
            tma_load_3d_pair(a + p.a_rows * 128, &tmB, bar, kb * 128, b_row, e);
            tma_load_3d_pair(sf + C::WPS * 512, &tmSB, bar, 0, kb * C::WPS, sfb_tile);
            tma_load_2d_pair(a, &tmA, bar, kb * 128, row0);
            tma_load_3d_pair(sf, &tmSA, bar, 0, kb * C::WPS, sfa_tile);
          }
        }
        __syncwarp();
        issued += w;
      };
      if (early) {
        // The ring is filled with weights, then, the cast done, with the rows.  The
        // weights may be read before this grid's wait: it is launched behind the
        // cast alone, every CTA of which has waited for whatever came before it
        // when it lets this grid start.
        for_stages([&](int step, int stage, uint32_t, int kb, auto... at) {
          if (step >= nst) return false;
          put(true, false, stage, kb, at...);
          return true;
        });
        pdl_wait();
        pdl_trigger();
        for_stages([&](int step, int stage, uint32_t, int kb, auto... at) {
          if (step >= nst) return false;
          put(false, true, stage, kb, at...);
          return true;
        });
      }
      for_stages([&](int step, int stage, uint32_t phase, int kb, auto... at) {
        if (early && step < nst) return true;
        ok = mbar_wait_warp(&S.empty[stage], phase ^ 1, vabort);
        if (ok) put(true, true, stage, kb, at...);
        return ok;
      });
      if (!ok && lane == 0) timeout();
    } else if (warp == 1) {
      int stage = 0, acc = 0, slot = 0;
      uint32_t phase = 0, acc_phase = 0, slot_phase = 0;
      bool ok = true;
      // (a pair: the even CTA issues for both)
      for (int t = t_first; t < total && ok && rank == 0; t += t_step) {
        const F4Tile ti = f4_tile<PAIR>(t, g, p, S, av, na, rank);
        const int n0 = uniform(ti.n0);
        const uint32_t idesc = (uint32_t)uniform((int)f4_idesc(PAIR ? 256 : 128, tile_cols(n0), C::NV ? 0u : 1u));
        // a tile of 64 or 192 columns may start in the middle of a 128-column scale tile
        const uint32_t sfb_off = (uint32_t)uniform((n0 & 64) ? 2 : 0);
        const uint32_t d_tmem = (uint32_t)uniform((int)tmem_base + acc * acc_cols);
        if (!mbar_wait_warp(&S.tempty[acc], acc_phase ^ 1, vabort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < kb_count; ++kb) {
          const uint32_t a = (uint32_t)uniform((int)op0 + stage * op_bytes);
          const uint32_t sfa_t = (uint32_t)uniform((int)tmem_base + sf_col0 + slot * kSlotCols), sfb_t = sfa_t + 4 * C::WPS;
          const bool here = mbar_wait(&S.full[stage], phase, vabort) && mbar_wait(&S.sf_ready[slot], slot_phase, vabort);
          if (!__all_sync(0xffffffffu, here)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = smem_desc_sw128(a, 16, 1024), bd = smem_desc_sw128(a + p.a_rows * 128, 16, 1024);
            auto step = [&](int k) {  // (descriptors advance by bytes >> 4)
              const int j = C::NV ? k : k / 2;
              const uint32_t id = C::NV ? 0u : (uint32_t)(k & 1) * 2u;
              mma_f4<FMT, PAIR>(d_tmem, ad + 2 * k, bd + 2 * k, idesc | (id << 4) | (id << 29), sfa_t + 4 * j,
                                sfb_t + 4 * j * NT + sfb_off, (kb | k) != 0);
            };
            if (kb * 256 + 256 <= p.K) {
#pragma unroll
              for (int k = 0; k < 4; ++k) step(k);
            } else {  // the contraction ends inside this stage
              const int steps = (p.K - kb * 256 + 63) / 64;
              for (int k = 0; k < steps; ++k) step(k);
            }
            if constexpr (PAIR) mma_commit_pair(&S.empty[stage], 0x3);
            else mma_commit(&S.empty[stage]);
          }
          __syncwarp();
          if (++slot == slots) {
            slot = 0;
            slot_phase ^= 1;
          }
          if (++stage == nst) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (elect_one()) {
          if constexpr (PAIR) mma_commit_pair(&S.tfull[acc], 0x3);
          else mma_commit(&S.tfull[acc]);
        }
        __syncwarp();
        if (++acc == nacc) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (!ok && lane == 0) timeout();
      if (rank == 0 && elect_one()) {
        if constexpr (PAIR) mma_commit_pair(&S.drain, 0x1);
        else mma_commit(&S.drain);
        mbar_wait_drain(&S.drain, 0);
      }
      __syncwarp();
    } else if (warp == 2) {
      int stage = 0, slot = 0, old = 0, it = 0;  // old: the stage of `slots` iterations ago
      uint32_t phase = 0, old_phase = 0;
      bool ok = true;
      for (int t = t_first; t < total && ok && rank == 0; t += t_step) {
        for (int kb = 0; kb < kb_count; ++kb) {
          const uint32_t sf = (uint32_t)uniform((int)sf0 + stage * sf_bytes);
          const uint32_t sfa_t = (uint32_t)uniform((int)tmem_base + sf_col0 + slot * kSlotCols), sfb_t = sfa_t + 4 * C::WPS;
          bool here = mbar_wait(&S.full[stage], phase, vabort);
          // the slot's last readers have completed (a ring of no more stages than slots says so by itself)
          const bool reuse = it >= slots && nst > slots;
          if (reuse) here = here && mbar_wait(&S.empty[old], old_phase, vabort);
          if (!__all_sync(0xffffffffu, here)) {
            ok = false;
            break;
          }
          if (reuse && ++old == nst) {
            old = 0;
            old_phase ^= 1;
          }
          it += it < slots;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t sd = smem_desc_rows16(sf);
            auto copy = [&](int j) {
              copy_scale_tile<PAIR>(sfa_t + 4 * j, sd + 32 * j);
              copy_scale_tile<PAIR>(sfb_t + 4 * j * NT, sd + 32 * (C::WPS + j));
              if (NT == 2) copy_scale_tile<PAIR>(sfb_t + 4 * j * NT + 4, sd + 32 * (2 * C::WPS + j));
            };
            if (kb * 256 + 256 <= p.K) {
#pragma unroll
              for (int j = 0; j < C::WPS; ++j) copy(j);
            } else {  // the words of the last steps
              const int steps = (p.K - kb * 256 + 63) / 64, words = C::NV ? steps : (steps + 1) / 2;
              for (int j = 0; j < words; ++j) copy(j);
            }
            if constexpr (PAIR) mma_commit_pair(&S.sf_ready[slot], 0x1);
            else mma_commit(&S.sf_ready[slot]);
          }
          __syncwarp();
          if (++slot == slots) slot = 0;
          if (++stage == nst) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok && lane == 0) timeout();
      if (rank == 0 && elect_one()) {  // every copy has landed before tensor memory is freed
        if constexpr (PAIR) mma_commit_pair(&S.sf_drain, 0x1);
        else mma_commit(&S.sf_drain);
        mbar_wait_drain(&S.sf_drain, 0);
      }
      __syncwarp();
    }
  } else {
    reg_alloc<C::EPI_REGS>();
    const int ew = warp - 4, q = warp & 3, h = ew >> 2;
    const int r = q * 32 + lane;  // the thread's row of the tile
    const int half = bn / 2;      // columns per warp: 32, 64, 96 or 128
    float *cinv = S.cinv[ew];
    int acc = 0;
    uint32_t acc_phase = 0;
    // A tile's factors are fetched while the one before it is scaled and stored.
    F4Tile ti{};
    bool row_ok = false;
    int64_t dst = 0;
    float weight = 1.f, rx = 1.f, rw[4] = {};
    auto fetch = [&]() {
      row_ok = r < ti.rows;
      dst = (int64_t)ti.row0 + r;
      if (C::NV && row_ok) rx = __ldg(p.rx + dst);
      if (p.row_map) {
        const int32_t d = row_ok ? __ldg(p.row_map + dst) : -1;
        row_ok = d >= 0 && d < p.map_limit;
        if (row_ok && p.row_weight) weight = __ldg(p.row_weight + d);
        dst = row_ok ? d : 0;
      }
      if (C::NV) {
        const int n = ti.n0 + h * half + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c * 32 < half) rw[c] = n + c * 32 < p.N ? __ldg(p.rw + (int64_t)ti.e * p.N + n + c * 32) : 1.f;
      }
    };
    if (t_first < total) {
      ti = f4_tile<PAIR>(t_first, g, p, S, av, na, rank);
      fetch();
    }
    for (int t = t_first; t < total; t += t_step) {
      if (C::NV) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c * 32 < half) cinv[c * 32 + lane] = f4_recip(rw[c]);
        __syncwarp();
      }
      // the row's factor, its place and the tile's
      float f = C::NV ? weight * f4_recip(rx) : weight;
      const int col0 = ti.n0 + h * half, row0 = ti.row0 + q * 32;
      const bool store = row_ok, whole = !p.row_map && q * 32 + 32 <= ti.rows;  // the warp's 32 rows are all the group's
      __nv_bfloat16 *o = p.out + dst * p.N + col0;
      // (the next tile's place before the wait, or, where its factors follow, after the accumulator's read)
      if (!C::NV && t + t_step < total) ti = f4_tile<PAIR>(t + t_step, g, p, S, av, na, rank);
      if (!mbar_wait_warp(&S.tfull[acc], acc_phase, vabort)) {
        if (lane == 0) timeout();
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * acc_cols + h * half;
      // the accumulator first, so that it is handed back at once
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c * 32 < half) tmem_ld_32x32b_x32(taddr + c * 32, v[c]);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&S.tempty[acc]);
        else mbar_arrive_remote(cluster_addr(&S.tempty[acc], 0));
      }
      if (++acc == nacc) {
        acc = 0;
        acc_phase ^= 1;
      }
      if (t + t_step < total) {
        if (C::NV) ti = f4_tile<PAIR>(t + t_step, g, p, S, av, na, rank);
        fetch();
      }
      const float far = C::NV ? f4_far(f) : 1.f;
      const bool any_far = C::NV && __any_sync(0xffffffffu, far != 1.f);
      const uint64_t f2 = f32x2(f, f);
      uint8_t *buf = sOut + ew * kF4Stage;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c * 32 >= half || col0 + c * 32 >= p.N) break;
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const uint32_t *w = &v[c][2 * j];
          uint64_t a = f32x2(w[0], w[1]), b = f32x2(w[2], w[3]);
          if (C::NV) {
            const float4 ci = *reinterpret_cast<const float4 *>(cinv + c * 32 + 2 * j);
            a = mul_f32x2(a, mul_f32x2(f2, f32x2(ci.x, ci.y)));
            b = mul_f32x2(b, mul_f32x2(f2, f32x2(ci.z, ci.w)));
          } else if (p.row_weight) {
            a = mul_f32x2(a, f2);
            b = mul_f32x2(b, f2);
          }
          pk[j] = pack_bf16x2_u64(a);
          pk[j + 1] = pack_bf16x2_u64(b);
        }
        if (any_far) {
          const __nv_bfloat162 m = __float2bfloat162_rn(far);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&pk[j]), m);
            pk[j] = *reinterpret_cast<const uint32_t *>(&y);
          }
        }
        if (whole) {
          if (lane == 0) bulk_wait_read<0>();  // the buffer's last store has read it
          __syncwarp();
          // 64-byte rows, 16-byte unit j of row r at unit j ^ (r / 2 % 4) (the 64-byte swizzle)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, buf, col0 + c * 32, row0);
            bulk_commit();
          }
        } else if (store) {
          if (p.vec32) {  // whole 32-byte sectors (N % 16 == 0)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (col0 + c * 32 + j * 16 < p.N) store_32b(o + c * 32 + j * 16, &pk[8 * j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (col0 + c * 32 + j * 8 < p.N)
                *reinterpret_cast<uint4 *>(o + c * 32 + j * 8) =
                    make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          }
        }
      }
      __syncwarp();  // the column factors are read
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (*vabort && warp == 0 && lane == 0) {
    // wait for the copies this CTA armed, bounded
    for (int i = 0; i < nst && rank == 0; ++i) {
      const uint32_t armed = issued / nst + ((uint32_t)i < issued % nst ? 1u : 0u);
      if (armed) mbar_wait_drain(&S.full[i], (armed - 1) & 1);
    }
    // pair: copies of a CTA that the other's barriers never counted get far longer than a copy takes
    if constexpr (PAIR) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
    }
  }
  if constexpr (PAIR) cluster_sync();  // every MMA into either CTA's TMEM and every remote arrival is done
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 512);
    else tmem_dealloc(tmem_base, 512);
  }
  if constexpr (PAIR) cluster_sync();  // neither CTA leaves while the other may still address it
}

template <int FMT, bool PAIR, int NT>
int launch_fp4(const uint8_t *x, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, Fp4Params p, int64_t M, int bn,
               int sms, cudaStream_t s) {
  using C = F4Cfg<FMT, PAIR>;
  const int E = p.E, K = p.K, N = p.N;
  p.bn = bn;
  p.n_tiles = (N + bn - 1) / bn;
  p.a_rows = M < 128 ? (int)((M + 7) / 8 * 8) : 128;
  p.vec32 = N % 16 == 0 && ((uintptr_t)p.out & 31) == 0;
  p.stage_bytes = C::stage_bytes(p.a_rows, bn);
  // the MMA reads 128 A rows from a stage's start whatever the box holds: room behind the last stage
  const size_t fixed = 1024 + kF4EpiWarps * kF4Stage + sizeof(F4Shared) + (size_t)(128 - p.a_rows) * 128;
  int st = (int)((kF4Limit - fixed) / p.stage_bytes);
  if (st > kF4MaxStages) st = kF4MaxStages;
  p.stages = st;
  const size_t smem = fixed + (size_t)st * p.stage_bytes;
  const int W = fp4_words(FMT, K);
  CUtensorMap ta, tb, tsa, tsb, to;
  {
    const uint64_t d[2] = {(uint64_t)K / 2, (uint64_t)M}, str[1] = {(uint64_t)K / 2};
    const uint32_t box[2] = {128, (uint32_t)p.a_rows};
    if (!make_tensor_map(&ta, true, 2, x, d, str, box)) return MGEMM_ECUDA;
  }
  {
    const uint64_t d[3] = {(uint64_t)K / 2, (uint64_t)N, (uint64_t)E};
    const uint64_t str[2] = {(uint64_t)K / 2, (uint64_t)N * (K / 2)};
    const uint32_t box[3] = {128, (uint32_t)(PAIR ? bn / 2 : bn), 1};
    if (!make_tensor_map(&tb, true, 3, w, d, str, box)) return MGEMM_ECUDA;
  }
  // scales: 512-byte word tiles as 256 two-byte elements, {256, words, row tiles}
  auto sf_map = [&](CUtensorMap *m, const uint8_t *base, int64_t tiles, int box_tiles) {
    const uint64_t d[3] = {256, (uint64_t)W, (uint64_t)tiles};
    const uint64_t str[2] = {512, (uint64_t)W * 512};
    const uint32_t box[3] = {256, (uint32_t)C::WPS, (uint32_t)box_tiles};
    return make_tensor_map(m, false, 3, base, d, str, box, false);
  };
  if (!sf_map(&tsa, sx, mgemm_colwise_ld(M, E) / 128, 1)) return MGEMM_ECUDA;
  if (!sf_map(&tsb, sw, (int64_t)E * ((N + 127) / 128), NT)) return MGEMM_ECUDA;
  {  // the output rows (a scattered output is stored directly: the map is then not used)
    const uint64_t d[2] = {(uint64_t)N, (uint64_t)(p.row_map ? p.map_limit > 0 ? p.map_limit : 1 : M)};
    const uint64_t str[1] = {(uint64_t)N * 2};
    const uint32_t box[2] = {32, 32};
    if (!make_tensor_map(&to, false, 2, p.out, d, str, box, true, true)) return MGEMM_ECUDA;
  }
  static bool attr_done[64] = {};
  int dev = 0;
  int rc = cuda_rc(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc) return rc;
  if (dev < 0 || dev >= 64) return MGEMM_EINVAL;
  if (!attr_done[dev]) {
    rc = cuda_rc(cudaFuncSetAttribute(fp4_gemm_kernel<FMT, PAIR, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)kF4Limit),
                 "cudaFuncSetAttribute");
    if (rc) return rc;
    cudaFuncAttributes attr;
    rc = cuda_rc(cudaFuncGetAttributes(&attr, fp4_gemm_kernel<FMT, PAIR, NT>), "cudaFuncGetAttributes");
    if (rc) return rc;
    if (attr.numRegs != kF4Regs) {  // see FEW_REGS
      note_error("mgemm_fwd_fp4: its kernel's registers a thread are not those its warps share out", attr.numRegs);
      return MGEMM_ECUDA;
    }
    attr_done[dev] = true;
  }
  const int64_t groups = M < E ? M : E;
  const int64_t upper = PAIR ? 2 * ((M + 255) / 256 + groups) * p.n_tiles : ((M + 127) / 128 + groups) * p.n_tiles;
  const int64_t cap = PAIR ? sms / 2 * 2 : sms;
  const unsigned grid = (unsigned)(upper < cap ? upper : cap);
  return launch_pdl(fp4_gemm_kernel<FMT, PAIR, NT>, dim3(grid), dim3(kF4Threads), smem, s, PAIR ? 2u : 1u,
                    PAIR ? "mgemm_fwd_fp4 launch (CTA pairs)" : "mgemm_fwd_fp4 launch", ta, tb, tsa, tsb, to, p);
}

// The tiles of h rows that a group of about `rows` rows takes on average (its size anywhere within an eighth of that).
double tiles_of(double rows, int h) {
  auto sum = [h](double v) {  // the integral of ceil(n / h) up to v
    const double k = floor(v / h);
    return h * k * (k + 1) / 2 + (v - k * h) * (k + 1);
  };
  const double lo = 0.875 * rows, hi = 1.125 * rows;
  return (sum(hi) - sum(lo)) / (hi - lo);
}

// How a product is tiled: columns per tile, and whether CTA pairs compute 256 rows of them.
struct F4Form {
  int bn;
  bool pairs;
};
template <int FMT>
F4Form fp4_form(int64_t M, int K, int N, int E, int sms) {
  const int64_t groups = M < E ? M : E;
  const double rows = (double)M / groups;
  auto rounds = [&](double row_tiles, int bn, int places) {
    return ceil(groups * row_tiles * ((N + bn - 1) / bn) / places);
  };
  // Columns per tile: the fewest rounds of tiles over the SMs, weighted by the bytes of a stage (A's rows, the
  // columns and their scales); wider at equal cost (fewer reads of A).  1024 rows in 8 groups of about 128 are 12
  // row tiles, not 8: 256 columns, 29.7 us; at 8 it would be 192 and 31.8.
  const int a_rows = M < 128 ? (int)M : 128;
  int bn = 256;
  double best = -1;
  for (int c : {256, 192, 128, 64}) {
    const double cost = rounds(tiles_of(rows, 128), c, sms) * (F4Cfg<FMT, false>::stage_bytes(a_rows, c) + 2048);
    if (best < 0 || cost < best) {
      best = cost;
      bn = c;
    }
  }
  // Pairs where fewer bytes pass through shared memory with them, in with the copies and out to the MMAs, 2^18 more
  // counted for their start and end.  Groups of 144, 192 and 256 rows, 8 of 6400 x 4096: 30.6, 31.4 and 37.4 us in
  // pairs, 35.8, 36.4 and 44.5 not; 5 of 1000 x 8192: 17.4, 17.9 and 18.4 in pairs, 15.7, 16.0 and 16.2 not.
  bool pairs = false;
  if (rows >= 128) {
    const double kb2 = (K + 255) / 256 * 2;
    const int pair_bn = N > 128 ? 256 : 128;
    const double one = rounds(tiles_of(rows, 128), bn, sms) * F4Cfg<FMT, false>::stage_bytes(128, bn);
    const double two = rounds(tiles_of(rows, 256), pair_bn, sms / 2) * F4Cfg<FMT, true>::stage_bytes(128, pair_bn);
    pairs = kb2 * two + (1 << 18) < kb2 * one;
  }
  return {pairs ? N > 128 ? 256 : 128 : bn, pairs};
}

template <int FMT>
int launch_fp4(const uint8_t *x, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, const Fp4Params &p, int64_t M,
               int sms, cudaStream_t s) {
  const F4Form form = fp4_form<FMT>(M, p.K, p.N, p.E, sms);
  if (form.pairs)
    return form.bn > 128 ? launch_fp4<FMT, true, 2>(x, sx, w, sw, p, M, form.bn, sms, s)
                         : launch_fp4<FMT, true, 1>(x, sx, w, sw, p, M, form.bn, sms, s);
  return form.bn > 128 ? launch_fp4<FMT, false, 2>(x, sx, w, sw, p, M, form.bn, sms, s)
                       : launch_fp4<FMT, false, 1>(x, sx, w, sw, p, M, form.bn, sms, s);
}

bool a16(const void *p) { return ((uintptr_t)p & 15) == 0; }

int fwd_fp4(int fmt, const uint8_t *x, const uint8_t *sx, const uint8_t *w, const uint8_t *sw, const Fp4Params &p,
            int64_t M, cudaStream_t s) {
  const int rc = ensure_context();
  if (rc) return rc;
  const int sms = sm_count_cached();
  if (sms <= 0) return MGEMM_ECUDA;
  return fmt == MGEMM_NVFP4 ? launch_fp4<MGEMM_NVFP4>(x, sx, w, sw, p, M, sms, s)
                            : launch_fp4<MGEMM_MXFP4>(x, sx, w, sw, p, M, sms, s);
}

// The sizes and pointers both entry points take (out is checked by each).
int fp4_checks(int fmt, const uint8_t *w, const uint8_t *sw, const float *rw, const void *out, int64_t M, int K, int N,
               int E) {
  if (!fp4_format(fmt) || E < 1) return MGEMM_EINVAL;
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (M < 0 || M >= (int64_t(1) << 31) || K <= 0 || N <= 0 || (int64_t)E * N >= (int64_t(1) << 31)) return MGEMM_EINVAL;
  if (!w || !sw || (M > 0 && !out) || (fmt == MGEMM_NVFP4 && !rw)) return MGEMM_EINVAL;
  if (K % 32 || N % 8) return MGEMM_EALIGN;
  if (!a16(w) || !a16(sw) || !a16(out) || ((uintptr_t)rw & 3)) return MGEMM_EALIGN;
  return MGEMM_OK;
}

struct Workspace {
  size_t args, codes, sf, rows, bytes;
};
Workspace fp4_workspace(int fmt, int64_t M, int K, int E) {
  Workspace w{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  w.codes = up(mgemm_args_bytes(E));
  w.sf = w.codes + up((size_t)M * (K / 2));
  w.rows = w.sf + up((size_t)mgemm_fp4_scale_bytes(fmt, mgemm_colwise_ld(M, E), K));
  w.bytes = w.rows + up(fmt == MGEMM_NVFP4 ? (size_t)M * 4 : 0);
  return w;
}

}  // namespace
}  // namespace mgemm

using namespace mgemm;

extern "C" int mgemm_fwd_fp4(const void *args, int fmt, const uint8_t *x, const uint8_t *sx, const float *rx,
                             const uint8_t *w, const uint8_t *sw, const float *rw, void *out, const int32_t *row_map,
                             int64_t map_limit, const float *row_weight, int64_t M, int K, int N, int E,
                             mgemm_stream_t stream) {
  int rc = fp4_checks(fmt, w, sw, rw, out, M, K, N, E);
  if (rc) return rc;
  if (!args || !x || !sx || (fmt == MGEMM_NVFP4 && !rx) || map_limit < 0) return MGEMM_EINVAL;
  if (!a16(args) || !a16(x) || !a16(sx) || ((uintptr_t)rx & 3) || ((uintptr_t)row_map & 3) || ((uintptr_t)row_weight & 3))
    return MGEMM_EALIGN;
  if (M == 0) return MGEMM_OK;
  Fp4Params p{};
  p.args = (const uint8_t *)args;
  p.rx = rx;
  p.rw = rw;
  p.out = (__nv_bfloat16 *)out;
  p.row_map = row_map;
  p.map_limit = map_limit;
  p.row_weight = row_weight;
  p.K = K;
  p.N = N;
  p.E = E;
  return fwd_fp4(fmt, x, sx, w, sw, p, M, (cudaStream_t)stream);
}

extern "C" int mgemm_fp4_form(int fmt, int64_t M, int K, int N, int E, int sms, int *pairs) {
  if (!fp4_format(fmt) || M < 1 || M >= (int64_t(1) << 31) || K <= 0 || N <= 0 || E < 1 || !pairs) return MGEMM_EINVAL;
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (sms <= 0) sms = sm_count_cached();
  if (sms <= 0) return MGEMM_ECUDA;
  const F4Form form = fmt == MGEMM_NVFP4 ? fp4_form<MGEMM_NVFP4>(M, K, N, E, sms) : fp4_form<MGEMM_MXFP4>(M, K, N, E, sms);
  *pairs = form.pairs;
  return form.bn;
}

extern "C" int64_t mgemm_gmm_fp4_workspace_bytes(int fmt, int64_t M, int K, int E) {
  if (!fp4_format(fmt) || M < 0 || M >= (int64_t(1) << 31) || K <= 0 || K % 32 || E < 1 || E > MGEMM_MAX_EXPERTS) return -1;
  return (int64_t)fp4_workspace(fmt, M, K, E).bytes;
}

extern "C" int mgemm_gmm_fp4(const int64_t *group_sizes, int E, int fmt, const void *x, int64_t ld_x, const uint8_t *w,
                             const uint8_t *sw, const float *rw, void *out, int64_t M, int K, int N, void *workspace,
                             int64_t workspace_bytes, mgemm_stream_t stream) {
  int rc = fp4_checks(fmt, w, sw, rw, out, M, K, N, E);
  if (rc) return rc;
  if (!group_sizes || !workspace || ld_x < K || (M > 0 && !x)) return MGEMM_EINVAL;
  if (((uintptr_t)group_sizes & 7) || !a16(workspace) || !a16(x) || ld_x % 8) return MGEMM_EALIGN;
  if (M == 0) return MGEMM_OK;
  const Workspace ws = fp4_workspace(fmt, M, K, E);
  if (workspace_bytes < (int64_t)ws.bytes) return MGEMM_EINVAL;
  uint8_t *b = (uint8_t *)workspace;
  float *rx = fmt == MGEMM_NVFP4 ? (float *)(b + ws.rows) : nullptr;
  // Fill and cast in one launch for up to 2^26 elements: 2 us less for a few rows (256 x 4096: 11.6, 13.6 us in
  // two); past that the scans in front of every CTA's rows cost more (32768 x 4096: 102, 98 in two).
  if (E <= kFp4FillMaxE && M * K < (int64_t(1) << 26)) {
    rc = fp4_fill_quant_rows(group_sizes, E, M, b, (const __nv_bfloat16 *)x, K, ld_x, fmt, b + ws.codes, b + ws.sf, rx,
                             (cudaStream_t)stream);
  } else {
    rc = mgemm_fill_args(group_sizes, E, M, b, stream);
    if (!rc)
      rc = mgemm_quant_fp4_rows(b, E, M, x, M, K, ld_x, nullptr, 0, 1, 0, fmt, b + ws.codes, b + ws.sf, rx, stream);
  }
  if (rc) return rc;
  Fp4Params p{};
  p.args = b;
  p.rx = rx;
  p.rw = rw;
  p.out = (__nv_bfloat16 *)out;
  p.K = K;
  p.N = N;
  p.E = E;
  p.M = M;
  if (E <= kFp4FillMaxE && (M < E ? M : E) <= kF4Groups) p.sizes = group_sizes;  // (launched behind the cast)
  return fwd_fp4(fmt, b + ws.codes, b + ws.sf, w, sw, p, M, (cudaStream_t)stream);
}
