// mgemm_quant_int4_groups / mgemm_gmm_int4: weights in 4 bits with a bf16 scale (and a
// whole zero point) for 32, 64 or 128 elements of a row, and the grouped product of few
// bf16 token rows with them.
//
//   out[r, n] = sum over groups g of s[e, n, g] sum_{k in g} (q[e, n, k] - z[e, n, g]) x[r, k]
//
// The codes become bf16 whole numbers over 64 ((q - z) / 64, exact), a group's products are
// summed in float32 by mma.sync with the weights as its 16 rows and the tokens as its 8
// columns, and the scale multiplies that sum: no rounding but float32's.
//
// No unit is full: 16 rows at 16 experts of 8192 x 5120 in groups of 128 with zero points
// take 77 us, the stream of their 352 MB 52, and 325 warp instructions for 32 rows by 128
// elements 43 at full issue (152 unpack, 16 are MMAs, 18 load from shared memory; the rest
// copies, scales, addresses and loops).  65% of the issue slots and 53% of the logic pipe are
// used, by 14 warps an SM that wait for their own chains: load from shared memory, unpack,
// MMA, scaled sum.  (A form on tcgen05, with unpacked weights through shared memory and every
// group's sums back from tensor memory, took 94 us for 128 rows over 8 experts of 6400 x 4096
// when this one took 68; what bounded it was not found, and it had not the scale windows,
// dropped columns and balanced passes that brought this one to 52.)
//
// A CTA's warps form crews of WK teams of WN warps.  A crew has a tile: WN x MT x 16 rows of
// weights by NT x 8 tokens; its teams take the contraction's steps of 128 in turn and add up
// at the end.  Codes and tokens come through rings of kStages steps, one for a team
// (cp.async).  In a step's 32-element chunk c of a row, the lane t of a quad takes the 8 codes
// of word t and the tokens' matching 8 values: two MMAs, each over 4 elements of each lane.
#include <type_traits>

#include "common.cuh"

namespace mgemm {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kStep = 128;      // contraction elements of a step
constexpr int kParts = 1024, kMaxParts = MGEMM_MAX_EXPERTS + kParts;  // (parts: ceil(rows / p.rows) of each group)

struct GmmParams {
  const int64_t *sizes;
  const __nv_bfloat16 *x;
  const uint8_t *codes;
  const uint16_t *scales;  // bf16 bits
  const uint8_t *zeros;    // or NULL: 8
  __nv_bfloat16 *out;
  int *status;
  int64_t ld_x;
  int E, M, K, N;
  int rows;  // of a group that make a tile: a pass's tokens, or a multiple of them
};

// d (+)= a b for a bf16 [16 x 16] (rows g, g + 8), b bf16 [16 x 8], float32 sums
__device__ __forceinline__ void mma16816(float (&d)[4], bool add, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(add ? d[0] : 0.f), "f"(add ? d[1] : 0.f), "f"(add ? d[2] : 0.f),
        "f"(add ? d[3] : 0.f));
}

// Codes to bf16.  Bits 0 .. 7 of a bf16 stand for their whole number times 2^-133 (subnormals, and the first normals,
// which have the same step), so a pair of nibbles needs neither a shift to bit 0 nor an exponent: masked, it is q 2^-133
// or, from the upper half of a byte, q 2^-129, and one fused multiply-add makes it (q - z) / 64, exactly.  (The 64 is
// put back into the sums.  5 instructions of the logic pipe, the fullest one, for 8 codes; with a shift and 128's
// exponent for each pair there were 7, and 16 rows at 16 experts of 8192 x 5120 took 85 us instead of 77.)
__device__ __forceinline__ __nv_bfloat162 bits(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); }
constexpr uint32_t kLow = 0x7F007F00u, kHigh = 0x7D007D00u;  // 2^127 and 2^123, twice
template <uint32_t MASK, uint32_t FACTOR>
__device__ __forceinline__ uint32_t code_pair(uint32_t word, uint32_t zero2) {
  const __nv_bfloat162 d = __hfma2(bits(word & MASK), bits(FACTOR), bits(zero2));
  return *reinterpret_cast<const uint32_t *>(&d);
}
// - z / 64, twice
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  const __nv_bfloat162 d = __hmul2(bits(z * 0x00010001u), bits(kLow ^ 0x80008000u));
  return *reinterpret_cast<const uint32_t *>(&d);
}

// NT x 8 tokens by WN warps of MT x 16 weight rows, WK teams to a tile.
template <int NT, int MT, int WN, int WK>
struct Tile {
  static constexpr int kWarps = WN * WK > 8 ? WN * WK : 8, kThreads = kWarps * 32;
  static constexpr int kTeams = kWarps / WN, kCrews = kTeams / WK;
  static constexpr int kWarpRows = MT * 16;
  static constexpr int kCtas = NT * MT <= 4 && kWarps == 8 ? 2 : 1;     // on an SM
  static constexpr int BN = WN * kWarpRows;
  static constexpr int kCodeBytes = BN * (kStep / 2), kTokenBytes = NT * 8 * kStep * 2;
  static constexpr int kStageBytes = kCodeBytes + kTokenBytes;
  static constexpr int kStagesFit = (kCtas == 2 ? 104 : 200) * 1024 / (kTeams * kStageBytes), kStages = kStagesFit < 5 ? kStagesFit : 5;
  static constexpr int kRingBytes = kStages * kStageBytes;  // of one team
  static_assert(kTeams + kCrews < 16, "named barriers");
  // a team's partial sums take the place of the step it used last
  static constexpr int kRow = BN + (NT * 8 * (BN + 4) * 4 <= kStageBytes ? 4 : 0);  // floats from token to token (4 more: banks)
  static_assert(NT * 8 * kRow * 4 <= kStageBytes, "partial sums fit a stage");
  static constexpr int kSmem = kTeams * kRingBytes;
};

template <int NT, int MT, int WN, int WK, int GROUP>
__global__ void __launch_bounds__(Tile<NT, MT, WN, WK>::kThreads, Tile<NT, MT, WN, WK>::kCtas) gmm_int4_kernel(const GmmParams p) {
  using T = Tile<NT, MT, WN, WK>;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStages = T::kStages, kWarpRows = T::kWarpRows, kWarps = T::kWarps;
  __shared__ int act_start[kMaxParts + 1];  // (the parts' rows follow each other)
  __shared__ uint16_t act_expert[kMaxParts];
  __shared__ int warp_rows[kWarps], warp_active[kWarps], sums_at[kWarps];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3, row8 = lane >> 2;

  // the groups' parts, in order: as few as p.rows rows allow, alike but for a multiple of 8 (30 rows: 16 and 14, not 24
  // and 6, whose pass takes the same two columns).  Thread i looks at sizes 4 i .. 4 i + 3
  int n_active;
  {
    int rows[4], part[4], sum = 0, active = 0;
    bool negative = false, large = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = threadIdx.x * 4 + j;
      const int64_t v = e < p.E ? __ldg(p.sizes + e) : 0;
      negative |= v < 0;
      large |= v > p.M;
      rows[j] = v < 0 || v > p.M ? 0 : (int)v;
      sum = min(sum + rows[j], 0x3FFFFFFF);  // (M is below 2^24: more is refused below)
      part[j] = p.rows;
      int parts = rows[j] > 0;
      if (rows[j] > p.rows) {
        parts = (rows[j] + p.rows - 1) / p.rows;
        part[j] = ((rows[j] + parts - 1) / parts + 7) & ~7;
      }
      active += parts;
    }
    int a = sum, b = active;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, a, o), v = __shfl_up_sync(kFull, b, o);
      if (lane >= o) a = min(a + u, 0x3FFFFFFF), b += v;
    }
    if (lane == 31) warp_rows[warp] = a, warp_active[warp] = b;
    const int bad = __syncthreads_or(negative ? 1 : 0);
    const int over = __syncthreads_or(large ? 1 : 0);
    int start = a - sum, at = b - active;
    int total = 0;
    n_active = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) start += warp_rows[w], at += warp_active[w];
      total = min(total + warp_rows[w], 0x3FFFFFFF);
      n_active += warp_active[w];
    }
    if (bad || over || total != p.M) {
      if (p.status && threadIdx.x == 0 && blockIdx.x == 0)
        *p.status = bad ? MGEMM_STATUS_NEGATIVE_SIZE : MGEMM_STATUS_SUM_MISMATCH;
      return;
    }
    if (p.status && threadIdx.x == 0 && blockIdx.x == 0) *p.status = MGEMM_STATUS_OK;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      for (int r = 0; r < rows[j]; r += part[j], ++at)
        act_start[at] = start + r, act_expert[at] = (uint16_t)(threadIdx.x * 4 + j);
      start += rows[j];
    }
    if (threadIdx.x == 0) act_start[n_active] = p.M;
    __syncthreads();
  }
  auto rows_of_group = [&](int a) { return act_start[a + 1] - act_start[a]; };

  const int team_id = warp / WN, member = warp % WN, in_team = member * 32 + lane;
  const int crew = team_id / WK, team = team_id % WK;  // a crew's teams share its tile
  constexpr int kTeam = WN * 32, kCrew = WK * kTeam;   // threads
  const int in_crew = threadIdx.x - crew * kCrew;
  uint8_t *ring = smem + team_id * T::kRingBytes;
  const int steps = (p.K + kStep - 1) / kStep, tiles_n = (p.N + T::BN - 1) / T::BN;
  const int tiles = n_active * tiles_n, first_tile = blockIdx.x + gridDim.x * crew, tile_step = gridDim.x * T::kCrews;
  const int groups = p.K / GROUP;
  auto team_sync = [&]() {
    if constexpr (WN == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + team_id), "r"(kTeam) : "memory");
  };
  auto crew_sync = [&]() {
    if constexpr (T::kCrews == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(T::kTeams + 1 + crew), "r"(kCrew) : "memory");
  };

  // What is loaded next: step l_step of rows l_first .. of tile l_tile.  Absent weight rows and tokens keep what the
  // slot held before (their products stay in their own row or column, which is not stored); tokens past K are zeros.
  int l_tile = first_tile, l_m0 = 0, l_step = team, l_slot = 0, l_rows = 0, l_turns = 0, l_n = 0;
  bool l_whole = false;
  const uint8_t *l_codes = nullptr;
  const __nv_bfloat16 *l_x = nullptr;
  constexpr int kCodeRow = kTeam / 4, kTokenRow = kTeam / 16;  // rows that a team's threads copy at a time
  const int code_row = in_team >> 2, code_at = in_team & 3, token_row = in_team >> 4, token_at = in_team & 15;
  const uint32_t code_dst = smem_u32(ring) + code_row * 64 + ((code_at ^ ((code_row >> 1) & 3)) << 4);
  const uint32_t token_dst = smem_u32(ring) + T::kCodeBytes + token_row * 256 + ((token_at ^ ((token_row & 1) << 2)) << 4);
  uint32_t code_off[T::BN / kCodeRow];  // (K is at most 2^26: 128 rows of K / 2 bytes stay below 2^32)
#pragma unroll
  for (int i = 0; i < T::BN / kCodeRow; ++i) code_off[i] = (uint32_t)(i * kCodeRow) * (uint32_t)(p.K / 2);
  const int64_t token_off = kTokenRow * p.ld_x;
  auto aim = [&]() {  // at the rows of the tile and pass
    const int a = l_tile / tiles_n, n0 = (l_tile - a * tiles_n) * T::BN;
    const int rows = rows_of_group(a) - l_m0;
    l_rows = rows - token_row;
    l_turns = (rows + kTokenRow - 1) / kTokenRow;
    l_n = p.N - n0 - code_row;
    l_whole = n0 + T::BN <= p.N;
    l_codes = p.codes + ((int64_t)act_expert[a] * p.N + n0 + code_row) * (p.K / 2) + code_at * 16 + l_step * (kStep / 2);
    l_x = p.x + (int64_t)(act_start[a] + l_m0 + token_row) * p.ld_x + token_at * 8 + l_step * kStep;
  };
  if (steps <= team) l_tile = tiles;  // (this team has no steps at all)
  if (l_tile < tiles) aim();
  auto load_step = [&]() {
    if (l_tile < tiles) {
      const uint32_t ring_at = l_slot * T::kStageBytes;
      const int left = p.K - l_step * kStep;
      // (nothing of the tile or the step is absent: no test for each copy.  64 weight rows a warp: 78.5 us without, 76.3; of 32
      // the second path costs more than it saves, 8.6 us against 9.2 for 61 rows of 1440 x 1000)
      if (MT == 4 && l_whole && left >= kStep) {
#pragma unroll
        for (int i = 0; i < T::BN / kCodeRow; ++i) cp_async16(code_dst + ring_at + i * kCodeRow * 64, l_codes + code_off[i], 16);
#pragma unroll
        for (int i = 0; i < NT * 8 / kTokenRow; ++i) {
          if (i >= l_turns) break;
          if (i * kTokenRow < l_rows) cp_async16(token_dst + ring_at + i * kTokenRow * 256, l_x + i * token_off, 16);
        }
      } else {
        if (code_at * 32 < left) {
#pragma unroll
          for (int i = 0; i < T::BN / kCodeRow; ++i)
            if (i * kCodeRow < l_n) cp_async16(code_dst + ring_at + i * kCodeRow * 64, l_codes + code_off[i], 16);
        }
        const uint32_t bytes = token_at * 8 < left ? 16 : 0;
#pragma unroll
        for (int i = 0; i < NT * 8 / kTokenRow; ++i)
          if (i * kTokenRow < l_rows) cp_async16(token_dst + ring_at + i * kTokenRow * 256, bytes ? l_x + i * token_off : p.x, bytes);
      }
      l_codes += WK * (kStep / 2);
      l_x += WK * kStep;
      l_step += WK;
      if (l_step >= steps) {
        l_step = team, l_m0 += NT * 8;
        if (l_m0 >= rows_of_group(l_tile / tiles_n)) l_m0 = 0, l_tile += tile_step;
        if (l_tile < tiles) aim();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    l_slot = l_slot + 1 == kStages ? 0 : l_slot + 1;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load_step();

  // Scales (bf16 bits) and zero points of kWindow of the warp's steps ahead, 4 groups of each row: lane 4 r + q has
  // group q of the rows r + 8 i, so that a load meets 8 rows.  (A row a lane, each step, is 32 rows a load: the first
  // cache's tags, not the codes, bounded the kernel then: 81 us against 42 for 8 rows at 8 experts of 4096 x 6400 in
  // groups of 32.)  They are left as they come: whatever is made of them at once would be waited for.
  constexpr int kGroups = kStep / GROUP, kWindow = 4 / kGroups;  // groups of a step, steps of a window
  uint32_t next_s[2 * MT], next_z[2 * MT];
  const uint16_t *s_at = nullptr;
  const uint8_t *z_at = nullptr;
  int s_n = 0;
  auto aim_scales = [&](int tile) {
    const int a = tile / tiles_n, n = (tile - a * tiles_n) * T::BN + member * kWarpRows + row8;
    const int64_t at = ((int64_t)act_expert[a] * p.N + n) * groups;
    s_at = p.scales + at, z_at = p.zeros + at, s_n = p.N - n;
  };
  auto fetch = [&](int step) {
    const int g = (step + quad / kGroups * WK) * kGroups + quad % kGroups;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      const bool in = i * 8 < s_n && g < groups;
      next_s[i] = in ? __ldg(s_at + i * 8 * groups + g) : 0u;
      next_z[i] = in && p.zeros ? __ldg(z_at + i * 8 * groups + g) : 8u;
    }
  };
  if (first_tile < tiles && team < steps) aim_scales(first_tile), fetch(team);

  int slot = 0;
  for (int tile = first_tile; tile < tiles; tile += tile_step) {
    const int a = tile / tiles_n, n0 = (tile - a * tiles_n) * T::BN, rows_of = rows_of_group(a);
    for (int m0 = 0; m0 < rows_of; m0 += NT * 8) {
      const int live = min(rows_of - m0, NT * 8);
      float acc[MT][NT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.f;
      uint32_t sz[2 * MT];  // of this window: bf16 in the upper half, the zero point below
      int turn = 0;         // the step's place in it
      for (int step = team; step < steps; step += WK, turn = turn + 1 == kWindow ? 0 : turn + 1) {
        if (turn == 0) {
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) sz[i] = next_s[i] << 16 | next_z[i];
          if (step + kWindow * WK < steps) {
            fetch(step + kWindow * WK);
          } else if (m0 + NT * 8 < rows_of) {
            fetch(team);
          } else if (tile + tile_step < tiles) {
            aim_scales(tile + tile_step);
            fetch(team);
          }
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        team_sync();
        load_step();  // (into the slot of the step before, which the team is done with)
        const uint8_t *codes = ring + slot * T::kStageBytes + member * kWarpRows * 64;
        const uint8_t *tokens = ring + slot * T::kStageBytes + T::kCodeBytes;
        slot = slot + 1 == kStages ? 0 : slot + 1;
        // (a pass whose last 8 token columns are empty leaves them out)
        auto work = [&](auto columns) {
          constexpr int kTiles = columns.value;
          float part[MT][kTiles][4];
          uint32_t zero[2 * MT];
          float scale[2 * MT];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c * 32 % GROUP == 0) {
#pragma unroll
              for (int i = 0; i < 2 * MT; ++i) {
                const uint32_t v = __shfl_sync(kFull, sz[i], (lane & ~3) + turn * kGroups + c * 32 / GROUP);
                zero[i] = zero_pair(v & 0xFFu);
                scale[i] = __uint_as_float(v & 0xFFFF0000u);
              }
            }
            uint32_t b[kTiles][4];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              const int m = j * 8 + row8;
              const uint4 w = *reinterpret_cast<const uint4 *>(tokens + m * 256 + (((c * 4 + quad) ^ ((m & 1) << 2)) << 4));
              b[j][0] = __byte_perm(w.x, w.z, 0x5410), b[j][1] = __byte_perm(w.x, w.z, 0x7632);
              b[j][2] = __byte_perm(w.y, w.w, 0x5410), b[j][3] = __byte_perm(w.y, w.w, 0x7632);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              const int r = i * 16 + row8;  // (r and r + 8 have the same swizzle: 8 >> 1 is 0 modulo 4)
              const uint32_t lo = *reinterpret_cast<const uint32_t *>(codes + r * 64 + ((c ^ ((r >> 1) & 3)) << 4) + quad * 4);
              const uint32_t hi = *reinterpret_cast<const uint32_t *>(codes + (r + 8) * 64 + ((c ^ ((r >> 1) & 3)) << 4) + quad * 4);
              constexpr uint32_t kL = 0x000F000Fu, kH = 0x00F000F0u;
              const uint32_t z0 = zero[2 * i], z1 = zero[2 * i + 1], lo8 = lo >> 8, hi8 = hi >> 8;
              const uint32_t a0 = code_pair<kL, kLow>(lo, z0), a1 = code_pair<kL, kLow>(hi, z1);
              const uint32_t a2 = code_pair<kH, kHigh>(lo, z0), a3 = code_pair<kH, kHigh>(hi, z1);
              const uint32_t a4 = code_pair<kL, kLow>(lo8, z0), a5 = code_pair<kL, kLow>(hi8, z1);
              const uint32_t a6 = code_pair<kH, kHigh>(lo8, z0), a7 = code_pair<kH, kHigh>(hi8, z1);
#pragma unroll
              for (int j = 0; j < kTiles; ++j) {
                mma16816(part[i][j], c * 32 % GROUP != 0, a0, a1, a2, a3, b[j][0], b[j][1]);
                mma16816(part[i][j], true, a4, a5, a6, a7, b[j][2], b[j][3]);
              }
            }
            if ((c + 1) * 32 % GROUP == 0) {
#pragma unroll
              for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) acc[i][j][k] = fmaf(part[i][j][k], scale[2 * i + k / 2], acc[i][j][k]);
                }
            }
          }
        };
        if (NT > 1 && live <= 8 * (NT - 1)) work(std::integral_constant<int, NT == 1 ? 1 : NT - 1>());
        else work(std::integral_constant<int, NT>());
      }
      // the teams' sums, [token][row of weights] each
      team_sync();  // (the team is done with the step)
      const int last = (slot == 0 ? kStages : slot) - 1;
      float *mine = reinterpret_cast<float *>(ring + last * T::kStageBytes) + member * kWarpRows;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) mine[(j * 8 + quad * 2 + (k & 1)) * T::kRow + i * 16 + (k / 2) * 8 + row8] = acc[i][j][k];
      if (lane == 0 && member == 0) sums_at[team_id] = team_id * T::kRingBytes + last * T::kStageBytes;
      crew_sync();
      for (int at = in_crew; at < live * (T::BN / 2); at += kCrew) {
        const int m = at / (T::BN / 2), n = at % (T::BN / 2) * 2;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < WK; ++k) {
          const float2 u = *reinterpret_cast<const float2 *>(smem + sums_at[crew * WK + k] + (m * T::kRow + n) * 4);
          v.x += u.x, v.y += u.y;
        }
        if (n0 + n < p.N)  // (N is even)
          *reinterpret_cast<__nv_bfloat162 *>(p.out + (int64_t)(act_start[a] + m0 + m) * p.N + n0 + n) =
              __floats2bfloat162_rn(v.x * 64.f, v.y * 64.f);
      }
      crew_sync();
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One warp for a row, 8 elements a lane: a group is 4, 8 or 16 lanes.
template <int GROUP>
__global__ void __launch_bounds__(256) quant_int4_groups_kernel(const __nv_bfloat16 *__restrict__ in, int64_t rows, int K,
                                                                int64_t ld_in, uint8_t *__restrict__ codes,
                                                                uint16_t *__restrict__ scales, uint8_t *__restrict__ zeros) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows; row += (int64_t)gridDim.x * 8) {
    for (int c0 = 0; c0 < K; c0 += 256) {
      const int c = c0 + lane * 8;
      const bool live = c < K;  // (K is a multiple of the group: its lanes agree)
      const uint4 u = live ? ldg_nc_v4(in + row * ld_in + c) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      float v[8], lo = 0.f, hi = 0.f, odd = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
        odd += v[i] * 0.f;  // NaN where a value is not finite
      }
#pragma unroll
      for (int o = 1; o < GROUP / 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
        odd += __shfl_xor_sync(kFull, odd, o);
      }
      // (halves: the range itself may pass float32)
      const float range = zeros ? __fdiv_rn(hi * 0.5f - lo * 0.5f, 7.5f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
      __nv_bfloat16 sb = __float2bfloat16_rn(range + odd);
      if (__bfloat162float(sb) == 0.f) sb = __float2bfloat16_rn(1.f);
      const float s = __bfloat162float(sb);
      const float z = zeros ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 8.f;
      uint32_t packed = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(v[i], s)) + z, 0.f), 15.f);
        packed |= (uint32_t)q << (4 * i);
      }
      if (live) {
        *reinterpret_cast<uint32_t *>(codes + row * (K / 2) + c / 2) = packed;
        if (lane % (GROUP / 8) == 0) {
          const int64_t at = row * (K / GROUP) + c / GROUP;
          scales[at] = __bfloat16_as_ushort(sb);
          if (zeros) zeros[at] = (uint8_t)z;
        }
      }
    }
  }
}

bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }

template <int NT, int MT, int WN, int WK, int GROUP>
int launch_gmm(GmmParams p, cudaStream_t s) {
  using T = Tile<NT, MT, WN, WK>;
  static bool attr_done[64] = {};
  int dev = 0, rc;
  if ((rc = cuda_rc(cudaGetDevice(&dev), "cudaGetDevice"))) return rc;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    if ((rc = cuda_rc(cudaFuncSetAttribute(gmm_int4_kernel<NT, MT, WN, WK, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem),
                      "cudaFuncSetAttribute")))
      return rc;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  const int sms = sm_count_cached();
  if (sms <= 0) return MGEMM_ECUDA;
  // A group's passes are tiles of their own, so that the CTAs' work differs by one pass at most: 160 rows
  // over 8 experts of 4096 x 6400 took 67 us with a group's passes one after another, 52 this way, 250 rows 95 and 82.
  // (16 rows at 16 experts of 8192 x 5120, one each: 76 and 76.7.)
  const int64_t tiles_n = (p.N + T::BN - 1) / T::BN;
  p.rows = NT * 8 * (1 + (p.M - 1) / (NT * 8 * kParts));
  if ((p.E + p.M / p.rows) * tiles_n >= int64_t(1) << 30) p.rows = p.M;
  const int64_t parts = p.E + p.M / p.rows, tiles = (p.M < parts ? p.M : parts) * tiles_n, most = T::kCtas * (int64_t)sms;
  const int64_t need = (tiles + T::kCrews - 1) / T::kCrews;
  return launch_pdl(gmm_int4_kernel<NT, MT, WN, WK, GROUP>, dim3((unsigned)(need < most ? need : most)), dim3(T::kThreads), T::kSmem, s, 1,
                    "mgemm_gmm_int4 launch", p);
}

// The variant, by the rows of a group that M and E make likely (their sizes are on the device) and the tiles there are at
// most.  Token columns of a pass, us: 8 experts of 4096 x 6400, groups of 64, with 8, 16 and 24 columns: 32 rows 33, 36, 46;
// 64 rows 44, 39, 46; 96 rows 43 with 16 columns, 47 with 24; 128 rows 56 and 51, 250 rows 95 and 82.  24 columns share tokens
// between 4 warps over 128 weight rows: with few tiles (255 rows of 3 experts of 2048 x 5120) they take 42, 16 columns 35.
// Teams of a tile: 8 where two CTAs an SM hold about all tiles (one row each of 4 experts of 2560 x 5120, 320 tiles: 12.7,
// 14.2 with 4; 16 columns, 32 rows of one expert of 4096 x 5120: 11.2, 17.6), else 4 (4 experts of 4096 x 5120, 512 tiles:
// 14.8, 15.7 with 8; 63 rows of one: 18.5, 19.8).  64 weight rows a warp where that leaves tiles enough: one row each of 4
// experts of 8192 x 5120 23.7 (32 weight rows 25.8), of 16 77 (80); of 4 experts of 4096 x 5120 15.2 (14.8).
template <int GROUP>
int launch_gmm_rows(const GmmParams &p, cudaStream_t s) {
  const int64_t active = p.M < p.E ? p.M : p.E, parts = (p.M + 15) / 16, tiles_n = (p.N + 31) / 32, sms = sm_count_cached();
  const int64_t tiles = active * tiles_n, few = 3 * sms;
  if (p.M <= 8 || p.M <= 4 * p.E) {
    if (tiles <= few) return launch_gmm<1, 2, 1, 8, GROUP>(p, s);
    return p.M <= p.E && tiles >= 6 * sms ? launch_gmm<1, 4, 1, 4, GROUP>(p, s) : launch_gmm<1, 2, 1, 4, GROUP>(p, s);
  }
  if (p.M > 12 * p.E && tiles >= 8 * sms) return launch_gmm<3, 2, 4, 3, GROUP>(p, s);
  return (active > parts ? active : parts) * tiles_n <= few ? launch_gmm<2, 2, 1, 8, GROUP>(p, s) : launch_gmm<2, 2, 1, 4, GROUP>(p, s);
}

constexpr int kMaxRows = 1 << 24, kMaxSide = 1 << 26, kMaxCastK = 1 << 30;  // (the cast's columns stay an int)

}  // namespace
}  // namespace mgemm

using namespace mgemm;

extern "C" int mgemm_quant_int4_groups(const void *in, int64_t rows, int K, int64_t ld_in, int group, uint8_t *codes,
                                       void *scales, uint8_t *zeros, mgemm_stream_t stream) {
  if (rows < 0 || K < 1 || K > kMaxCastK || ld_in < K || !group_ok(group)) return MGEMM_EINVAL;
  if (K % group) return MGEMM_EALIGN;
  if (rows == 0) return MGEMM_OK;
  if (!in || !codes || !scales) return MGEMM_EINVAL;
  if (((uintptr_t)in & 15) || ld_in % 8 || ((uintptr_t)codes & 15) || ((uintptr_t)scales & 1)) return MGEMM_EALIGN;
  const int sms = sm_count_cached();
  const int64_t need = (rows + 7) / 8, most = (int64_t)(sms > 0 ? sms : 152) * 32;
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)(need < most ? need : most)), dim3(256), 0, (cudaStream_t)stream, 1,
                      "mgemm_quant_int4_groups launch", (const __nv_bfloat16 *)in, rows, K, ld_in, codes, (uint16_t *)scales, zeros);
  };
  return group == 32 ? go(quant_int4_groups_kernel<32>) : group == 64 ? go(quant_int4_groups_kernel<64>) : go(quant_int4_groups_kernel<128>);
}

extern "C" int mgemm_gmm_int4(const int64_t *group_sizes, int E, const void *x, int64_t ld_x, const uint8_t *codes,
                              const void *scales, const uint8_t *zeros, int group, void *out, int64_t M, int K, int N,
                              int *status, mgemm_stream_t stream) {
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (E < 1 || M < 0 || M >= kMaxRows || K < 1 || N < 1 || ld_x < K || !group_ok(group)) return MGEMM_EINVAL;
  if (K > kMaxSide || N > kMaxSide || (int64_t)E * ((N + 31) / 32) >= (int64_t(1) << 30)) return MGEMM_EINVAL;
  if (K % group || N % 8) return MGEMM_EALIGN;
  if (M == 0) return MGEMM_OK;
  if (!group_sizes || !x || !codes || !scales || !out) return MGEMM_EINVAL;
  if (((uintptr_t)x & 15) || ld_x % 8 || ((uintptr_t)codes & 15) || ((uintptr_t)scales & 1) || ((uintptr_t)out & 15) ||
      ((uintptr_t)group_sizes & 7) || ((uintptr_t)status & 3))
    return MGEMM_EALIGN;
  const GmmParams p{group_sizes, (const __nv_bfloat16 *)x, codes, (const uint16_t *)scales, zeros, (__nv_bfloat16 *)out, status,
                    ld_x, E, (int)M, K, N, 0};
  cudaStream_t s = (cudaStream_t)stream;
  return group == 32 ? launch_gmm_rows<32>(p, s) : group == 64 ? launch_gmm_rows<64>(p, s) : launch_gmm_rows<128>(p, s);
}
