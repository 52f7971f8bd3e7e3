// Block-scaled E4M3 products (the format of fp8_block.cuh) on CTA pairs (tcgen05, sm_100a), and a
// warp-level form for experts with few rows.
//
// gemm (WGRAD = false): expert g's rows of a [rows, k] against its weight w[g] [n, k]:
//   out[r, c] = sum over 128-wide blocks kb of 2^(sa[r, kb] + sw[g, c / 128, kb])
//               * sum over k in kb of a[r, k] w[g, c, k]
// wgrad (WGRAD = true): both operands are transposed and K is the token: expert g owns the columns
//   128 start[g] .. 128 start[g + 1] of a_t [n, pitch] and b_t [k, pitch],
//   dw[g][r, c] = sum over its blocks tb of 2^(sa[tb, r] + sb[tb, c]) sum over t in tb of a_t b_t.
//
// The scales are applied by the tensor core (kind::mxf8f6f4, block_scale): one E8M0 byte per row of A and
// per row of B for each K = 32 instruction, read from TMEM. A TMEM word holds four bytes and the
// instruction names one of them, so a word serves four blocks of 128, and the four instructions of a block
// name the same byte. The fp32 accumulator of a tile stays in TMEM over the whole of K and is read once;
// each instruction's addition to it is cut off, not rounded, so that sums of one sign lose up to 2^-23 of
// themselves per 32 of K (3e-5 measured at K = 65,536). Steps of the Quartz gate|up product (24,576 rows,
// n 1,280, k 1,024, six experts): scales applied outside, a TMEM read and an fp32 multiply-add of every
// element per block of K, 59.6 us; in the tensor core, one block per scale word, 42.0; four blocks per
// word, read once per CTA, 36.0; streaming stores and the issuing thread's loop unrolled over a stage,
// 35.0.
//
// Clusters, stages and barriers are those of gemm_tc2.cuh: a tile of 256 x N (N = 16 .. 224) per CTA
// pair, CTA r loads rows 128 r .. of the A tile and half of the N rows of B, the leader issues
// M = 256 instructions. A stage holds one or two K blocks of 128 bytes (two by one 3-D box when K is a
// multiple of 128). Warps: 0-3 write the scales to TMEM (one per lane quarter: the instruction
// wants them in all four), 4-11 store finished tiles, 12 loads, 13 issues.
// TMEM: accumulator b in columns 256 b .. 256 b + N; the 32 columns from 256 b + 224 hold two of the
// four scale buffers, each for four blocks of K (4 columns for 128 rows of A, up to 7 for N of B; 32
// rows per column, one per lane).
//
// Bound: the operands' way from L2. A stage is 60 KB per CTA for about 950 cycles of the tensor core;
// three stages (all that shared memory holds) cycle in about 1,350, i.e. 45 bytes per cycle and SM (13
// TB/s in all), and a tile of four stages takes 6,000, 63% of them the tensor core's. Over the Quartz call
// with its rows on all 24 experts the pipe is 46% busy (39.5 us, 1.6 PFLOP/s, start-up and last stores
// included; 35.0 us on six experts). 131,072 x 1,536 x 1,536: 280 us on 48 experts, 268 on four (2.2 - 2.3
// PFLOP/s; 316 - 326 at the clocks of the power cap, 1,300 MHz, when repeated for seconds). One block per
// stage (43 us against 36), wider spacing of the tiles' K order (53 us: concurrent reads of one line no
// longer meet), narrower tiles (47.5 us at 192), L2 prefetches and stores by the TMA unit (37 us each)
// were slower. The weight gradient waits for its operands too (a tile is stored before its accumulator is
// needed again), beside 126 MB of fp32 stores: the Quartz gate|up gradient takes 49 - 54 us with the rows
// on all 24 experts (56 in expert order). On six of them (32 blocks of K each, the rest zeros) the same
// binary took 52 to 80 us in different processes, 61 and 72 on one machine, for a reason not found; the
// side that gives 24 tiles per expert instead of 25 as rows took 52 against 60.
#pragma once
#include "fp8_block.cuh"
#include "gemm_tc2.cuh"

namespace moe {

constexpr int F8G_N = 224;           // most columns of a tile
constexpr int F8G_THREADS = 14 * 32;
constexpr int F8G_STORE_WARPS = 8;
constexpr int F8G_STG = F8G_STORE_WARPS * 4096;  // staging of 32 rows x 128 bytes per storing warp
constexpr int F8G_SF_BUFS = 4;       // scale buffers ...
constexpr int F8G_SF_K = 4;          // ... of four K blocks
constexpr int F8G_SF_BYTES = 2 * 384 * 4;  // their words on the way to TMEM
// The wait for a finished tile lasts as long as the tile, without a bound on K (a weight gradient of 2^31
// rows has 2^24 blocks): its limit grows by four times what a block takes at the power cap's clocks.
constexpr uint64_t F8G_BLOCK_NS = 2000;

struct F8Gemm {
  CUtensorMap ma, mb;
  const int32_t *offsets;  // [E + 1] device, clamped to [0, rows]; null: one group of all rows
  const uint8_t *a_scale, *b_scale;
  void *out;
  long long rows;          // rows of a (gemm) or grouped rows (wgrad)
  int E, M, N, K;          // gemm: N = n, K = k; wgrad: M = n, N = k, K = blocks the buffers hold
  int tn;                  // columns per tile, a multiple of 16 up to F8G_N
  int nt;                  // column tiles
  unsigned nt_mul;         // floor(2^32 / nt) + 1: x / nt = umulhi(x, nt_mul), or one less (nt > 1)
  int per;                 // wgrad: tiles of a group, the same for all
  unsigned per_mul;
  int out_f32;
  int swap;                // wgrad: out is [E, N, M] (the operands changed places)
  int stages, kpb;
};

// Columns per tile: as few tiles as 224 columns allow, of about the same width.
inline int f8g_tile_n(int n) {
  const int tiles = (n + F8G_N - 1) / F8G_N;
  return ((n + tiles - 1) / tiles + 15) / 16 * 16;
}
inline size_t f8g_fixed_bytes(int E) {
  return 1024 + (size_t)F8G_STG + 256 + F8G_SF_BYTES + (size_t)(2 * E + 2 + F8G_THREADS / 32 + 1) * sizeof(int);
}
inline int f8g_stage_bytes(int tn, int kpb) { return (16384 + tn * 64) * kpb; }
constexpr int F8G_MAX_SMEM = 227 * 1024;
inline int f8g_stages(int E, int tn, int kpb) {
  const long long n = ((long long)F8G_MAX_SMEM - (long long)f8g_fixed_bytes(E)) / f8g_stage_bytes(tn, kpb);
  return n > 8 / kpb ? 8 / kpb : (int)n;
}

struct F8Tile {
  int g, m0, n0;
  int rows;         // rows of the group (gemm) or M (wgrad)
  long long row0;   // its first row in a (gemm) and in out
  int kofs, nk;     // first K block and K blocks
};

// x / d by its multiplier floor(2^32 / d) + 1 (any 32-bit x >= 0; d = 1 needs none).
__device__ __forceinline__ int f8_div(int x, int d, unsigned mul) {
  if (d == 1) return x;
  const int q = (int)__umulhi((unsigned)x, mul);
  return q * d > x ? q - 1 : q;
}

constexpr int F8G_SORT = 256;  // most groups that are put in order of K

// start[0 .. E]: the groups' first rows (gemm) or first K blocks (wgrad). gemm: tile counts scanned into
// prefix[0 .. E]. wgrad: every group has p.per tiles, and prefix[i] is the group at position i of the
// list, longest K first (its rank, counted against every other group); with the rounds dealt to the
// pairs in alternating direction the pairs' sums of K are nearly the same.
template <bool WGRAD>
__device__ __forceinline__ int f8_tile_prefix(const F8Gemm &p, int *prefix, int *start, int *tmp) {
  bool bad = false;
  for (int g = threadIdx.x; g <= p.E; g += blockDim.x) {
    const long long a = p.offsets ? expert_bound(p.offsets, g, p.rows) : g ? p.rows : 0;
    long long n = 0;
    if (g < p.E)
      n = (p.offsets ? expert_bound(p.offsets, g + 1, p.rows) : p.rows) - a;
    bad |= n < 0;
    if (WGRAD) {
      start[g] = (int)((n + QB - 1) / QB);
    } else {
      prefix[g] = (int)((n + 255) / 256) * p.nt;
      start[g] = (int)a;
    }
  }
  if (offsets_decrease(__syncthreads_or(bad))) return 0;
  if (WGRAD) {
    for (int g = threadIdx.x; g < p.E; g += blockDim.x) {
      int rank = g;
      if (p.E <= F8G_SORT) {
        rank = 0;
        for (int h = 0; h < p.E; ++h) rank += start[h] > start[g] || (start[h] == start[g] && h < g);
      }
      prefix[rank] = g;
    }
    __syncthreads();
    const int all = block_excl_scan_inplace(start, p.E, tmp);
    if (threadIdx.x == 0) start[p.E] = all;
    __syncthreads();
    return p.E * p.per;
  }
  const int total = block_excl_scan_inplace(prefix, p.E, tmp);
  if (threadIdx.x == 0) prefix[p.E] = total;
  __syncthreads();
  return total;
}

// The tile of a pair in round r (>= total: none in this round).
template <bool WGRAD> __device__ __forceinline__ int f8_tile(int r, int pair, int npairs) {
  return r * npairs + (WGRAD && (r & 1) ? npairs - 1 - pair : pair);
}

// The group of a tile and the tile's number in it.
template <bool WGRAD>
__device__ __forceinline__ int f8_group(const F8Gemm &p, int tile, const int *prefix, int *local) {
  if (WGRAD) {
    const int pos = f8_div(tile, p.per, p.per_mul);
    *local = tile - pos * p.per;
    return prefix[pos];
  }
  int lo = 0, hi = p.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  *local = tile - prefix[lo];
  return lo;
}
// Its K blocks (all that the issuing warp needs); 0 past the last tile.
template <bool WGRAD>
__device__ __forceinline__ int f8_blocks(const F8Gemm &p, int tile, int total, const int *prefix,
                                         const int *start) {
  if (tile >= total) return 0;
  if (!WGRAD) return (p.K + QB - 1) / QB;
  int local;
  const int g = f8_group<WGRAD>(p, tile, prefix, &local);
  return min(start[g + 1], p.K) - min(start[g], p.K);
}

template <bool WGRAD>
__device__ __forceinline__ F8Tile f8_decode(const F8Gemm &p, int tile, const int *prefix, const int *start) {
  F8Tile t;
  int local;
  t.g = f8_group<WGRAD>(p, tile, prefix, &local);
  const int row = f8_div(local, p.nt, p.nt_mul);
  t.m0 = row * 256;
  t.n0 = (local - row * p.nt) * p.tn;
  if (WGRAD) {
    t.rows = p.M;
    t.row0 = (long long)t.g * p.M;
    t.kofs = min(start[t.g], p.K);
    t.nk = min(start[t.g + 1], p.K) - t.kofs;
  } else {
    t.row0 = start[t.g];
    t.rows = start[t.g + 1] - start[t.g];
    t.kofs = 0;
    t.nk = (p.K + QB - 1) / QB;
  }
  return t;
}

// One K = 32 step with the E8M0 scales of A and B at TMEM addresses sfa, sfb.
__device__ __forceinline__ void f8_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Barrier of warps 0 .. 3: true when all 128 threads passed true.
__device__ __forceinline__ bool bar_all_128(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool f8_wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                             uint64_t limit, long long info) {
  bool ok = true;
  if (!mbar_try_wait(bar, parity)) ok = mbar_wait(bar, parity, abort_flag, limit, info);
  return __all_sync(0xffffffffu, ok);
}

template <bool WGRAD, int KPB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(F8G_THREADS, 1)
    gemm_fp8_block_kernel(const __grid_constant__ F8Gemm p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int NST = p.stages;
  const uint32_t b_bytes = (uint32_t)p.tn * 64;                     // this CTA's half of B, one K block
  const uint32_t a_stage = 16384u * KPB, stage_bytes = a_stage + b_bytes * KPB;
  // E4M3 operands, E8M0 scales, fp32 sums; the scales' byte (bits 4 and 29) is set per K block
  const uint32_t IDESC = (1u << 23) | ((uint32_t)p.tn >> 3 << 17) | (256u >> 4 << 24);

  const uint32_t raw = smem_u32(smem_raw);
  unsigned char *base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char *stg_all = base + (size_t)NST * stage_bytes;
  uint64_t *bars = (uint64_t *)(stg_all + F8G_STG);
  uint32_t *tmem_slot = (uint32_t *)(bars + 2 * NST + 5 + 2 * F8G_SF_BUFS);
  volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
  int *prefix = (int *)(stg_all + F8G_STG + 256 + F8G_SF_BYTES);
  int *start = prefix + p.E + 1;
  int *scan_tmp = start + p.E + 1;
  uint32_t *sf_words = (uint32_t *)(stg_all + F8G_STG + 256);  // [2][A 128, B 256]

  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + NST + s); };
  auto accf_bar = [&](int b) { return smem_u32(bars + 2 * NST + b); };
  auto acce_bar = [&](int b) { return smem_u32(bars + 2 * NST + 2 + b); };
  auto sff_bar = [&](int u) { return smem_u32(bars + 2 * NST + 4 + u); };
  auto sfe_bar = [&](int u) { return smem_u32(bars + 2 * NST + 4 + F8G_SF_BUFS + u); };
  const uint32_t drain_bar = smem_u32(bars + 2 * NST + 4 + 2 * F8G_SF_BUFS);

  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 2 * F8G_STORE_WARPS);
    }
    for (int u = 0; u < F8G_SF_BUFS; ++u) {
      mbar_init(sff_bar(u), 2 * 4);  // the scale warps of both CTAs
      mbar_init(sfe_bar(u), 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 13) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * 12) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&p.ma) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&p.mb) : "memory");
  }
  // all of this before the grid wait, so that it overlaps the previous kernel's end
  const KernelStamp stamp(WGRAD ? K_F8B_WGRAD : K_F8B_GEMM);
  const uint64_t limit = g_wait_limit_ns;
  tc_fence_before();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  stamp.started();
  griddep_launch();
  const int total = f8_tile_prefix<WGRAD>(p, prefix, start, scan_tmp);
  // scale buffer i (0 .. 3): 16 columns, 4 for A then up to 8 for B
  auto sf_col = [&](int i) { return tmem_base + (uint32_t)(256 * (i >> 1) + F8G_N + 16 * (i & 1)); };

  if (warp < 4) {
    // ------------------------------------------------------------ scales (both CTAs)
    // Unit: up to four K blocks of a tile. Each of the 128 threads reads the bytes of one row of A and
    // two of B, one unit ahead, and hands them to all four warps through shared memory.
    const int nkb = (p.K + QB - 1) / QB, nnb = (p.N + QB - 1) / QB;
    const bool word_a = !WGRAD && nkb % 4 == 0 && ((uintptr_t)p.a_scale & 3u) == 0;
    const bool word_b = !WGRAD && nkb % 4 == 0 && ((uintptr_t)p.b_scale & 3u) == 0;
    int round = 0, kb = 0, nk = 0;
    bool more = true;
    const uint8_t *src[3];
    bool on[3];
    auto enter = [&]() {  // the next tile that has K blocks
      F8Tile t;
      for (;; ++round) {
        more = (long long)round * npairs < total;
        if (!more) return;
        const int tile = f8_tile<WGRAD>(round, pair, npairs);
        if (tile >= total) continue;
        t = f8_decode<WGRAD>(p, tile, prefix, start);
        if (t.nk > 0) break;
      }
      kb = 0;
      nk = t.nk;
      const int r = t.m0 + (int)rank * 128 + tid;
      on[0] = r < t.rows;
      src[0] = WGRAD ? p.a_scale + (size_t)t.kofs * p.M + r : p.a_scale + (size_t)(t.row0 + r) * nkb;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = t.n0 + 128 * i + tid;
        on[1 + i] = 128 * i + tid < p.tn && c < p.N;
        src[1 + i] = WGRAD ? p.b_scale + (size_t)t.kofs * p.N + c
                           : p.b_scale + ((size_t)t.g * nnb + c / QB) * nkb;
      }
    };
    // the bytes of K blocks kb .. kb + 3 (as one word in w[.][0] where they are one aligned word);
    // rows and columns past the last, and K blocks past the last, read as 0
    uint32_t w[3][F8G_SF_K];
    auto fetch = [&]() {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int j = 0; j < F8G_SF_K; ++j) w[i][j] = 0u;
        if (!on[i]) continue;
        if (i == 0 ? word_a : word_b) {
          w[i][0] = __ldg((const uint32_t *)(src[i] + kb));
          continue;
        }
#pragma unroll
        for (int j = 0; j < F8G_SF_K; ++j)
          if (kb + j < nk) w[i][j] = __ldg(src[i] + (size_t)(kb + j) * (WGRAD ? (i == 0 ? p.M : p.N) : 1));
      }
    };
    enter();
    if (more) fetch();
    const uint32_t quarter = (uint32_t)(warp * 32) << 16;
    int unit = 0;
    uint32_t phase = 0;
    while (more) {
      uint32_t *mine = sf_words + (unit & 1) * 384;
#pragma unroll
      for (int i = 0; i < 3; ++i) mine[128 * i + tid] = w[i][0] | w[i][1] << 8 | w[i][2] << 16 | w[i][3] << 24;
      kb += F8G_SF_K;
      if (kb >= nk) {
        ++round;
        enter();
      }
      if (more) fetch();
      // released by the tensor core, and the words of all four warps written; all four leave together
      if (!bar_all_128(f8_wait_warp(sfe_bar(unit), phase ^ 1u, abort_flag, limit, INFO_WAIT_MMA_EMPTY))) break;
      tc_fence_after();
      uint32_t v[12];
#pragma unroll
      for (int i = 0; i < 12; ++i) v[i] = mine[32 * i + lane];
      tmem_st4(sf_col(unit) + quarter, v);
      tmem_st8(sf_col(unit) + 4 + quarter, v + 4);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta0(sff_bar(unit));
      if (++unit == F8G_SF_BUFS) { unit = 0; phase ^= 1u; }
    }
  } else if (warp == 12) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint32_t issued = 0, issued_parity = 0;  // bit s: stage s was filled, with that parity
      for (int r = 0; (long long)r * npairs < total && ok; ++r) {
        const int tile = f8_tile<WGRAD>(r, pair, npairs);
        if (tile >= total) continue;
        const F8Tile t = f8_decode<WGRAD>(p, tile, prefix, start);
        // CTA 1's 128 rows may hold none of the group: never stored, so not loaded (gemm_tc2.cuh)
        const bool a1_void = t.m0 + 128 >= t.rows;
        const uint32_t tx = 2 * stage_bytes - (a1_void ? a_stage : 0);
        const int a_row = (WGRAD ? 0 : (int)t.row0) + t.m0 + (int)rank * 128;
        const int b_row = (WGRAD ? 0 : t.g * p.N) + t.n0 + (int)rank * (p.tn / 2);
        for (int kb = 0; kb < t.nk; kb += KPB) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, limit, INFO_WAIT_MMA_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t sA = smem_u32(base + (size_t)stage * stage_bytes), sB = sA + a_stage;
          if (rank == 0) mbar_expect_tx(full_bar(stage), tx);
          if (KPB == 2) {
            if (rank == 0 || !a1_void)
              tma_load_3d_pair(sA, &p.ma, 0, a_row, t.kofs + kb, full_bar(stage));
            tma_load_3d_pair(sB, &p.mb, 0, b_row, t.kofs + kb, full_bar(stage));
          } else {
            if (rank == 0 || !a1_void)
              tma_load_2d_pair(sA, &p.ma, (t.kofs + kb) * QB, a_row, full_bar(stage));
            tma_load_2d_pair(sB, &p.mb, (t.kofs + kb) * QB, b_row, full_bar(stage));
          }
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == NST) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && rank == 0) {
        for (int s = 0; s < NST; ++s)
          if (issued >> s & 1u) {
            volatile int never = 0;
            mbar_wait(full_bar(s), issued_parity >> s & 1u, &never, limit, INFO_WAIT_DRAIN);
          }
      }
    }
    __syncwarp();
  } else if (warp == 13) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (rank == 0 && lane == 0) {
      // the tensor core drains its queue in a few hundred cycles, so every cycle of this thread between
      // two stages counts (300 more per tile cost 5%): inlined barrier tests, a stage's instructions
      // unrolled, the next tile's K looked up ahead
      int stage = 0, acc = 0, unit = 0;
      uint32_t phase = 0, acc_phase = 0, unit_phase = 0;
      uint32_t sf = sf_col(0);
      bool ok = true, any = false;
      const uint64_t adesc0 = make_sdesc(smem_u32(base)), bdesc0 = make_sdesc(smem_u32(base) + a_stage);
      int nk = f8_blocks<WGRAD>(p, pair, total, prefix, start);
      for (int r = 0; (long long)r * npairs < total && ok; ++r) {
        const int left0 = nk;
        nk = f8_blocks<WGRAD>(p, f8_tile<WGRAD>(r + 1, pair, npairs), total, prefix, start);
        if (left0 == 0) continue;
        if (!mbar_try_wait(acce_bar(acc), acc_phase ^ 1u) &&
            !mbar_wait(acce_bar(acc), acc_phase ^ 1u, abort_flag, limit, INFO_WAIT_ACC_EMPTY)) {
          ok = false;
          break;
        }
        const uint32_t d = tmem_base + (uint32_t)(acc * 256);
        for (int kb = 0; kb < left0; kb += KPB) {
          const uint32_t pos = (uint32_t)kb % F8G_SF_K;  // in the scale unit
          if ((!mbar_try_wait(full_bar(stage), phase) &&
               !mbar_wait(full_bar(stage), phase, abort_flag, limit, INFO_WAIT_TMA_FULL)) ||
              (pos == 0 && !mbar_try_wait(sff_bar(unit), unit_phase) &&
               !mbar_wait(sff_bar(unit), unit_phase, abort_flag, limit, INFO_WAIT_TMA_FULL))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t off = ((uint32_t)stage * stage_bytes) >> 4;
          const uint64_t ad = adesc0 + off, bd = bdesc0 + off;
          const uint32_t idesc = IDESC | pos << 4 | pos << 29;
#pragma unroll
          for (int j = 0; j < KPB; ++j) {
            if (j > 0 && kb + j >= left0) break;
#pragma unroll
            for (int k32 = 0; k32 < 4; ++k32)  // 32 bytes of K: two 16-byte units further
              f8_mma(d, ad + (j * 1024 + 2 * k32), bd + (j * (b_bytes >> 4) + 2 * k32),
                     idesc + j * (1u << 4 | 1u << 29), sf, sf + 4, j == 0 && k32 == 0 ? kb > 0 : 1u);
          }
          any = true;
          tc2_commit_both(empty_bar(stage));
          if (++stage == NST) { stage = 0; phase ^= 1u; }
          if (pos + KPB == F8G_SF_K || kb + KPB >= left0) {
            tc2_commit_both(sfe_bar(unit));
            if (++unit == F8G_SF_BUFS) { unit = 0; unit_phase ^= 1u; }
            sf = sf_col(unit);
          }
        }
        if (!ok) break;
        tc2_commit_both(accf_bar(acc));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (!ok && any) {
        tc2_commit_both(drain_bar);
        volatile int never = 0;
        mbar_wait(drain_bar, 0u, &never, limit, INFO_WAIT_DRAIN);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ store (warps 4 .. 11)
    const int q = warp & 3, half = (warp - 4) >> 2;
    unsigned char *stg = stg_all + (warp - 4) * 4096;
    const int ebytes = p.out_f32 ? 4 : 2, cpp = 128 / ebytes;  // columns per pass: 128 bytes of a row
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int r = 0; (long long)r * npairs < total; ++r) {
      const int tile = f8_tile<WGRAD>(r, pair, npairs);
      if (tile >= total) continue;
      const F8Tile t = f8_decode<WGRAD>(p, tile, prefix, start);
      const int rbase = t.m0 + (int)rank * 128 + q * 32;
      const int nrows = min(32, t.rows - rbase), ncols = min(p.tn, p.N - t.n0);
      if (t.nk > 0) {
        if (!f8_wait_warp(accf_bar(acc), acc_phase, abort_flag, limit + F8G_BLOCK_NS * t.nk, INFO_WAIT_ACC_FULL))
          break;
        tc_fence_after();
      }
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 256);
      unsigned char *out = (unsigned char *)p.out + ((size_t)(t.row0 + rbase) * p.N + t.n0) * ebytes;
      const size_t pitch = (size_t)p.N * ebytes;
      // The two warps of a lane quarter take every other pass: 32 rows of the staging buffer, written
      // lane = row, read 8 lanes per row (whole 128-byte lines). Streaming stores, so that the operands
      // stay in L2 (35.0 us instead of 36.0, Quartz gate|up).
      if (WGRAD && p.swap) {
        // a column of the tile is a row of out: 32 lanes write 128 bytes of it
        float *col = (float *)p.out + ((size_t)t.g * p.N + t.n0) * p.M + rbase + lane;
        if (nrows > 0)
          for (int c = half * 32; c < ncols; c += 64) {
            uint32_t r[32];
            if (t.nk > 0) {
              tmem_ld32(tb + c, r);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = 0u;
            }
            if (lane < nrows) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c + i < ncols) __stcs(col + (size_t)(c + i) * p.M, __uint_as_float(r[i]));
            }
          }
      } else if (nrows > 0)
        for (int c = half * cpp; c < ncols; c += 2 * cpp) {
          if (p.out_f32) {
            uint32_t r[32];
            if (t.nk > 0) {
              tmem_ld32(tb + c, r);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *(uint4 *)(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                  make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          } else {
            uint32_t r[64];
            tmem_ld32(tb + c, *(uint32_t(*)[32])r);
            tmem_ld32(tb + c + 32, *(uint32_t(*)[32])(r + 32));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(r[8 * i + 2 * j]),
                                                               __uint_as_float(r[8 * i + 2 * j + 1]));
                w[j] = *(const uint32_t *)&v;
              }
              *(uint4 *)(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), ch = lane & 7;
            if (rr < nrows && c + ch * (cpp >> 3) < ncols)
              __stcs((uint4 *)(out + rr * pitch + (size_t)c * ebytes + ch * 16),
                     *(const uint4 *)(stg + rr * 128 + ((ch ^ (rr & 7)) << 4)));
          }
          __syncwarp();
        }
      if (t.nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta0(acce_bar(acc));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still read its smem or TMEM
  if (warp == 13) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u)
                 : "memory");
  }
}

// ------------------------------------------------------------------ few rows
// The same product when the experts have few rows (a served token: one row of each of its top-k
// experts): the weights' bytes are the work, so one CTA takes 16 weight rows of one expert, its 8 warps
// share K block by block, and the rows are the narrow side of m16n8k32 instructions. A lane reads 16
// consecutive codes of a weight row and of a token row; which codes an instruction calls k = 0 .. 31 is
// free as long as both operands agree, so no shuffle or shared memory lies between the load and the
// tensor core. Each block of 128 is summed from zero and added with its scales; the warps' sums are
// added in warp order. Grid: 16-row weight tiles x groups of 16 rows of one expert.
constexpr int F8F_WARPS = 8, F8F_ROWS = 16, F8F_CHUNK = 16;  // tokens per CTA

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct F8Few {
  const uint8_t *a, *a_scale, *w, *w_scale;
  const int32_t *offsets;  // null: one expert with all rows
  void *out;
  long long rows;
  int E, n, k, out_f32;
};

// Work item j: the j-th group of F8F_CHUNK rows, counted through the experts. Every lane of a warp
// calls; a lane looks at four experts at a time.
struct FewItem {
  int e, cnt;
  long long row;
};
__device__ __forceinline__ bool find_few(const F8Few &p, int j, FewItem *it) {
  if (!p.offsets) {
    it->e = 0;
    it->row = (long long)j * F8F_CHUNK;
    it->cnt = (int)min((long long)F8F_CHUNK, p.rows - it->row);
    return it->cnt > 0;
  }
  const int lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < p.E; e0 += 128) {
    int off[5], sum = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) off[i] = (int)expert_bound(p.offsets, min(e0 + 4 * lane + i, p.E), p.rows);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bad |= off[i + 1] < off[i];
      sum += (off[i + 1] - off[i] + F8F_CHUNK - 1) / F8F_CHUNK;
    }
    if (offsets_decrease(__any_sync(0xffffffffu, bad))) return false;
    const int incl = warp_incl_scan(sum);
    const unsigned past = __ballot_sync(0xffffffffu, incl > j);
    if (past) {
      const int src = __ffs(past) - 1;
      j -= __shfl_sync(0xffffffffu, incl - sum, src);
#pragma unroll
      for (int i = 0; i < 5; ++i) off[i] = __shfl_sync(0xffffffffu, off[i], src);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = (off[i + 1] - off[i] + F8F_CHUNK - 1) / F8F_CHUNK;
        if (j >= 0 && j < n) {
          it->e = e0 + 4 * src + i;
          it->row = off[i] + j * F8F_CHUNK;
          it->cnt = min(F8F_CHUNK, off[i + 1] - off[i] - j * F8F_CHUNK);
          return true;
        }
        j -= n;
      }
    }
    j -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// NT groups of 8 tokens against 16 weight rows.
template <int NT>
__device__ __forceinline__ void few_chunk(const F8Few &p, int e, long long row, int cnt, int n0, float *red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int nkb = (p.k + QB - 1) / QB, nnb = (p.n + QB - 1) / QB;
  const uint8_t *wrow = p.w + ((size_t)e * p.n + n0 + g) * p.k + 16 * t;
  const uint8_t *wsc = p.w_scale + ((size_t)e * nnb + n0 / QB) * nkb;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int kb = warp; kb < nkb; kb += F8F_WARPS) {
    uint4 wa[2][2], xb[NT][2];  // [weight row g, g + 8][64-byte half], [token group][half]
    float sx[NT][2];
    const float sw = e8m0_value(__ldg(wsc + kb));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k0 = kb * QB + 64 * h;
      const bool ok = k0 + 16 * t < p.k;
      wa[0][h] = wa[1][h] = make_uint4(0u, 0u, 0u, 0u);
      if (ok) {
        wa[0][h] = __ldg((const uint4 *)(wrow + k0));
        wa[1][h] = __ldg((const uint4 *)(wrow + (size_t)8 * p.k + k0));
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        xb[i][h] = make_uint4(0u, 0u, 0u, 0u);
        if (ok && 8 * i + g < cnt)
          xb[i][h] = __ldg((const uint4 *)(p.a + (size_t)(row + 8 * i + g) * p.k + k0 + 16 * t));
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int tok = 8 * i + 2 * t + j;
        sx[i][j] = tok < cnt ? e8m0_value(__ldg(p.a_scale + (size_t)(row + tok) * nkb + kb)) : 0.0f;
      }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_e4m3(c, wa[0][h].x, wa[1][h].x, wa[0][h].y, wa[1][h].y, xb[i][h].x, xb[i][h].y);
        mma_e4m3(c, wa[0][h].z, wa[1][h].z, wa[0][h].w, wa[1][h].w, xb[i][h].z, xb[i][h].w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // the smaller scale first: their product alone may leave the range where the sum does not
        const float s = sx[i][j & 1];
        acc[i][j] = fmaf(c[j] * (s < sw ? s : sw), s < sw ? sw : s, acc[i][j]);
      }
    }
  }
  // red[warp][token][16 weight rows]
  float *mine = red + (size_t)warp * NT * 8 * 16;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) mine[(8 * i + 2 * t + (j & 1)) * 16 + g + 8 * (j >> 1)] = acc[i][j];
  __syncthreads();
  for (int o = threadIdx.x; o < min(cnt, NT * 8) * 16; o += 32 * F8F_WARPS) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < F8F_WARPS; ++w) s += red[(size_t)w * NT * 8 * 16 + o];
    const size_t at = (size_t)(row + o / 16) * p.n + n0 + o % 16;
    if (p.out_f32) ((float *)p.out)[at] = s;
    else ((__nv_bfloat16 *)p.out)[at] = __float2bfloat16_rn(s);
  }
}

__global__ void __launch_bounds__(32 * F8F_WARPS, 4) gemm_fp8_few_kernel(const __grid_constant__ F8Few p) {
  __shared__ float red[F8F_WARPS * F8F_CHUNK * 16];
  const KernelStamp stamp(K_F8B_GEMM);
  griddep_wait();
  stamp.started();
  griddep_launch();
  FewItem it;
  if (!find_few(p, blockIdx.y, &it)) return;
  if (it.cnt <= 8) few_chunk<1>(p, it.e, it.row, it.cnt, blockIdx.x * F8F_ROWS, red);
  else few_chunk<F8F_CHUNK / 8>(p, it.e, it.row, it.cnt, blockIdx.x * F8F_ROWS, red);
  if (p.offsets && blockIdx.x == 0 && blockIdx.y == gridDim.y - 1 && threadIdx.x < 32)
    check_offsets(p.offsets, p.E, p.rows);
}

}  // namespace moe
