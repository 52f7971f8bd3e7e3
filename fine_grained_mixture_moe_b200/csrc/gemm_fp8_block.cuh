// Block-scaled E4M3 products (the format of fp8_block.cuh) on CTA pairs (tcgen05, sm_100a), and a
// warp-level form for experts with few rows.
//
// gemm (WGRAD = false): expert g's rows of a [rows, k] against its weight w[g] [n, k]:
//   out[r, c] = sum over 128-wide blocks kb of 2^(sa[r, kb] + sw[g, c / 128, kb])
//               * sum over k in kb of a[r, k] w[g, c, k]
// wgrad (WGRAD = true): both operands are transposed and K is the token: expert g owns the columns
//   128 koff[g] .. 128 koff[g + 1] of a_t [n, pitch] and b_t [k, pitch],
//   dw[g][r, c] = sum over its blocks tb of 2^(sa[tb, r] + sb[tb, c]) sum over t in tb of a_t b_t.
//
// The scales change with every 128 of K, so the tensor core sums one block at a time: four K = 32
// instructions (kind::f8f6f4, products exact, fp32 sums) fill one of two 256-column TMEM buffers,
// and the epilogue warps add the block, times its scales, into fp32 registers (128 columns of one
// row per thread) while the other buffer fills. Powers of two make the scaling exact: the result
// carries the rounding of fp32 sums only.
//
// Tiles, clusters and barriers are those of gemm_tc2.cuh: 256 x 256 per CTA pair, CTA r loads 128
// rows of each operand, the leader issues M = 256, N = 256. A stage holds one or two K blocks of
// 128 bytes (two by one 3-D box when K is a multiple of 128).
#pragma once
#include "fp8_block.cuh"
#include "gemm_tc2.cuh"

namespace moe {

struct F8Gemm {
  CUtensorMap ma, mb;
  const int32_t *offsets;  // [E + 1] device, clamped to [0, rows]; null: one group of all rows
  const uint8_t *a_scale, *b_scale;
  void *out;
  long long rows;          // rows of a (gemm) or grouped rows (wgrad)
  int E, M, N, K;          // gemm: N = n, K = k; wgrad: M = n, N = k, K = blocks the buffers hold
  int out_f32;
  int stages, kpb;
};

struct F8Tile {
  int g, m0, n0;
  int rows;         // rows of the group (gemm) or M (wgrad)
  long long row0;   // its first row in a and out (gemm)
  int kofs, nk;     // first K block and K blocks
};

constexpr int F8G_STAGE = 32768;  // one K block of both operands (this CTA's halves)
constexpr int F8G_STG = TC_EPI_WARPS * 4096;
constexpr size_t f8g_fixed_bytes(int E) {
  return 1024 + (size_t)F8G_STG + 256 + (size_t)(2 * E + 2 + TC_THREADS / 32 + 1) * sizeof(int);
}
constexpr int f8g_stages(int E, int kpb) {
  const long long n = (227LL * 1024 - (long long)f8g_fixed_bytes(E)) / ((long long)F8G_STAGE * kpb);
  return n > 8 / kpb ? 8 / kpb : (int)n;
}
constexpr size_t f8g_smem_bytes(int E, int kpb) {
  return f8g_fixed_bytes(E) + (size_t)f8g_stages(E, kpb) * F8G_STAGE * kpb;
}

// Tile counts per group scanned into prefix[0 .. E]; wgrad also the groups' K-block offsets.
template <bool WGRAD>
__device__ __forceinline__ int f8_tile_prefix(const F8Gemm &p, int *prefix, int *koff, int *tmp) {
  const int nt = (p.N + 255) / 256;
  for (int g = threadIdx.x; g < p.E; g += blockDim.x) {
    long long n = p.rows;
    if (p.offsets)
      n = max(expert_bound(p.offsets, g + 1, p.rows) - expert_bound(p.offsets, g, p.rows), 0ll);
    if (WGRAD) {
      prefix[g] = ((p.M + 255) / 256) * nt;
      koff[g] = (int)((n + QB - 1) / QB);
    } else {
      prefix[g] = (int)((n + 255) / 256) * nt;
    }
  }
  __syncthreads();
  if (WGRAD) {
    const int all = block_excl_scan_inplace(koff, p.E, tmp);
    if (threadIdx.x == 0) koff[p.E] = all;
  }
  const int total = block_excl_scan_inplace(prefix, p.E, tmp);
  if (threadIdx.x == 0) prefix[p.E] = total;
  __syncthreads();
  return total;
}

template <bool WGRAD>
__device__ __forceinline__ F8Tile f8_decode(const F8Gemm &p, int tile, const int *prefix, const int *koff) {
  int lo = 0, hi = p.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int nt = (p.N + 255) / 256, local = tile - prefix[lo];
  F8Tile t;
  t.g = lo;
  t.m0 = (local / nt) * 256;
  t.n0 = (local % nt) * 256;
  if (WGRAD) {
    t.rows = p.M;
    t.row0 = (long long)lo * p.M;
    t.kofs = min(koff[lo], p.K);
    t.nk = min(koff[lo + 1], p.K) - t.kofs;
  } else {
    t.row0 = p.offsets ? expert_bound(p.offsets, lo, p.rows) : 0;
    t.rows = (int)((p.offsets ? expert_bound(p.offsets, lo + 1, p.rows) : p.rows) - t.row0);
    t.kofs = 0;
    t.nk = (p.K + QB - 1) / QB;
  }
  return t;
}

// 16 accumulator columns times their scales into the running sums.
__device__ __forceinline__ void f8_fma16(float *acc, const uint32_t (&r)[16], float s) {
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = fmaf(__uint_as_float(r[i]), s, acc[i]);
}
__device__ __forceinline__ void f8_fma16(float *acc, const uint32_t (&r)[16], float s, const float *col) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 c = *(const float4 *)(col + 4 * i);
    acc[4 * i] = fmaf(__uint_as_float(r[4 * i]) * c.x, s, acc[4 * i]);
    acc[4 * i + 1] = fmaf(__uint_as_float(r[4 * i + 1]) * c.y, s, acc[4 * i + 1]);
    acc[4 * i + 2] = fmaf(__uint_as_float(r[4 * i + 2]) * c.z, s, acc[4 * i + 2]);
    acc[4 * i + 3] = fmaf(__uint_as_float(r[4 * i + 3]) * c.w, s, acc[4 * i + 3]);
  }
}

template <bool WGRAD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(TC_THREADS, 1)
    gemm_fp8_block_kernel(const __grid_constant__ F8Gemm p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int NST = p.stages, KPB = p.kpb;
  const uint32_t stage_bytes = (uint32_t)F8G_STAGE * KPB, half_bytes = stage_bytes / 2;
  constexpr uint32_t IDESC = (1u << 4) | (256u >> 3 << 17) | (256u >> 4 << 24);  // E4M3, fp32 sums

  const uint32_t raw = smem_u32(smem_raw);
  unsigned char *base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char *stg_all = base + (size_t)NST * stage_bytes;
  uint64_t *bars = (uint64_t *)(stg_all + F8G_STG);
  uint32_t *tmem_slot = (uint32_t *)(bars + 2 * NST + 5);
  volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
  int *prefix = (int *)(stg_all + F8G_STG + 256);
  int *koff = prefix + p.E + 1;
  int *scan_tmp = koff + p.E + 1;

  auto full_bar = [&](int s) { return smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return smem_u32(bars + NST + s); };
  auto accf_bar = [&](int b) { return smem_u32(bars + 2 * NST + b); };
  auto acce_bar = [&](int b) { return smem_u32(bars + 2 * NST + 2 + b); };
  const uint32_t drain_bar = smem_u32(bars + 2 * NST + 4);

  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 2 * TC_EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  const KernelStamp stamp(WGRAD ? K_F8B_WGRAD : K_F8B_GEMM);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const int total = f8_tile_prefix<WGRAD>(p, prefix, koff, scan_tmp);
  tc_fence_before();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t limit = g_wait_limit_ns;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      uint32_t issued = 0, issued_parity = 0;  // bit s: stage s was filled, with that parity
      for (int tile = pair; tile < total && ok; tile += npairs) {
        const F8Tile t = f8_decode<WGRAD>(p, tile, prefix, koff);
        // CTA 1's 128 rows may hold none of the group: never stored, so not loaded (gemm_tc2.cuh)
        const bool a1_void = t.m0 + 128 >= t.rows;
        const uint32_t tx = 2 * stage_bytes - (a1_void ? half_bytes : 0);
        const int a_row = (WGRAD ? 0 : (int)t.row0) + t.m0 + (int)rank * 128;
        const int b_row = (WGRAD ? 0 : t.g * p.N) + t.n0 + (int)rank * 128;
        for (int kb = 0; kb < t.nk; kb += KPB) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, limit, INFO_WAIT_MMA_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t sA = smem_u32(base + (size_t)stage * stage_bytes), sB = sA + half_bytes;
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
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader only)
    if (rank == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true, any = false;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        const F8Tile t = f8_decode<WGRAD>(p, tile, prefix, koff);
        for (int kb = 0; kb < t.nk && ok; kb += KPB) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag, limit, INFO_WAIT_TMA_FULL)) {
            ok = false;
            break;
          }
          const uint32_t sA0 = smem_u32(base + (size_t)stage * stage_bytes), sB0 = sA0 + half_bytes;
          for (int j = 0; j < KPB && kb + j < t.nk; ++j) {
            if (!mbar_wait(acce_bar(acc), acc_phase ^ 1u, abort_flag, limit, INFO_WAIT_ACC_EMPTY)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(acc * 256);
            const uint32_t sA = sA0 + j * 16384, sB = sB0 + j * 16384;
#pragma unroll
            for (int k32 = 0; k32 < 4; ++k32)
              tc2_mma_f8(d, make_sdesc(sA + k32 * 32), make_sdesc(sB + k32 * 32), IDESC, k32 > 0);
            any = true;
            tc2_commit_both(accf_bar(acc));
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
          }
          if (!ok) break;
          tc2_commit_both(empty_bar(stage));
          if (++stage == NST) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && any) {
        tc2_commit_both(drain_bar);
        volatile int never = 0;
        mbar_wait(drain_bar, 0u, &never, limit, INFO_WAIT_DRAIN);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ accumulate and store (warps 2..9)
    const int q = warp & 3, half = (warp - 2) >> 2;
    unsigned char *stg = stg_all + (warp - 2) * 4096;
    int acc_buf = 0;
    uint32_t acc_phase = 0;
    const int nkb = (p.K + QB - 1) / QB, nnb = (p.N + QB - 1) / QB;
    for (int tile = pair; tile < total; tile += npairs) {
      const F8Tile t = f8_decode<WGRAD>(p, tile, prefix, koff);
      const int rbase = t.m0 + (int)rank * 128 + q * 32, row = rbase + lane;
      const int col0 = t.n0 + half * 128;
      const bool live = rbase < t.rows && col0 < p.N;  // this warp stores something
      const bool row_ok = live && row < t.rows;
      // the row's scales: one byte per K block; wgrad: the 128 columns' scales too, 4 per lane
      const uint8_t *sa = nullptr, *sb = nullptr;
      if (WGRAD) {
        sa = p.a_scale + (size_t)t.kofs * p.M + row;
        sb = p.b_scale + (size_t)t.kofs * p.N + col0 + 4 * lane;
      } else {
        sa = p.a_scale + (size_t)(t.row0 + row) * nkb;
        sb = p.b_scale + ((size_t)t.g * nnb + col0 / QB) * nkb;
      }
      const bool col_ok = live && (!WGRAD || col0 + 4 * lane < p.N);
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
      bool ok = true;
      for (int kb = 0; kb < t.nk; ++kb) {
        uint32_t ba = 0, bb = 0;
        if (row_ok) ba = __ldg(sa + (size_t)kb * (WGRAD ? p.M : 1));
        if (col_ok) bb = WGRAD ? __ldg((const uint32_t *)(sb + (size_t)kb * p.N)) : __ldg(sb + kb);
        float s = e8m0_value(ba);
        const float *cs = (const float *)stg + (kb & 1) * 128;
        if (WGRAD) {
          *(float4 *)(stg + (kb & 1) * 512 + lane * 16) =
              make_float4(e8m0_value(bb & 255u), e8m0_value(bb >> 8 & 255u),
                          e8m0_value(bb >> 16 & 255u), e8m0_value(bb >> 24));
          __syncwarp();
        } else {
          s *= e8m0_value(bb);
        }
        if (!mbar_try_wait(accf_bar(acc_buf), acc_phase))
          ok = mbar_wait(accf_bar(acc_buf), acc_phase, abort_flag, limit, INFO_WAIT_ACC_FULL);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc_buf * 256 + half * 128);
          uint32_t r0[16], r1[16];
          tmem_ld16(tb, r0);
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            tmem_wait_ld();
            tmem_ld16(tb + c + 16, r1);
            if (WGRAD) f8_fma16(acc + c, r0, s, cs + c);
            else f8_fma16(acc + c, r0, s);
            tmem_wait_ld();
            if (c + 32 < 128) tmem_ld16(tb + c + 32, r0);
            if (c + 32 == 128) {  // the buffer is read: the next block may fill it
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cta0(acce_bar(acc_buf));
            }
            if (WGRAD) f8_fma16(acc + c + 16, r1, s, cs + c + 16);
            else f8_fma16(acc + c + 16, r1, s);
          }
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive_cta0(acce_bar(acc_buf));
        }
        if (++acc_buf == 2) { acc_buf = 0; acc_phase ^= 1u; }
      }
      if (!ok) break;
      if (!live) continue;
      // 32 rows x 128 bytes at a time through the warp's staging buffer: lane = row in, then 8
      // lanes per row out (whole 128-byte lines)
      __syncwarp();
      const int ebytes = p.out_f32 ? 4 : 2, cpp = 128 / ebytes;  // columns per pass
      unsigned char *out = (unsigned char *)p.out + ((size_t)(t.row0 + rbase) * p.N + col0) * ebytes;
      const size_t pitch = (size_t)p.N * ebytes;
      const int nrows = min(32, t.rows - rbase), ncols = min(128, p.N - col0);
      auto flush = [&](int c) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3), ch = lane & 7;
          if (rr < nrows && c + ch * (cpp >> 3) < ncols)
            *(uint4 *)(out + rr * pitch + (size_t)c * ebytes + ch * 16) =
                *(const uint4 *)(stg + rr * 128 + ((ch ^ (rr & 7)) << 4));
        }
        __syncwarp();
      };
      if (p.out_f32) {
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *(float4 *)(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_float4(acc[c + 4 * i], acc[c + 4 * i + 1], acc[c + 4 * i + 2], acc[c + 4 * i + 3]);
          flush(c);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 128; c += 64) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(acc[c + 8 * i + 2 * j], acc[c + 8 * i + 2 * j + 1]);
              w[j] = *(const uint32_t *)&b;
            }
            *(uint4 *)(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          flush(c);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its peer may still read its smem or TMEM
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u)
                 : "memory");
  }
}

}  // namespace moe
