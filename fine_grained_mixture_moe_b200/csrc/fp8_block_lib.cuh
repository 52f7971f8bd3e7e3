// Launches of the block-scaled E4M3 operators (fp8_block.cuh, gemm_fp8_block.cuh). Included by
// moe_lib.cu inside its unnamed namespace.
#pragma once

// [rows, cols] bytes seen as {128 columns, rows, cols / 128 K blocks} (cols a multiple of 128): a
// box {128, box_rows, 2} is the tiles of two K blocks, one after the other. Rows past the last, and the
// second K block past the last, read as zeros.
bool make_map3_u8(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {128, rows, cols / 128};
  cuuint64_t strides[2] = {cols, 128};
  cuuint32_t box[3] = {128, box_rows, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// CTAs of a row-wise kernel over `blocks` blocks, `per` of them per CTA and pass: all that are resident
// at once (4 per SM), or a multiple that leaves each CTA about five passes. One resident wave falls
// behind on the slower SMs in a long call (SwiGLU backward, 131,072 x 768: 229 us, against 192 with
// eight waves); in a short one more waves only add their start-up (SwiGLU forward, 24,576 x 640: 20 us
// with one, 24 with eight).
int fp8_row_grid(long long blocks, int per) {
  const long long need = (blocks + per - 1) / per, wave = 4LL * num_sms();
  const long long waves = std::max<long long>(1, (need + 5 * wave / 2) / (5 * wave));
  return (int)std::max<long long>(1, std::min(need, waves * wave));
}

template <typename Tin>
moe_status_t launch_quantize_block(const void *in, long long rows, int cols, const int32_t *n_rows,
                                   uint8_t *q, uint8_t *scale, cudaStream_t st) {
  const int nblk = ceil_div(cols, QB);
  auto kern = cols % QB ? quantize_block_rows_kernel<Tin, false> : quantize_block_rows_kernel<Tin, true>;
  ProfScope ps(K_F8B_QUANT, st);
  return launch_pdl(kern, dim3(fp8_row_grid(rows * nblk, F8Q_U * RT_TEAMS)), dim3(256), 0, st, (const Tin *)in, rows, cols,
                    nblk, n_rows, q, scale);
}

template <typename Tin>
moe_status_t launch_quantize_weight(const void *in, int E, int rows, int cols, uint8_t *q,
                                    uint8_t *scale, uint8_t *q_t, uint8_t *scale_t, cudaStream_t st) {
  ProfScope ps(K_F8B_QUANT, st);
  return launch_pdl(quantize_block_weight_kernel<Tin>, dim3(ceil_div(cols, QB), ceil_div(rows, QB), E),
                    dim3(F8T_THREADS), 0, st, (const Tin *)in, rows, cols, q, scale, q_t, scale_t);
}

long long token_blocks(long long rows, int E) {
  return (rows + 127 * std::min<long long>(rows, E)) / QB;
}

template <typename Tin>
moe_status_t launch_quantize_tokens(const void *in, const uint8_t *in_scale, long long rows, int cols,
                                    const int32_t *offsets, int E, uint8_t *q_t, uint8_t *scale_t,
                                    cudaStream_t st) {
  const long long nb = token_blocks(rows, E);
  ProfScope ps(K_F8B_QUANT, st);
  return launch_pdl(quantize_block_tokens_kernel<Tin>, dim3((unsigned)(nb * ceil_div(cols, QB))),
                    dim3(F8T_THREADS), 0, st, (const Tin *)in, in_scale, rows, cols, offsets, E, q_t,
                    (size_t)(nb * QB), scale_t);
}

template <bool WGRAD>
moe_status_t launch_gemm_fp8_block(F8Gemm &p, const uint8_t *a, const uint8_t *b, cudaStream_t st) {
  // a tile is 256 rows by up to 224 columns: the weight gradient takes as rows the side that gives
  // fewer tiles (1,280 x 1,024: 24 instead of 25, 896 x 1,024: 16 instead of 20)
  if (WGRAD && ceil_div(p.N, 256) * ceil_div(p.M, f8g_tile_n(p.M)) <
                   ceil_div(p.M, 256) * ceil_div(p.N, f8g_tile_n(p.N))) {
    p.swap = 1;
    std::swap(a, b);
    std::swap(p.a_scale, p.b_scale);
    std::swap(p.M, p.N);
  }
  // one row of a (b) is K codes; wgrad: the token columns of every block
  const uint64_t lda = WGRAD ? (uint64_t)p.K * QB : (uint64_t)p.K;
  const uint64_t a_rows = WGRAD ? p.M : p.rows, b_rows = WGRAD ? (uint64_t)p.N : (uint64_t)p.E * p.N;
  if (WGRAD) p.K = (int)(lda / QB);
  p.tn = f8g_tile_n(p.N);
  p.nt = ceil_div(p.N, p.tn);
  p.nt_mul = p.nt > 1 ? (unsigned)((1ull << 32) / p.nt) + 1u : 0u;
  p.per = WGRAD ? ceil_div(p.M, 256) * p.nt : 1;
  p.per_mul = p.per > 1 ? (unsigned)((1ull << 32) / p.per) + 1u : 0u;
  // two K blocks per copy when a row is whole K blocks (one box instead of two copies) and the tile
  // lists of E experts leave room for two such stages
  p.kpb = lda % QB == 0 && f8g_stages(p.E, p.tn, 2) >= 2 ? 2 : 1;
  p.stages = f8g_stages(p.E, p.tn, p.kpb);
  const uint32_t bb = p.tn / 2;
  auto kern = p.kpb == 2 ? gemm_fp8_block_kernel<WGRAD, 2> : gemm_fp8_block_kernel<WGRAD, 1>;
  // Before the maps: it binds the device's context to a thread that has made no call yet, which the
  // driver's encoder asks for. One value for every call: a call's own size could be lowered by another
  // thread's before the launch.
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F8G_MAX_SMEM) != cudaSuccess)
    return MOE_ERR_CUDA;
  const bool ok = p.kpb == 2
                      ? make_map3_u8(&p.ma, a, a_rows, lda, 128) && make_map3_u8(&p.mb, b, b_rows, lda, bb)
                      : make_map(&p.ma, a, a_rows, lda, 128, 1) && make_map(&p.mb, b, b_rows, lda, bb, 1);
  if (!ok) return MOE_ERR_CUDA;
  const long long tiles = WGRAD ? (long long)p.E * ceil_div(p.M, 256) * ceil_div(p.N, p.tn)
                                : (ceil_div(p.rows, 256) + std::min<long long>(p.E, p.rows)) *
                                      ceil_div(p.N, p.tn);
  const int pairs = (int)std::min<long long>(num_sms() / 2, tiles);
  const size_t smem = f8g_fixed_bytes(p.E) + (size_t)p.stages * f8g_stage_bytes(p.tn, p.kpb);
  const int kind = WGRAD ? K_F8B_WGRAD : K_F8B_GEMM;
  ProfScope ps(kind, st);
  return launch_pdl(kern, dim3(2 * pairs), dim3(F8G_THREADS), smem, st, p);
}

// The form for few rows is chosen by its CTAs (16 weight rows x 16 rows; half a group of rows per expert
// taken as unfilled) times the K blocks that each of a CTA's 8 warps does in turn, against the CTA-pair
// form's start-up, K, and tiles of many experts. Measured on both sides, few / pairs in us, rows on the first experts | spread:
//   24 experts, n 1280, k 1024:  6 rows 4.4 / 8.2 | 4.4 / 8.3;     48: 5.8 / 8.2 | 10.5 / 13.1;
//                                96: 8.2 / 8.1 | 12.3 / 13.1;      192: 12.4 / 8.2 | 15.6 / 13.2
//   24 experts, n 1024, k 640:   96: 6.0 / 6.9 | 9.3 / 10.6;       192: 8.7 / 7.0 | 11.5 / 10.8
//   97 experts, n = k = 512:     48: 4.1 / 6.0 | 6.9 / 8.8;        96: 6.6 / 6.1 | 10.9 / 10.8
//   256 experts, n = k = 1024:   32: 7.4 / 7.7 | 12.9 / 14.9;      64: 13.2 / 7.7 | 21.9 / 20.0
//   8 experts, n 512, k 2048:    128: 9.7 / 10.4 | 10.1 / 10.9;    256: 10.1 / 10.8 | 11.7 / 10.9
//   1 expert, n = k = 1024:      128: 7.0 / 8.2;                   256: 11.4 / 8.2
//   1 expert, n = k = 4096:      16: 11.1 / 16.5;                  64: 28 / 17
bool few_rows(long long rows, int E, int n, int k) {
  if (rows > 4096) return false;
  const int nkb = ceil_div(k, QB);
  const long long groups2 = 2 * rows / F8F_CHUNK + std::min<long long>(E, rows);  // twice the groups
  return groups2 * (n / F8F_ROWS) * ceil_div(nkb, F8F_WARPS) <=
         400 + 110LL * nkb + 75 * std::min<long long>(std::min(E, 24), rows);
}

moe_status_t launch_gemm_fp8_few(const F8Few &p, cudaStream_t st) {
  // groups of F8F_CHUNK rows: each of the experts that can have rows wastes at most F8F_CHUNK - 1
  const long long items = p.offsets ? (p.rows + (F8F_CHUNK - 1) * std::min<long long>(p.E, p.rows)) / F8F_CHUNK
                                    : ceil_div(p.rows, F8F_CHUNK);
  ProfScope ps(K_F8B_GEMM, st);
  return launch_pdl(gemm_fp8_few_kernel, dim3(p.n / F8F_ROWS, (unsigned)items), dim3(32 * F8F_WARPS), 0, st, p);
}
