// C ABI entry points of the block-scaled E4M3 operators: argument checks and the calls into
// fp8_block_lib.cuh. Included by moe_lib.cu inside its extern "C" block.
#pragma once

// rows of one call (32-bit row coordinates inside the kernels) and row widths in codes
#define MOE_F8B_ROWS(rows) \
  do {                     \
    if ((rows) < 0) return MOE_ERR_INVALID_ARG; \
    if ((rows) > (1ll << 31) - 4096) return MOE_ERR_UNSUPPORTED; \
  } while (0)
#define MOE_F8B_WIDTH(w) \
  do {                   \
    if ((w) <= 0) return MOE_ERR_INVALID_ARG; \
    if ((w) % 16 || (w) > (1 << 20)) return MOE_ERR_UNSUPPORTED; \
  } while (0)
#define MOE_F8B_EXPERTS(E) \
  do {                     \
    if ((E) <= 0) return MOE_ERR_INVALID_ARG; \
    if ((E) > 1024) return MOE_ERR_UNSUPPORTED; \
  } while (0)

// tiles of one launch: a 32-bit tile number with room for one more stride
#define MOE_F8B_TILES ((1ll << 31) - 65536)

static inline bool f8b_dtype(int32_t t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }
// a product's output: its rows, multiples of 32 bytes, then fill whole sectors of L2
static inline bool aligned32(const void *p) { return p && ((uintptr_t)p & 31u) == 0; }
static inline bool aligned4(const void *p) { return p && ((uintptr_t)p & 3u) == 0; }

moe_status_t moe_quantize_fp8_block(const void *in, int32_t in_dtype, int64_t rows, int32_t cols,
                                    const int32_t *n_rows, uint8_t *q, uint8_t *scale, void *stream) {
  MOE_F8B_ROWS(rows);
  MOE_F8B_WIDTH(cols);
  if (!f8b_dtype(in_dtype)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  MOE_REQUIRE(aligned16(in) && aligned16(q) && scale && (!n_rows || aligned4(n_rows)));
  cudaStream_t st = (cudaStream_t)stream;
  return in_dtype == MOE_DTYPE_BF16
             ? launch_quantize_block<__nv_bfloat16>(in, rows, cols, n_rows, q, scale, st)
             : launch_quantize_block<float>(in, rows, cols, n_rows, q, scale, st);
}

moe_status_t moe_quantize_fp8_weight(const void *in, int32_t in_dtype, int32_t E, int32_t rows,
                                     int32_t cols, uint8_t *q, uint8_t *scale, uint8_t *q_t,
                                     uint8_t *scale_t, void *stream) {
  MOE_F8B_EXPERTS(E);
  MOE_F8B_WIDTH(rows);
  MOE_F8B_WIDTH(cols);
  if (!f8b_dtype(in_dtype)) return MOE_ERR_UNSUPPORTED;
  MOE_REQUIRE(aligned16(in) && aligned16(q) && scale && !q_t == !scale_t && (!q_t || aligned16(q_t)));
  cudaStream_t st = (cudaStream_t)stream;
  return in_dtype == MOE_DTYPE_BF16
             ? launch_quantize_weight<__nv_bfloat16>(in, E, rows, cols, q, scale, q_t, scale_t, st)
             : launch_quantize_weight<float>(in, E, rows, cols, q, scale, q_t, scale_t, st);
}

int64_t moe_fp8_token_blocks(int64_t rows, int32_t E) {
  if (rows < 0 || rows > (1ll << 31) - 4096 || E <= 0 || E > 1024) return -1;
  return token_blocks(rows, E);
}

moe_status_t moe_quantize_fp8_tokens(const void *in, int32_t in_dtype, const uint8_t *in_scale,
                                     int64_t rows, int32_t cols, const int32_t *offsets, int32_t E,
                                     uint8_t *q_t, uint8_t *scale_t, void *stream) {
  MOE_F8B_ROWS(rows);
  MOE_F8B_WIDTH(cols);
  MOE_F8B_EXPERTS(E);
  if (!f8b_dtype(in_dtype) && in_dtype != MOE_DTYPE_E4M3) return MOE_ERR_UNSUPPORTED;
  if (token_blocks(rows, E) * ceil_div(cols, QB) > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  MOE_REQUIRE(aligned16(in) && aligned4(offsets) && aligned16(q_t) && scale_t);
  MOE_REQUIRE((in_dtype == MOE_DTYPE_E4M3) == (in_scale != nullptr));
  cudaStream_t st = (cudaStream_t)stream;
  if (in_dtype == MOE_DTYPE_E4M3)
    return launch_quantize_tokens<uint8_t>(in, in_scale, rows, cols, offsets, E, q_t, scale_t, st);
  return in_dtype == MOE_DTYPE_BF16
             ? launch_quantize_tokens<__nv_bfloat16>(in, in_scale, rows, cols, offsets, E, q_t, scale_t, st)
             : launch_quantize_tokens<float>(in, in_scale, rows, cols, offsets, E, q_t, scale_t, st);
}

moe_status_t moe_gemm_fp8_block(const uint8_t *a, const uint8_t *a_scale, int64_t rows,
                                const int32_t *offsets, int32_t E, int32_t n, int32_t k,
                                const uint8_t *w, const uint8_t *w_scale, void *out,
                                int32_t out_dtype, void *stream) {
  MOE_F8B_ROWS(rows);
  MOE_F8B_EXPERTS(E);
  MOE_F8B_WIDTH(n);
  MOE_F8B_WIDTH(k);
  if (!f8b_dtype(out_dtype) || (long long)E * n > (1ll << 31) - 4096) return MOE_ERR_UNSUPPORTED;
  if ((ceil_div(rows, 256) + (long long)E) * ceil_div(n, f8g_tile_n(n)) > MOE_F8B_TILES) return MOE_ERR_UNSUPPORTED;
  MOE_REQUIRE(offsets || E == 1);
  if (rows == 0) return MOE_OK;
  MOE_REQUIRE(aligned16(a) && a_scale && aligned16(w) && w_scale && aligned32(out) &&
              (!offsets || aligned4(offsets)));
  if (few_rows(rows, E, n, k)) {
    const F8Few f = {a, a_scale, w, w_scale, offsets, out, rows, E, n, k, out_dtype == MOE_DTYPE_F32};
    return launch_gemm_fp8_few(f, (cudaStream_t)stream);
  }
  F8Gemm p;
  std::memset(&p, 0, sizeof(p));
  p.offsets = offsets;
  p.a_scale = a_scale;
  p.b_scale = w_scale;
  p.out = out;
  p.rows = rows;
  p.E = E;
  p.N = n;
  p.K = k;
  p.out_f32 = out_dtype == MOE_DTYPE_F32;
  return launch_gemm_fp8_block<false>(p, a, w, (cudaStream_t)stream);
}

moe_status_t moe_wgrad_fp8_block(const uint8_t *a_t, const uint8_t *a_scale, const uint8_t *b_t,
                                 const uint8_t *b_scale, int64_t rows, const int32_t *offsets,
                                 int32_t E, int32_t n, int32_t k, float *dw, void *stream) {
  MOE_F8B_ROWS(rows);
  MOE_F8B_EXPERTS(E);
  MOE_F8B_WIDTH(n);
  MOE_F8B_WIDTH(k);
  if (token_blocks(rows, E) > (1ll << 24) - 1) return MOE_ERR_UNSUPPORTED;  // K coordinates
  if ((long long)E * ceil_div(n, 128) * ceil_div(k, 128) > MOE_F8B_TILES) return MOE_ERR_UNSUPPORTED;
  MOE_REQUIRE(aligned32(dw));
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0)
    return cudaMemsetAsync(dw, 0, (size_t)E * n * k * sizeof(float), st) == cudaSuccess ? MOE_OK
                                                                                       : MOE_ERR_CUDA;
  MOE_REQUIRE(aligned16(a_t) && a_scale && aligned16(b_t) && b_scale && aligned4(offsets));
  F8Gemm p;
  std::memset(&p, 0, sizeof(p));
  p.offsets = offsets;
  p.a_scale = a_scale;
  p.b_scale = b_scale;
  p.out = dw;
  p.rows = rows;
  p.E = E;
  p.M = n;
  p.N = k;
  p.K = (int)token_blocks(rows, E);
  p.out_f32 = 1;
  return launch_gemm_fp8_block<true>(p, a_t, b_t, st);
}

moe_status_t moe_swiglu_fp8_forward(const void *gu, int32_t in_dtype, int64_t rows, int32_t ffn,
                                    const int32_t *n_rows, void *h, uint8_t *h_q, uint8_t *h_scale,
                                    uint8_t *gu_q, uint8_t *gu_scale, void *stream) {
  MOE_F8B_ROWS(rows);
  MOE_F8B_WIDTH(ffn);
  if (ffn % QB || !f8b_dtype(in_dtype)) return MOE_ERR_UNSUPPORTED;
  MOE_REQUIRE(!h_q == !h_scale && !gu_q == !gu_scale && (h || h_q || gu_q || rows == 0));
  if (rows == 0) return MOE_OK;
  MOE_REQUIRE(aligned16(gu) && (!h || aligned16(h)) && (!h_q || aligned16(h_q)) &&
              (!gu_q || aligned16(gu_q)) && (!n_rows || aligned4(n_rows)));
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid(fp8_row_grid(rows * (ffn / QB), RT_TEAMS));
  ProfScope ps(K_F8B_SWIGLU, st);
  if (in_dtype == MOE_DTYPE_BF16)
    return launch_pdl(swiglu_checkpoint_kernel<__nv_bfloat16>, grid, dim3(256), 0, st,
                      (const __nv_bfloat16 *)gu, (long long)rows, ffn, n_rows, (__nv_bfloat16 *)h, h_q,
                      h_scale, gu_q, gu_scale);
  return launch_pdl(swiglu_checkpoint_kernel<float>, grid, dim3(256), 0, st, (const float *)gu,
                    (long long)rows, ffn, n_rows, (__nv_bfloat16 *)h, h_q, h_scale, gu_q, gu_scale);
}

moe_status_t moe_swiglu_fp8_backward(const uint8_t *gu_q, const uint8_t *gu_scale, const void *dh,
                                     int32_t dh_dtype, int64_t rows, int32_t ffn,
                                     const int32_t *n_rows, void *dgu, uint8_t *dgu_q,
                                     uint8_t *dgu_scale, void *h, void *stream) {
  MOE_F8B_ROWS(rows);
  MOE_F8B_WIDTH(ffn);
  if (ffn % QB || !f8b_dtype(dh_dtype)) return MOE_ERR_UNSUPPORTED;
  MOE_REQUIRE(!dgu_q == !dgu_scale && (dgu || dgu_q || h || rows == 0));
  if (rows == 0) return MOE_OK;
  MOE_REQUIRE(aligned16(gu_q) && gu_scale && aligned16(dh) && (!dgu || aligned16(dgu)) &&
              (!dgu_q || aligned16(dgu_q)) && (!h || aligned16(h)) && (!n_rows || aligned4(n_rows)));
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid(fp8_row_grid(rows * (ffn / QB), RT_TEAMS));
  ProfScope ps(K_F8B_SWIGLU, st);
  if (dh_dtype == MOE_DTYPE_BF16)
    return launch_pdl(swiglu_checkpoint_backward_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, gu_q,
                      gu_scale, (const __nv_bfloat16 *)dh, (long long)rows, ffn, n_rows,
                      (__nv_bfloat16 *)dgu, dgu_q, dgu_scale, (__nv_bfloat16 *)h);
  return launch_pdl(swiglu_checkpoint_backward_kernel<float>, grid, dim3(256), 0, st, gu_q, gu_scale,
                    (const float *)dh, (long long)rows, ffn, n_rows, (__nv_bfloat16 *)dgu, dgu_q,
                    dgu_scale, (__nv_bfloat16 *)h);
}
