// Block-scaled E4M3: quantisers and the SwiGLU with an 8-bit activation checkpoint.
//
// A block of 128 values shares one E8M0 scale byte b, worth 2^(b - 127): the least power of two
// with amax / scale <= 448 (not below 2^-126; 1 for an all-zero block). Dividing by a power of two
// is exact in fp32 (a quotient that underflows is far below half the least E4M3 value), so a code
// is the value's nearest E4M3 number, ties to even, and that is the only rounding anywhere here.
// Blocks run along a row (1 x 128), are square (128 x 128, weights), or run along the rows of one
// expert (128 x 1, the operands of a weight gradient, whose inner dimension is the token).
//
// All of these kernels move each byte once and are bound by HBM: 16-byte loads per lane, the block
// maximum by warp shuffles, the values held in registers between the maximum and the conversion.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr int QB = 128;  // values per block

// ------------------------------------------------------------------ the format
// Scale byte of a block from the bits of its largest magnitude: amax = m 2^e with 1 <= m < 2 and
// 448 = 1.75 * 2^8, so the exponent is e - 8, one more when m > 1.75 (the carry of the addition).
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t amax_bits) {
  if (amax_bits == 0) return 127;
  const int b = (int)((amax_bits + 0x1FFFFFu) >> 23) - 8;
  return (uint32_t)max(b, 1);
}
// 2^(b - 127) and its reciprocal, both normal for the bytes 1 .. 248 that e8m0_of_amax returns
__device__ __forceinline__ float e8m0_value(uint32_t b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ float e8m0_inverse(uint32_t b) {
  return __uint_as_float((254u - b) << 23);
}
// Codes of two values, the first in the low byte (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Values of two codes (exact in fp16).
__device__ __forceinline__ float2 e4m3x2_values(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*(const __half2 *)&h);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// Largest over the `L` consecutive lanes of this lane's team (bits of non-negative floats order
// as integers).
template <int L> __device__ __forceinline__ uint32_t team_max(uint32_t v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// `V` consecutive elements as fp32, and back.
template <typename T, int V> struct Pack;
template <int V> struct Pack<float, V> {
  static_assert(V % 4 == 0, "16-byte loads");
  float4 r[V / 4];
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) r[i] = __ldg((const float4 *)p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void values(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      v[4 * i] = r[i].x;
      v[4 * i + 1] = r[i].y;
      v[4 * i + 2] = r[i].z;
      v[4 * i + 3] = r[i].w;
    }
  }
};
template <int V> struct Pack<__nv_bfloat16, V> {
  static_assert(V % 8 == 0, "16-byte loads");
  uint4 r[V / 8];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) r[i] = __ldg((const uint4 *)p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) r[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void values(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
};
// E4M3 codes (a row's block scale applied by the caller).
template <int V> struct Pack<uint8_t, V> {
  static_assert(V == 16, "one 16-byte load");
  uint4 r;
  __device__ __forceinline__ void load(const uint8_t *p) { r = __ldg((const uint4 *)p); }
  __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void values(float (&v)[V]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e4m3x2_values(w[j] & 0xffffu), b = e4m3x2_values(w[j] >> 16);
      v[4 * j] = a.x;
      v[4 * j + 1] = a.y;
      v[4 * j + 2] = b.x;
      v[4 * j + 3] = b.y;
    }
  }
};

template <int V> __device__ __forceinline__ uint32_t amax_bits(const float (&v)[V]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, abs_bits(v[i]));
  return m;
}
// V codes of v * inv to q (V-byte aligned), V = 4, 8 or 16.
template <int V> __device__ __forceinline__ void store_codes(uint8_t *q, const float (&v)[V], float inv) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    w[i] = e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  if (V == 4) *(uint32_t *)q = w[0];
  if (V == 8) *(uint2 *)q = make_uint2(w[0], w[V / 4 > 1 ? 1 : 0]);
  if (V == 16)
    *(uint4 *)q = make_uint4(w[0], w[V / 4 > 1 ? 1 : 0], w[V / 4 > 2 ? 2 : 0], w[V / 4 > 3 ? 3 : 0]);
}
__device__ __forceinline__ void store_bf16x8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *(const uint32_t *)&b;
  }
  *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows to process: all, or as many as the device counter says.
__device__ __forceinline__ long long valid_rows(long long rows, const int32_t *n_rows) {
  return n_rows ? min(rows, (long long)max(__ldg(n_rows), 0)) : rows;
}

// A thread's walk over the (row, block) pairs of a [rows, nblk] grid of blocks in steps of
// `step` blocks: one division at the start, none per step.
struct BlockWalk {
  long long row, drow;
  int blk, dblk, nblk;
  __device__ __forceinline__ BlockWalk(long long first, long long step, int nb) : nblk(nb) {
    row = first / nb;
    blk = (int)(first - row * nb);
    drow = step / nb;
    dblk = (int)(step - drow * nb);
  }
  __device__ __forceinline__ void next() {
    row += drow;
    blk += dblk;
    if (blk >= nblk) {
      blk -= nblk;
      ++row;
    }
  }
};

// ------------------------------------------------------------------ rows, 1 x 128 blocks
// A team of 128 / V lanes per block (V elements in one 16-byte load per lane), so a warp's loads
// and stores are contiguous.
template <typename Tin>
__global__ void __launch_bounds__(256)
    quantize_block_rows_kernel(const Tin *__restrict__ in, long long rows, int cols, int nblk,
                               const int32_t *__restrict__ n_rows, uint8_t *__restrict__ q,
                               uint8_t *__restrict__ scale) {
  constexpr int V = 16 / sizeof(Tin), L = QB / V, TPB = 256 / L;
  const KernelStamp stamp(K_F8B_QUANT);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const long long nr = valid_rows(rows, n_rows);
  const int c0 = (threadIdx.x % L) * V;
  BlockWalk w((long long)blockIdx.x * TPB + threadIdx.x / L, (long long)gridDim.x * TPB, nblk);
  // whole warps walk together (the shuffles need every lane): a lane past the end works on zeros
  const long long total = nr * nblk;
  for (long long b0 = (long long)blockIdx.x * TPB + (threadIdx.x / 32) * (32 / L); b0 < total;
       b0 += (long long)gridDim.x * TPB, w.next()) {
    const int col = w.blk * QB + c0;
    const bool ok = w.row < nr && col < cols;
    Pack<Tin, V> p;
    if (ok) p.load(in + w.row * cols + col);
    else p.zero();
    float v[V];
    p.values(v);
    const uint32_t b = e8m0_of_amax(team_max<L>(amax_bits(v)));
    if (ok) store_codes(q + w.row * cols + col, v, e8m0_inverse(b));
    if (c0 == 0 && w.row < nr) scale[w.row * nblk + w.blk] = (uint8_t)b;
  }
}

// ------------------------------------------------------------------ a 128 x 128 tile, transposed
// The codes of a tile in shared memory as words of four rows: word a of column c (rows 4a .. 4a+3)
// at c * 32 + (a ^ key(c)). The key sends the V-column lanes of a warp's stores to 32 different
// banks and leaves the reads of one column a permutation of the banks.
constexpr int F8T_THREADS = 256;
template <int V> __device__ __forceinline__ int tile_key(int c) { return (c / V) * (V / 4); }

// 4 x 4 byte transpose: in[i] holds four columns of row i, out[j] the four rows of column j.
__device__ __forceinline__ void transpose4(const uint32_t (&in)[4], uint32_t (&out)[4]) {
  const uint32_t a = __byte_perm(in[0], in[1], 0x5140), b = __byte_perm(in[2], in[3], 0x5140);
  const uint32_t c = __byte_perm(in[0], in[1], 0x7362), d = __byte_perm(in[2], in[3], 0x7362);
  out[0] = __byte_perm(a, b, 0x5410);
  out[1] = __byte_perm(a, b, 0x7632);
  out[2] = __byte_perm(c, d, 0x5410);
  out[3] = __byte_perm(c, d, 0x7632);
}
// w[i][j]: codes of row 4a + i, columns col + 4j .. col + 4j + 3.
template <int V>
__device__ __forceinline__ void tile_put(uint32_t *tile, int a, int col, const uint32_t (&w)[4][V / 4]) {
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    const uint32_t in[4] = {w[0][j], w[1][j], w[2][j], w[3][j]};
    uint32_t out[4];
    transpose4(in, out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = col + 4 * j + i;
      tile[c * 32 + (a ^ tile_key<V>(c))] = out[i];
    }
  }
}
// Columns of the tile to dst[c * pitch + r], c < cols, r < rows (a multiple of 4): one warp per
// column, 4 rows per lane.
template <int V>
__device__ __forceinline__ void tile_write(const uint32_t *tile, uint8_t *dst, size_t pitch, int cols,
                                           int rows) {
  const int lane = threadIdx.x & 31;
  for (int c = threadIdx.x >> 5; c < cols; c += F8T_THREADS / 32)
    if (4 * lane < rows) *(uint32_t *)(dst + c * pitch + 4 * lane) = tile[c * 32 + (lane ^ tile_key<V>(c))];
}

// ------------------------------------------------------------------ weights, 128 x 128 blocks
// One CTA per block; q_t, scale_t (may be null) receive the transposed matrix, whose blocks and
// scales are the same ones.
template <typename Tin>
__global__ void __launch_bounds__(F8T_THREADS)
    quantize_block_weight_kernel(const Tin *__restrict__ in, int rows, int cols,
                                 uint8_t *__restrict__ q, uint8_t *__restrict__ scale,
                                 uint8_t *__restrict__ q_t, uint8_t *__restrict__ scale_t) {
  constexpr int V = 16 / sizeof(Tin), L = QB / V, A = F8T_THREADS / L, PASS = 32 / A;
  __shared__ uint32_t tile[QB * 32];
  __shared__ uint32_t wmax[F8T_THREADS / 32];
  const KernelStamp stamp(K_F8B_QUANT);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const int nbr = gridDim.y, nbc = gridDim.x, e = blockIdx.z;
  const int r0 = blockIdx.y * QB, c0 = (threadIdx.x % L) * V, col = blockIdx.x * QB + c0;
  const int a0 = threadIdx.x / L;
  const size_t base = (size_t)e * rows * cols;
  Pack<Tin, V> p[PASS][4];
#pragma unroll
  for (int s = 0; s < PASS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * (a0 + s * A) + i;
      if (r < rows && col < cols) p[s][i].load(in + base + (size_t)r * cols + col);
      else p[s][i].zero();
    }
  uint32_t m = 0;
#pragma unroll
  for (int s = 0; s < PASS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[V];
      p[s][i].values(v);
      m = max(m, amax_bits(v));
    }
  m = team_max<32>(m);
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < F8T_THREADS / 32; ++i) m = max(m, wmax[i]);
  const uint32_t b = e8m0_of_amax(m);
  const float inv = e8m0_inverse(b);
  if (threadIdx.x == 0) {
    scale[((size_t)e * nbr + blockIdx.y) * nbc + blockIdx.x] = (uint8_t)b;
    if (scale_t) scale_t[((size_t)e * nbc + blockIdx.x) * nbr + blockIdx.y] = (uint8_t)b;
  }
#pragma unroll
  for (int s = 0; s < PASS; ++s) {
    uint32_t w[4][V / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[V];
      p[s][i].values(v);
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        w[i][j] = e4m3x4(v[4 * j] * inv, v[4 * j + 1] * inv, v[4 * j + 2] * inv, v[4 * j + 3] * inv);
      const int r = r0 + 4 * (a0 + s * A) + i;
      if (r < rows && col < cols) {
        uint8_t *dst = q + base + (size_t)r * cols + col;
        if (V == 8) *(uint2 *)dst = make_uint2(w[i][0], w[i][V / 4 - 1]);
        else *(uint32_t *)dst = w[i][0];
      }
    }
    if (q_t) tile_put<V>(tile, a0 + s * A, c0, w);
  }
  if (!q_t) return;
  __syncthreads();
  tile_write<V>(tile, q_t + base + (size_t)blockIdx.x * QB * rows + r0, rows,
                min(QB, cols - (int)blockIdx.x * QB), min(QB, rows - r0));
}

// ------------------------------------------------------------------ tokens, 128 x 1 blocks
// Expert e's rows [offsets[e], offsets[e+1]) (clamped to [0, rows]) in blocks of 128 from its own
// first row; block number `blk` in expert order. Every lane of a warp calls; returns false when
// there are fewer blocks.
struct TokenBlock {
  long long row0;  // first row
  int n;           // rows in it (1 .. 128)
};
__device__ __forceinline__ long long expert_bound(const int32_t *offsets, int e, long long rows) {
  return min(max((long long)__ldg(offsets + e), 0ll), rows);
}
__device__ __forceinline__ bool find_token_block(const int32_t *offsets, int E, long long rows,
                                                 long long blk, TokenBlock *out) {
  const int lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    long long a = 0;
    int n = 0;
    if (e < E) {
      a = expert_bound(offsets, e, rows);
      n = (int)max(expert_bound(offsets, e + 1, rows) - a, 0ll);
    }
    const int nb = (n + QB - 1) / QB;
    const int incl = warp_incl_scan(nb);
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (blk < total) {
      const unsigned past = __ballot_sync(0xffffffffu, (long long)incl > blk);
      const int src = __ffs(past) - 1;
      const int j = (int)blk - (__shfl_sync(0xffffffffu, incl, src) - __shfl_sync(0xffffffffu, nb, src));
      out->row0 = __shfl_sync(0xffffffffu, a, src) + (long long)j * QB;
      out->n = min(QB, __shfl_sync(0xffffffffu, n, src) - j * QB);
      return true;
    }
    blk -= total;
  }
  return false;
}

// One CTA per (block, 128 columns): codes transposed to q_t [cols, pitch] at column 128 blk, scales
// to scale_t [., cols]. Rows past the expert's last are zeros. Tin uint8_t: E4M3 codes with 1 x 128
// scale bytes in_scale [rows, ceil(cols / 128)] (an 8-bit checkpoint), read without a bf16 copy.
template <typename Tin>
__global__ void __launch_bounds__(F8T_THREADS)
    quantize_block_tokens_kernel(const Tin *__restrict__ in, const uint8_t *__restrict__ in_scale,
                                 long long rows, int cols, const int32_t *__restrict__ offsets, int E,
                                 uint8_t *__restrict__ q_t, size_t pitch,
                                 uint8_t *__restrict__ scale_t) {
  constexpr int V = 16 / sizeof(Tin), L = QB / V, A = F8T_THREADS / L, PASS = 32 / A;
  __shared__ uint32_t tile[QB * 32];
  __shared__ uint32_t cmax[F8T_THREADS / 32][QB];
  const KernelStamp stamp(K_F8B_QUANT);
  griddep_wait();
  stamp.started();
  griddep_launch();
  TokenBlock tb;
  const int ntile = (cols + QB - 1) / QB, ct = blockIdx.x % ntile;  // column tiles of a block adjoin
  const int blk = blockIdx.x / ntile;
  if (!find_token_block(offsets, E, rows, blk, &tb)) return;
  const int c0 = (threadIdx.x % L) * V, col = ct * QB + c0, a0 = threadIdx.x / L;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pack<Tin, V> p[PASS][4];
  float rs[PASS][4];  // the rows' own scales (8-bit input)
#pragma unroll
  for (int s = 0; s < PASS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * (a0 + s * A) + i;
      rs[s][i] = 1.0f;
      if (r < tb.n && col < cols) {
        p[s][i].load(in + (tb.row0 + r) * cols + col);
        if (sizeof(Tin) == 1)
          rs[s][i] = e8m0_value(__ldg(in_scale + (tb.row0 + r) * ntile + ct));
      } else {
        p[s][i].zero();
      }
    }
  uint32_t m[V];
#pragma unroll
  for (int j = 0; j < V; ++j) m[j] = 0;
#pragma unroll
  for (int s = 0; s < PASS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[V];
      p[s][i].values(v);
#pragma unroll
      for (int j = 0; j < V; ++j) m[j] = max(m[j], abs_bits(v[j] * rs[s][i]));
    }
#pragma unroll
  for (int o = L; o < 32; o <<= 1)  // lanes of the warp that hold the same columns
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
  if (lane < L)
#pragma unroll
    for (int j = 0; j < V; ++j) cmax[warp][c0 + j] = m[j];
  __syncthreads();
  if (threadIdx.x < QB) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < F8T_THREADS / 32; ++i) x = max(x, cmax[i][threadIdx.x]);
    const uint32_t b = e8m0_of_amax(x);
    if (ct * QB + (int)threadIdx.x < cols)
      scale_t[(size_t)blk * cols + ct * QB + threadIdx.x] = (uint8_t)b;
    cmax[0][threadIdx.x] = __float_as_uint(e8m0_inverse(b));
  }
  __syncthreads();
  float inv[V];
#pragma unroll
  for (int j = 0; j < V; ++j) inv[j] = __uint_as_float(cmax[0][c0 + j]);
#pragma unroll
  for (int s = 0; s < PASS; ++s) {
    uint32_t w[4][V / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[V];
      p[s][i].values(v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] *= rs[s][i];
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        w[i][j] = e4m3x4(v[4 * j] * inv[4 * j], v[4 * j + 1] * inv[4 * j + 1],
                         v[4 * j + 2] * inv[4 * j + 2], v[4 * j + 3] * inv[4 * j + 3]);
    }
    tile_put<V>(tile, a0 + s * A, c0, w);
  }
  __syncthreads();
  tile_write<V>(tile, q_t + (size_t)ct * QB * pitch + (size_t)blk * QB, pitch, min(QB, cols - ct * QB),
                QB);
}

// ------------------------------------------------------------------ SwiGLU with a checkpoint
// sigmoid(z) = 1 / (1 + e^-z): for z below about -88 the exponential is infinite and the result 0.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// gu [rows, 2 f] = [gate | up]: h = silu(g) u, to h (bf16) and / or h_q + h_scale (the down product's
// operand, quantised from the fp32 value), and the E4M3 codes of gu itself to gu_q + gu_scale (the
// checkpoint of the backward pass). f a multiple of 128, so no block spans gate and up.
template <typename Tin>
__global__ void __launch_bounds__(256)
    swiglu_checkpoint_kernel(const Tin *__restrict__ gu, long long rows, int f,
                             const int32_t *__restrict__ n_rows, __nv_bfloat16 *__restrict__ h,
                             uint8_t *__restrict__ h_q, uint8_t *__restrict__ h_scale,
                             uint8_t *__restrict__ gu_q, uint8_t *__restrict__ gu_scale) {
  constexpr int V = 8, L = QB / V, TPB = 256 / L;
  const KernelStamp stamp(K_F8B_SWIGLU);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const long long nr = valid_rows(rows, n_rows);
  const int nb = f / QB, c0 = (threadIdx.x % L) * V;
  BlockWalk w((long long)blockIdx.x * TPB + threadIdx.x / L, (long long)gridDim.x * TPB, nb);
  const long long total = nr * nb;
  for (long long b0 = (long long)blockIdx.x * TPB + (threadIdx.x / 32) * (32 / L); b0 < total;
       b0 += (long long)gridDim.x * TPB, w.next()) {
    const int col = w.blk * QB + c0;
    const bool ok = w.row < nr;
    Pack<Tin, V> pg, pu;
    if (ok) {
      pg.load(gu + w.row * 2 * f + col);
      pu.load(gu + w.row * 2 * f + f + col);
    } else {
      pg.zero();
      pu.zero();
    }
    float g[V], u[V], hv[V];
    pg.values(g);
    pu.values(u);
#pragma unroll
    for (int i = 0; i < V; ++i) hv[i] = g[i] * sigmoid_f(g[i]) * u[i];
    if (gu_q) {
      const uint32_t bg = e8m0_of_amax(team_max<L>(amax_bits(g)));
      const uint32_t bu = e8m0_of_amax(team_max<L>(amax_bits(u)));
      if (ok) {
        store_codes(gu_q + w.row * 2 * f + col, g, e8m0_inverse(bg));
        store_codes(gu_q + w.row * 2 * f + f + col, u, e8m0_inverse(bu));
        if (c0 == 0) {
          gu_scale[w.row * 2 * nb + w.blk] = (uint8_t)bg;
          gu_scale[w.row * 2 * nb + nb + w.blk] = (uint8_t)bu;
        }
      }
    }
    if (h_q) {
      const uint32_t bh = e8m0_of_amax(team_max<L>(amax_bits(hv)));
      if (ok) {
        store_codes(h_q + w.row * f + col, hv, e8m0_inverse(bh));
        if (c0 == 0) h_scale[w.row * nb + w.blk] = (uint8_t)bh;
      }
    }
    if (h && ok) store_bf16x8(h + w.row * f + col, hv);
  }
}

// From the checkpoint and dh: s = sigmoid(g), du = dh g s, dg = dh u s (1 + g (1 - s)), h = g s u.
// dgu = [dg | du] in bf16 and / or as E4M3 codes (the input gradient's operand, quantised from the
// fp32 values); h in bf16 (the down weight gradient's operand).
template <typename Tin>
__global__ void __launch_bounds__(256)
    swiglu_checkpoint_backward_kernel(const uint8_t *__restrict__ gu_q,
                                      const uint8_t *__restrict__ gu_scale,
                                      const Tin *__restrict__ dh, long long rows, int f,
                                      const int32_t *__restrict__ n_rows,
                                      __nv_bfloat16 *__restrict__ dgu, uint8_t *__restrict__ dgu_q,
                                      uint8_t *__restrict__ dgu_scale, __nv_bfloat16 *__restrict__ h) {
  constexpr int V = 8, L = QB / V, TPB = 256 / L;
  const KernelStamp stamp(K_F8B_SWIGLU);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const long long nr = valid_rows(rows, n_rows);
  const int nb = f / QB, c0 = (threadIdx.x % L) * V;
  BlockWalk w((long long)blockIdx.x * TPB + threadIdx.x / L, (long long)gridDim.x * TPB, nb);
  const long long total = nr * nb;
  for (long long b0 = (long long)blockIdx.x * TPB + (threadIdx.x / 32) * (32 / L); b0 < total;
       b0 += (long long)gridDim.x * TPB, w.next()) {
    const int col = w.blk * QB + c0;
    const bool ok = w.row < nr;
    const long long at = w.row * 2 * f + col;
    uint2 cg = make_uint2(0u, 0u), cu = cg;
    float sg = 1.0f, su = 1.0f;
    Pack<Tin, V> pd;
    if (ok) {
      cg = __ldg((const uint2 *)(gu_q + at));
      cu = __ldg((const uint2 *)(gu_q + at + f));
      sg = e8m0_value(__ldg(gu_scale + w.row * 2 * nb + w.blk));
      su = e8m0_value(__ldg(gu_scale + w.row * 2 * nb + nb + w.blk));
      pd.load(dh + w.row * f + col);
    } else {
      pd.zero();
    }
    float d[V], dg[V], du[V], hv[V];
    pd.values(d);
    const uint32_t wg[2] = {cg.x, cg.y}, wu[2] = {cu.x, cu.y};
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 g2 = e4m3x2_values((wg[i / 4] >> (8 * (i % 4))) & 0xffffu);
      const float2 u2 = e4m3x2_values((wu[i / 4] >> (8 * (i % 4))) & 0xffffu);
      const float gg[2] = {g2.x * sg, g2.y * sg}, uu[2] = {u2.x * su, u2.y * su};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float s = sigmoid_f(gg[j]), gs = gg[j] * s;
        du[i + j] = d[i + j] * gs;
        dg[i + j] = d[i + j] * uu[j] * (s * (1.0f + gg[j] * (1.0f - s)));
        hv[i + j] = gs * uu[j];
      }
    }
    if (dgu_q) {
      const uint32_t bg = e8m0_of_amax(team_max<L>(amax_bits(dg)));
      const uint32_t bu = e8m0_of_amax(team_max<L>(amax_bits(du)));
      if (ok) {
        store_codes(dgu_q + at, dg, e8m0_inverse(bg));
        store_codes(dgu_q + at + f, du, e8m0_inverse(bu));
        if (c0 == 0) {
          dgu_scale[w.row * 2 * nb + w.blk] = (uint8_t)bg;
          dgu_scale[w.row * 2 * nb + nb + w.blk] = (uint8_t)bu;
        }
      }
    }
    if (ok && dgu) {
      store_bf16x8(dgu + at, dg);
      store_bf16x8(dgu + at + f, du);
    }
    if (ok && h) store_bf16x8(h + w.row * f + col, hv);
  }
}

}  // namespace moe
