// Block-scaled E4M3: quantisers and the SwiGLU with an 8-bit activation checkpoint.
//
// A block of 128 values shares one E8M0 scale byte b, worth 2^(b - 127): the least power of two
// with amax / scale <= 448 (not below 2^-126; 1 for an all-zero block). Dividing by a power of two
// is exact in fp32 (a quotient that underflows is far below half the least E4M3 value), so a code
// is the value's nearest E4M3 number, ties to even, and that is the only rounding anywhere here.
// Blocks run along a row (1 x 128), are square (128 x 128, weights), or run along the rows of one
// expert (128 x 1, the operands of a weight gradient, whose inner dimension is the token).
//
// All of these kernels move each byte once: 16-byte loads per lane, the block maximum by warp
// shuffles, the values held in registers between the maximum and the conversion. The row-wise ones and
// the weights are bound by HBM (inputs from DRAM: rows 131,072 x 1,536 bf16 90.3 us, 6.7 TB/s; weights
// 24 x 1,280 x 1,024 with the transposed copy 21.7 us, 5.8 TB/s; SwiGLU forward 24,576 x 640 23 us,
// 4.8 TB/s, backward 131,072 x 768 193 us, 6.3 TB/s). The token quantiser (24,576 x 1,024 over 24 experts:
// 18.8 us from E4M3 rows, 19.9 from bf16) is bound by the order of its phases: no pipe is full (issue slots
// 61%, ALU 45% of the active cycles), its warps wait for loads, for shared memory and at barriers in turn.
#pragma once
#include <cuda_fp8.h>

#include <cfloat>

#include "common.cuh"

namespace moe {

constexpr int QB = 128;  // values per block
constexpr long long INFO_OFFSETS_DECREASE = 4;  // detail code beside those of common.cuh

// ------------------------------------------------------------------ the format
// Scale byte of a block from the bits of its largest magnitude: amax = m 2^e with 1 <= m < 2 and
// 448 = 1.75 * 2^8, so the exponent is e - 8, one more when m > 1.75 (the carry of the addition).
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t amax_bits) {
  if (amax_bits == 0) return 127;
  const int b = (int)((amax_bits + 0x1FFFFFu) >> 23) - 8;
  return (uint32_t)max(b, 1);
}
// 2^(b - 127), and its reciprocal, a normal number for the bytes 1 .. 247 of finite fp32 values
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
  __device__ __forceinline__ void values4(int j, float (&v)[4]) const {  // elements 4 j .. 4 j + 3
    v[0] = r[j].x;
    v[1] = r[j].y;
    v[2] = r[j].z;
    v[3] = r[j].w;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      m = max(m, max(max(abs_bits(r[i].x), abs_bits(r[i].y)), max(abs_bits(r[i].z), abs_bits(r[i].w))));
    return m;
  }
};
// (amax: the bits of the largest magnitude)
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
  __device__ __forceinline__ void values4(int j, float (&v)[4]) const {
    const uint32_t a = j & 1 ? r[j / 2].z : r[j / 2].x, b = j & 1 ? r[j / 2].w : r[j / 2].y;
    v[0] = __uint_as_float(a << 16);
    v[1] = __uint_as_float(a & 0xffff0000u);
    v[2] = __uint_as_float(b << 16);
    v[3] = __uint_as_float(b & 0xffff0000u);
  }
  __device__ __forceinline__ uint32_t amax() const {  // two at a time: magnitudes order as integers
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V / 8; ++i) {
      const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
    }
    return max(m << 16, m & 0x7fff0000u);
  }
};
// E4M3 codes (a row's block scale applied by the caller).
template <int V> struct Pack<uint8_t, V> {
  static_assert(V == 16, "one 16-byte load");
  uint4 r;
  __device__ __forceinline__ void load(const uint8_t *p) { r = __ldg((const uint4 *)p); }
  __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void values4(int j, float (&v)[4]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    const float2 a = e4m3x2_values(w[j] & 0xffffu), b = e4m3x2_values(w[j] >> 16);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
  }
};

template <int V> __device__ __forceinline__ uint32_t amax_bits(const float (&v)[V]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, abs_bits(v[i]));
  return m;
}
// 8 codes of v * inv to q (8-byte aligned).
__device__ __forceinline__ void store_codes(uint8_t *q, const float (&v)[8], float inv) {
  *(uint2 *)q = make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                           e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
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

// Row-wise kernels: a team of 8 lanes per block of 128, 16 values per lane (8 at 8 l and 8 at
// 64 + 8 l, so that each 16-byte load of bf16 and 8-byte store of codes is contiguous over the team).
// With 8 values per lane the kernels issued twice the instructions per value and were bound by
// that. Teams take every `step`-th block of the flat list; a warp's four teams walk together (the
// shuffles need every lane), lanes past the end work on zeros.
constexpr int RT_LANES = 8, RT_TEAMS = 256 / RT_LANES;
struct RowTeam {
  long long first;  // this warp's first block
  long long step;
  int team, c;      // team in the warp, first column of this lane
  __device__ __forceinline__ RowTeam()
      : first((long long)blockIdx.x * RT_TEAMS + (threadIdx.x >> 5) * 4), step((long long)gridDim.x * RT_TEAMS),
        team((threadIdx.x & 31) / RT_LANES), c((threadIdx.x % RT_LANES) * 8) {}
};
// 16 values of a block at src + c and src + c + 64.
template <typename T> struct Lane16 {
  Pack<T, 8> p[2];
  __device__ __forceinline__ void load(const T *src) {
    p[0].load(src);
    p[1].load(src + 64);
  }
  __device__ __forceinline__ void zero() {
    p[0].zero();
    p[1].zero();
  }
  __device__ __forceinline__ uint32_t amax() const { return max(p[0].amax(), p[1].amax()); }
};
__device__ __forceinline__ uint32_t block_byte(uint32_t lane_amax) {
  return e8m0_of_amax(team_max<RT_LANES>(lane_amax));
}

// A lane's offset in rows of `pitch` elements that start with `nb` blocks, walked in flat block order
// (block b is block b % nb of row b / nb) without a division per step. SwiGLU: the gate blocks of
// [., 2 f] rows; the up columns are f further.
struct FlatWalk {
  long long off, doff;
  int blk, nb, dblk, wrap;
  __device__ __forceinline__ FlatWalk(const RowTeam &w, int nb_, int pitch) : nb(nb_), wrap(pitch - nb_ * QB) {
    const long long b = w.first + w.team, row = b / nb, drow = w.step / nb;
    blk = (int)(b - row * nb);
    off = row * pitch + blk * QB + w.c;
    dblk = (int)(w.step - drow * nb);
    doff = drow * pitch + dblk * QB;
  }
  __device__ __forceinline__ void next() {
    off += doff;
    blk += dblk;
    if (blk >= nb) {  // the next row, nb blocks back
      blk -= nb;
      off += wrap;
    }
  }
};

// ------------------------------------------------------------------ rows, 1 x 128 blocks
constexpr int F8Q_U = 2;  // blocks in flight per team: 64 bytes per lane, which HBM's latency asks for

// FULL: cols a multiple of 128, so a block's flat number places it without its row and column.
template <typename Tin, bool FULL>
__global__ void __launch_bounds__(256, 4)
    quantize_block_rows_kernel(const Tin *__restrict__ in, long long rows, int cols, int nblk,
                               const int32_t *__restrict__ n_rows, uint8_t *__restrict__ q,
                               uint8_t *__restrict__ scale) {
  constexpr int U = F8Q_U;
  const KernelStamp stamp(K_F8B_QUANT);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const RowTeam w;
  const long long total = valid_rows(rows, n_rows) * nblk;
  FlatWalk at(w, nblk, cols);
  for (long long b0 = w.first; b0 < total; b0 += U * w.step) {
    Lane16<Tin> x[U];
    long long off[U];
    bool ok[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long b = b0 + u * w.step + w.team;
      ok[u][0] = ok[u][1] = b < total;
      if (FULL) {
        off[u] = b * QB + w.c;
      } else {
        off[u] = at.off;
        ok[u][0] &= at.blk * QB + w.c < cols;
        ok[u][1] &= at.blk * QB + w.c + 64 < cols;
        at.next();
      }
      x[u].zero();
      if (ok[u][0]) x[u].p[0].load(in + off[u]);
      if (ok[u][1]) x[u].p[1].load(in + off[u] + 64);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long b = b0 + u * w.step + w.team;
      const uint32_t byte = block_byte(x[u].amax());
      const float inv = e8m0_inverse(byte);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
        x[u].p[h].values(v);
        if (ok[u][h]) store_codes(q + off[u] + 64 * h, v, inv);
      }
      if (w.c == 0 && b < total) scale[b] = (uint8_t)byte;
    }
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
// w[i][j]: codes of row 4a + i, columns col + 4j .. col + 4j + 3 (W columns).
template <int V, int W = V>
__device__ __forceinline__ void tile_put(uint32_t *tile, int a, int col, const uint32_t (&w)[4][W / 4]) {
#pragma unroll
  for (int j = 0; j < W / 4; ++j) {
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
// Columns of the tile to dst[c * pitch + r], c < cols, r < rows (a multiple of 16): 8 lanes per column,
// 16 rows per lane. The key permutes the words of a 16-byte group among themselves and the groups of
// a column among themselves.
template <int V>
__device__ __forceinline__ void tile_write(const uint32_t *tile, uint8_t *dst, size_t pitch, int cols,
                                           int rows) {
  const int g = threadIdx.x & 7;
  if (16 * g >= rows) return;
  dst += (threadIdx.x >> 3) * pitch + 16 * g;
#pragma unroll
  for (int c = threadIdx.x >> 3; c < QB; c += F8T_THREADS / 8, dst += F8T_THREADS / 8 * pitch) {
    if (c >= cols) break;
    const int key = tile_key<V>(c);
    uint4 v = *(const uint4 *)(tile + c * 32 + 4 * (g ^ (key >> 2)));
    if (key & 1) v = make_uint4(v.y, v.x, v.w, v.z);
    if (key & 2) v = make_uint4(v.z, v.w, v.x, v.y);
    *(uint4 *)dst = v;
  }
}

// ------------------------------------------------------------------ weights, 128 x 128 blocks
// One CTA per block; q_t, scale_t (may be null) receive the transposed matrix, whose blocks and
// scales are the same ones.
template <typename Tin>
__global__ void __launch_bounds__(F8T_THREADS, sizeof(Tin) == 4 ? 2 : 4)
    quantize_block_weight_kernel(const Tin *__restrict__ in, int rows, int cols,
                                 uint8_t *__restrict__ q, uint8_t *__restrict__ scale,
                                 uint8_t *__restrict__ q_t, uint8_t *__restrict__ scale_t) {
  constexpr int V = 16 / sizeof(Tin), L = QB / V, A = F8T_THREADS / L, PASS = 32 / A;
  __shared__ __align__(16) uint32_t tile[QB * 32];
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
    for (int i = 0; i < 4; ++i) m = max(m, p[s][i].amax());
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
  int row0;  // first row
  int n;     // rows in it (1 .. 128)
};
__device__ __forceinline__ long long expert_bound(const int32_t *offsets, int e, long long rows) {
  return min(max((long long)__ldg(offsets + e), 0ll), rows);
}
// Offsets must not decrease (their clamped values then add up to at most `rows`): otherwise an error
// is recorded and the caller does nothing.
__device__ __forceinline__ bool offsets_decrease(bool bad) {
  if (bad && threadIdx.x == 0) set_device_error(MOE_ERR_DEVICE_CHECK, INFO_OFFSETS_DECREASE);
  return bad;
}
// All offsets, by one warp: a CTA's search ends at its block or group of rows, so that the experts behind
// the last one's are seen by none. The grid's last CTA calls this when its own work is done (within the
// search it cost registers that the quantiser needs: 17.8 -> 20.4 us).
__device__ __forceinline__ void check_offsets(const int32_t *offsets, int E, long long rows) {
  bool bad = false;
  for (int e = threadIdx.x & 31; e < E; e += 32)
    bad |= expert_bound(offsets, e + 1, rows) < expert_bound(offsets, e, rows);
  offsets_decrease(__any_sync(0xffffffffu, bad));
}
__device__ __forceinline__ bool find_token_block(const int32_t *offsets, int E, long long rows, int blk,
                                                 TokenBlock *out) {
  const int lane = threadIdx.x & 31;
  for (int e0 = 0; e0 < E; e0 += 32) {
    int a = 0, n = 0;
    if (e0 + lane < E) {
      a = (int)expert_bound(offsets, e0 + lane, rows);
      n = (int)expert_bound(offsets, e0 + lane + 1, rows) - a;
    }
    if (offsets_decrease(__any_sync(0xffffffffu, n < 0))) return false;
    const int nb = (n + QB - 1) / QB;
    const int incl = warp_incl_scan(nb);
    const unsigned past = __ballot_sync(0xffffffffu, incl > blk);
    if (past) {
      const int src = __ffs(past) - 1;
      const int j = blk - __shfl_sync(0xffffffffu, incl - nb, src);
      out->row0 = __shfl_sync(0xffffffffu, a, src) + j * QB;
      out->n = min(QB, __shfl_sync(0xffffffffu, n, src) - j * QB);
      return true;
    }
    blk -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// A tile of codes with values past fp32's largest (2^-135 .. 448 2^127 are possible): its column bytes,
// and its codes into shared memory. 2^-8 of a value is exact in fp32, its subnormals included, and of an
// amax that small the byte is the exponent of the largest (that it is one of fp32's subnormals below
// 2^-118 makes no difference, as byte 1 is the least). A code times 2^(row's byte - column's byte) is one
// exact product: a factor past 2^127 meets only zero codes, and what one below 2^-126 (taken as 0) meets
// is far below half the least code. Rows of finite fp32 values have at most a few such values (above
// 1.9375 2^127 they round up to 2^128), so this reads its inputs again and is not made fast; a call of
// its own after the ordinary encoding, so that other tiles lose little (17.8 -> 18.2 us; 18.9 as a branch
// before the encoding, 21 inlined there).
__device__ __noinline__ void put_loud_tile(const uint8_t *src, const uint8_t *src_scale, int cols, int ntile,
                                           int n, int left_cols, uint32_t *tile, uint8_t *col_byte,
                                           uint8_t *scale_t) {
  const int c = threadIdx.x;
  if (c < QB) {
    uint32_t b = 127;
    if (c < left_cols) {
      float m = 0.0f;
      for (int r = 0; r < n; ++r) {
        const float v = e4m3x2_values(src[(size_t)r * cols + c]).x;
        m = fmaxf(m, fabsf(v * (e8m0_value(src_scale[(size_t)r * ntile]) * 0x1p-8f)));
      }
      if (m > 0.0f) b = max((__float_as_uint(m) + 0x1FFFFFu) >> 23, 1u);
      scale_t[c] = (uint8_t)b;
    }
    col_byte[c] = (uint8_t)b;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < QB / 4 * (QB / 4); i += F8T_THREADS) {  // words of 4 rows by 4 columns
    const int a = i / (QB / 4), c0 = i % (QB / 4) * 4;
    uint32_t w[4][1] = {};
    for (int r = 4 * a; r < min(n, 4 * a + 4) && c0 < left_cols; ++r) {
      const uint32_t codes = *(const uint32_t *)(src + (size_t)r * cols + c0);
      const int row = src_scale[(size_t)r * ntile];
      const float2 lo = e4m3x2_values(codes & 0xffffu), hi = e4m3x2_values(codes >> 16);
      float f[4];
      for (int x = 0; x < 4; ++x)
        f[x] = __uint_as_float((uint32_t)min(max(row - col_byte[c0 + x] + 127, 0), 254) << 23);
      w[r & 3][0] = e4m3x4(lo.x * f[0], lo.y * f[1], hi.x * f[2], hi.y * f[3]);
    }
    tile_put<16, 4>(tile, a, c0, w);
  }
}

// One CTA per (block, 128 columns): codes transposed to q_t [cols, pitch] at column 128 blk, scales
// to scale_t [., cols]. Rows past the expert's last are zeros. Tin uint8_t: E4M3 codes with 1 x 128
// scale bytes in_scale [rows, ceil(cols / 128)] (an 8-bit checkpoint), read without a bf16 copy.
template <typename Tin>
__global__ void __launch_bounds__(F8T_THREADS, sizeof(Tin) == 4 ? 2 : 4)
    quantize_block_tokens_kernel(const Tin *__restrict__ in, const uint8_t *__restrict__ in_scale,
                                 long long rows, int cols, const int32_t *__restrict__ offsets, int E,
                                 uint8_t *__restrict__ q_t, size_t pitch,
                                 uint8_t *__restrict__ scale_t) {
  constexpr int V = 16 / sizeof(Tin), L = QB / V, A = F8T_THREADS / L, PASS = 32 / A;
  constexpr bool CODES = sizeof(Tin) == 1;
  __shared__ int loud;  // set by a value past fp32's largest (codes alone can stand for one)
  __shared__ __align__(16) uint32_t tile[QB * 32];
  __shared__ __align__(16) float cmax[F8T_THREADS / 32][QB];
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
  const size_t row = (size_t)tb.row0 + 4 * a0;  // this thread's first
  const Tin *src = in + row * cols + col;
  const uint8_t *src_scale = in_scale + row * ntile + ct;
  const int left = col < cols ? tb.n - 4 * a0 : 0;
#pragma unroll
  for (int s = 0; s < PASS; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rs[s][i] = 1.0f;
      if (4 * A * s + i < left) {
        p[s][i].load(src + (size_t)(4 * A * s + i) * cols);
        if (sizeof(Tin) == 1) rs[s][i] = e8m0_value(__ldg(src_scale + (size_t)(4 * A * s + i) * ntile));
      } else {
        p[s][i].zero();
      }
    }
  // column maxima, four columns (one word of codes to come) at a time
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < PASS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
        p[s][i].values4(j, v);
#pragma unroll
        for (int x = 0; x < 4; ++x) m[x] = fmaxf(m[x], fabsf(v[x] * rs[s][i]));
      }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
#pragma unroll
      for (int o = L; o < 32; o <<= 1)  // lanes of the warp that hold the same columns
        m[x] = fmaxf(m[x], __shfl_xor_sync(0xffffffffu, m[x], o));
    }
    if (lane < L) *(float4 *)&cmax[warp][c0 + 4 * j] = make_float4(m[0], m[1], m[2], m[3]);
  }
  if (CODES && threadIdx.x == 0) loud = 0;
  __syncthreads();
  if (threadIdx.x < QB) {
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < F8T_THREADS / 32; ++i) x = fmaxf(x, cmax[i][threadIdx.x]);
    const uint32_t b = e8m0_of_amax(__float_as_uint(x));
    if (ct * QB + (int)threadIdx.x < cols)
      scale_t[(size_t)blk * cols + ct * QB + threadIdx.x] = (uint8_t)b;
    cmax[0][threadIdx.x] = e8m0_inverse(b);
    if (CODES && x > FLT_MAX) loud = 1;
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < PASS; ++s) {
    uint32_t w[4][V / 4];
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const float4 inv = *(const float4 *)&cmax[0][c0 + 4 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
        p[s][i].values4(j, v);
        w[i][j] = e4m3x4(v[0] * rs[s][i] * inv.x, v[1] * rs[s][i] * inv.y, v[2] * rs[s][i] * inv.z,
                         v[3] * rs[s][i] * inv.w);
      }
    }
    tile_put<V>(tile, a0 + s * A, c0, w);
  }
  __syncthreads();
  if (CODES && loud) {  // again, at the end, where the registers are free
    find_token_block(offsets, E, rows, blk, &tb);
    put_loud_tile((const uint8_t *)in + (size_t)tb.row0 * cols + ct * QB,
                  in_scale + (size_t)tb.row0 * ntile + ct, cols, ntile, tb.n, cols - ct * QB, tile,
                  (uint8_t *)cmax[1], scale_t + (size_t)blk * cols + ct * QB);
    __syncthreads();
  }
  tile_write<V>(tile, q_t + (size_t)ct * QB * pitch + (size_t)blk * QB, pitch, min(QB, cols - ct * QB),
                QB);
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x < 32) check_offsets(offsets, E, rows);
}

// ------------------------------------------------------------------ SwiGLU with a checkpoint
// sigmoid(z) = 1 / (1 + 2^(-z log2 e)) by the fast exponential and reciprocal (2 ulp and 1 ulp);
// for z below about -88 the exponential is infinite and the result 0.
__device__ __forceinline__ float sigmoid_f(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
// gu [rows, 2 f] = [gate | up]: h = silu(g) u, to h (bf16) and / or h_q + h_scale (the down product's
// operand, quantised from the fp32 value), and the E4M3 codes of gu itself to gu_q + gu_scale (the
// checkpoint of the backward pass). f a multiple of 128, so no block spans gate and up.
template <typename Tin>
__global__ void __launch_bounds__(256, 4)
    swiglu_checkpoint_kernel(const Tin *__restrict__ gu, long long rows, int f,
                             const int32_t *__restrict__ n_rows, __nv_bfloat16 *__restrict__ h,
                             uint8_t *__restrict__ h_q, uint8_t *__restrict__ h_scale,
                             uint8_t *__restrict__ gu_q, uint8_t *__restrict__ gu_scale) {
  const KernelStamp stamp(K_F8B_SWIGLU);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const RowTeam w;
  FlatWalk at(w, f / QB, 2 * f);
  const long long total = valid_rows(rows, n_rows) * at.nb;
  for (long long b0 = w.first; b0 < total; b0 += w.step, at.next()) {
    const long long b = b0 + w.team, off = b * QB + w.c;  // in h
    const bool ok = b < total;
    Lane16<Tin> xg, xu;
    xg.zero();
    xu.zero();
    if (ok) {
      xg.load(gu + at.off);
      xu.load(gu + at.off + f);
    }
    uint32_t bg = 0, bu = 0;
    if (gu_q) {
      bg = block_byte(xg.amax());
      bu = block_byte(xu.amax());
      // the gate block's scale sits where the block does, in rows of 2 nb
      if (ok && w.c == 0) {
        gu_scale[at.off / QB] = (uint8_t)bg;
        gu_scale[at.off / QB + at.nb] = (uint8_t)bu;
      }
    }
    float hv[2][8];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float g[8], u[8];
      xg.p[x].values(g);
      xu.p[x].values(u);
      if (gu_q && ok) {
        store_codes(gu_q + at.off + 64 * x, g, e8m0_inverse(bg));
        store_codes(gu_q + at.off + f + 64 * x, u, e8m0_inverse(bu));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[x][i] = g[i] * sigmoid_f(g[i]) * u[i];
      if (h && ok) store_bf16x8(h + off + 64 * x, hv[x]);
    }
    if (h_q) {
      const uint32_t bh = block_byte(max(amax_bits(hv[0]), amax_bits(hv[1])));
      if (ok) {
        store_codes(h_q + off, hv[0], e8m0_inverse(bh));
        store_codes(h_q + off + 64, hv[1], e8m0_inverse(bh));
        if (w.c == 0) h_scale[b] = (uint8_t)bh;
      }
    }
  }
}

// A block's scale in two factors: a code times the first is finite, the second (1 for the bytes up to 239)
// is applied last. A gate of the larger bytes is 0 or past 2^104, and smaller by 2^9 it has the same
// sigmoid and slope (1/2, 0 or 1).
__device__ __forceinline__ float2 split_scale(uint32_t b) {
  const bool big = b >= 240;
  return make_float2(e8m0_value(big ? b - 9 : b), big ? 512.0f : 1.0f);
}
// From the checkpoint and dh: s = sigmoid(g), du = dh g s, dg = dh u s (1 + g (1 - s)), h = g s u.
// dgu = [dg | du] in bf16 and / or as E4M3 codes (the input gradient's operand, quantised from the
// fp32 values); h in bf16 (the down weight gradient's operand).
template <typename Tin>
__global__ void __launch_bounds__(256, 4)
    swiglu_checkpoint_backward_kernel(const uint8_t *__restrict__ gu_q,
                                      const uint8_t *__restrict__ gu_scale,
                                      const Tin *__restrict__ dh, long long rows, int f,
                                      const int32_t *__restrict__ n_rows,
                                      __nv_bfloat16 *__restrict__ dgu, uint8_t *__restrict__ dgu_q,
                                      uint8_t *__restrict__ dgu_scale, __nv_bfloat16 *__restrict__ h) {
  const KernelStamp stamp(K_F8B_SWIGLU);
  griddep_wait();
  stamp.started();
  griddep_launch();
  const RowTeam w;
  FlatWalk at(w, f / QB, 2 * f);
  const long long total = valid_rows(rows, n_rows) * at.nb;
  for (long long b0 = w.first; b0 < total; b0 += w.step, at.next()) {
    const long long b = b0 + w.team, off = b * QB + w.c;
    const bool ok = b < total;
    uint2 cg[2], cu[2];
    uint32_t sg = 127, su = 127;
    Lane16<Tin> xd;
    xd.zero();
    cg[0] = cg[1] = cu[0] = cu[1] = make_uint2(0u, 0u);
    if (ok) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        cg[x] = __ldg((const uint2 *)(gu_q + at.off + 64 * x));
        cu[x] = __ldg((const uint2 *)(gu_q + at.off + f + 64 * x));
      }
      xd.load(dh + off);
      sg = __ldg(gu_scale + at.off / QB);
      su = __ldg(gu_scale + at.off / QB + at.nb);
    }
    const float2 vg = split_scale(sg), vu = split_scale(su);
    float dg[2][8], du[2][8];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float d[8], hv[8];
      xd.p[x].values(d);
      const uint32_t wg[2] = {cg[x].x, cg[x].y}, wu[2] = {cu[x].x, cu[x].y};
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 g2 = e4m3x2_values((wg[i / 4] >> (8 * (i % 4))) & 0xffffu);
        const float2 u2 = e4m3x2_values((wu[i / 4] >> (8 * (i % 4))) & 0xffffu);
        const float gg[2] = {g2.x * vg.x, g2.y * vg.x}, uu[2] = {u2.x * vu.x, u2.y * vu.x};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float s = sigmoid_f(gg[j]), gs = gg[j] * s;
          du[x][i + j] = d[i + j] * gs * vg.y;
          // s (1 + g (1 - s)) = s + g s (1 - s), between -0.1 and 1.1, times up's part (448 2^118 at most)
          // first: dh times it could pass fp32's largest, or lose bits below its least normal number
          dg[x][i + j] = fmaf(gs, 1.0f - s, s) * uu[j] * d[i + j] * vu.y;
          hv[i + j] = gs * uu[j] * (vg.y * vu.y);
        }
      }
      if (ok && dgu) {
        store_bf16x8(dgu + at.off + 64 * x, dg[x]);
        store_bf16x8(dgu + at.off + f + 64 * x, du[x]);
      }
      if (ok && h) store_bf16x8(h + off + 64 * x, hv);
    }
    if (dgu_q) {
      const uint32_t bg = block_byte(max(amax_bits(dg[0]), amax_bits(dg[1])));
      const uint32_t bu = block_byte(max(amax_bits(du[0]), amax_bits(du[1])));
      if (ok) {
        const float ig = e8m0_inverse(bg), iu = e8m0_inverse(bu);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          store_codes(dgu_q + at.off + 64 * x, dg[x], ig);
          store_codes(dgu_q + at.off + f + 64 * x, du[x], iu);
        }
        if (w.c == 0) {
          dgu_scale[at.off / QB] = (uint8_t)bg;
          dgu_scale[at.off / QB + at.nb] = (uint8_t)bu;
        }
      }
    }
  }
}

}  // namespace moe
