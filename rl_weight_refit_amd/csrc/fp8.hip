// Block-FP8 kernels for gfx950 (CDNA4, wave64): quantisation with one
// float32 scale per block of 128, and the product of two matrices so scaled.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "matmul_shape.hpp"
#include "ops.hpp"
#include "ops_device.hpp"

namespace rs {
namespace {

// --------------------------------------------------------------------------
// Quantisation.  scale = amax / 448, code = E4M3(v * (1 / scale)).  The
// largest magnitude is found on the bit patterns (sign cleared), where every
// infinity and NaN is larger than every finite value.
// --------------------------------------------------------------------------

struct QuantArgs {
  const void* x;
  const int32_t* row_count;
  uint8_t* codes;
  float* scales;
  int64_t rows, cols, x_stride, x_batch, code_stride, code_batch, scale_stride, scale_batch;
  int64_t tiles_m, tiles_n;
  uint64_t magic;  // 2^64 / tiles_n, rounded up
};

// silu(gate) * up, by e = exp(-|gate|), which is at most 1: a gate below 0
// gives gate * e / (1 + e), so that a sigmoid below 2^-126 loses no more than a
// subnormal e does.  Of gate and gate * e the larger is the one meant (of
// infinities and NaN either marks the block).  The reciprocal instruction's 2^-23 is refined once, to
// half a step: with exp (2^-23), the addition and three products below 7 steps
// of 2^-24 in all.
__device__ __forceinline__ float gated(float gate, float up) {
  const float e = expf(-fabsf(gate)), d = 1.0f + e, r = __builtin_amdgcn_rcpf(d);
  return __builtin_amdgcn_fmed3f(gate, gate * e, INFINITY) * fmaf(fmaf(-d, r, 1.0f), r, r) * up;
}

__device__ __forceinline__ uint32_t amax_bits(const float v[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) a = max(a, __float_as_uint(v[k]) & 0x7FFFFFFFu);
  return a;
}

struct Scale {
  float scale, inv;
  bool bad;
};
__device__ __forceinline__ Scale scale_of(uint32_t amax) {
  Scale s;
  s.bad = amax >= 0x7F800000u;
  s.scale = __uint_as_float(amax) / 448.0f;
  const bool none = s.scale < 1.17549435e-38f;
  if (none) s.scale = 0.0f;
  s.inv = none ? 0.0f : 1.0f / s.scale;
  if (s.bad) s.scale = __uint_as_float(0x7FC00000u);
  return s;
}

__device__ __forceinline__ uint32_t code4(const Scale& s, float a, float b, float c, float d) {
  if (s.bad) return 0x7F7F7F7Fu;
  auto cut = [&](float v) { return __builtin_amdgcn_fmed3f(v * s.inv, -448.0f, 448.0f); };
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(cut(a), cut(b), 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(cut(c), cut(d), r, true);
  return uint32_t(r);
}

// n (0..8) code bytes of one lane.
__device__ __forceinline__ void store_codes(uint8_t* q, uint32_t lo, uint32_t hi, int n) {
  if (n == 8) {
    __builtin_nontemporal_store(uint64_t(hi) << 32 | lo, reinterpret_cast<ou64_1*>(q));
    return;
  }
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < n) q[k] = uint8_t((k < 4 ? lo : hi) >> (8 * (k & 3)));
}

// One scale per row and 128 columns: sixteen lanes a block, eight values a
// lane, and as many blocks a lane as make two 16-byte loads (8192 x 7168 bf16:
// one block a lane 40.8 us, two 38.9, four 40.6; float32: one 51.2, two 53.3).
// Blocks are numbered through the rows; the row of one is its number times
// 2^64 / (blocks a row), in the upper 64 bits.
template <int DTYPE, bool GATED>
constexpr int kQuantUnroll = DTYPE == RS_F32 || GATED ? 1 : 2;

template <int DTYPE, bool GATED>
__global__ __launch_bounds__(256) void rs_quant_rows_kernel(QuantArgs p) {
  constexpr int kUnroll = kQuantUnroll<DTYPE, GATED>;
  const int64_t batch = blockIdx.y;
  const int64_t rows = p.row_count ? min(p.rows, int64_t(*p.row_count)) : p.rows;
  const int lane = threadIdx.x & 15;
  const char* x = static_cast<const char*>(p.x) + batch * p.x_batch * dtype_size(DTYPE);
  Raw8<DTYPE> v[kUnroll], up[GATED ? kUnroll : 1];
  int64_t row[kUnroll], col[kUnroll];
  int n[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint64_t block = uint64_t(blockIdx.x) * (16 * kUnroll) + u * 16 + (threadIdx.x >> 4);
    row[u] = int64_t(p.tiles_n == 1 ? block : __umul64hi(block, p.magic));
    col[u] = int64_t(block - uint64_t(row[u]) * uint64_t(p.tiles_n)) * kBlock + lane * 8;
    n[u] = row[u] < rows ? int(max(int64_t(0), min(int64_t(8), p.cols - col[u]))) : 0;
    if (n[u] > 0) {
      v[u].load(x, row[u] * p.x_stride + col[u], n[u]);
      if (GATED) up[u].load(x, row[u] * p.x_stride + p.cols + col[u], n[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (row[u] >= rows) continue;  // sixteen lanes together
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = n[u] > 0 ? v[u].get(k) : 0.0f;
      if (GATED && n[u] > 0) f[k] = gated(f[k], up[u].get(k));
    }
    uint32_t a = amax_bits(f);
#pragma unroll
    for (int d = 8; d; d >>= 1) a = max(a, uint32_t(__shfl_xor(int(a), d, 16)));
    const Scale s = scale_of(a);
    store_codes(p.codes + batch * p.code_batch + row[u] * p.code_stride + col[u], code4(s, f[0], f[1], f[2], f[3]),
                code4(s, f[4], f[5], f[6], f[7]), n[u]);
    if (lane == 0) p.scales[batch * p.scale_batch + row[u] * p.scale_stride + col[u] / kBlock] = s.scale;
  }
}

template <int DTYPE, bool GATED>
void quant_rows(const QuantArgs& p, int64_t batch, hipStream_t stream) {
  constexpr int64_t kEach = 16 * kQuantUnroll<DTYPE, GATED>;
  const dim3 grid(uint32_t((p.rows * p.tiles_n + kEach - 1) / kEach), uint32_t(batch));
  rs_quant_rows_kernel<DTYPE, GATED><<<grid, 256, 0, stream>>>(p);
}

// The value of eight columns of a row as it lies in memory (gated values as
// float32); zeros behind the row's end and for absent rows.
template <int DTYPE, bool GATED>
struct Values8 : Raw8<GATED ? int(RS_F32) : DTYPE> {
  using Raw = Raw8<GATED ? int(RS_F32) : DTYPE>;
  __device__ __forceinline__ void load_row(const QuantArgs& p, const char* x, int64_t row, int64_t col, int n) {
    Raw::a = Raw::b = ou32x4{0, 0, 0, 0};
    if (n == 0) return;
    const int64_t at = row * p.x_stride + col;
    if constexpr (GATED) {
      Raw8<DTYPE> gate, up;
      gate.load(x, at, n);
      up.load(x, at + p.cols, n);
#pragma unroll
      for (int k = 0; k < 8; ++k) (k < 4 ? Raw::a : Raw::b)[k & 3] = __float_as_uint(gated(gate.get(k), up.get(k)));
    } else {
      Raw::load(x, at, n);
    }
  }
};

// One 128 x 128 tile of x per workgroup, held in registers as it lies in
// memory (eight rows and eight columns a lane; gated values as float32).
// COLUMN: a scale per column of the tile (a row of the transposed output),
// else one for the tile.  TRANSPOSE: the codes turn in LDS.
template <int DTYPE, bool GATED, bool COLUMN, bool TRANSPOSE>
__global__ __launch_bounds__(256) void rs_quant_tile_kernel(QuantArgs p) {
  constexpr int kPitch = 136;
  __shared__ uint32_t amax[COLUMN ? kBlock : 1];
  __shared__ __attribute__((aligned(8))) uint8_t turn[TRANSPOSE ? kBlock * kPitch : 16];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t tile_n = blockIdx.x % p.tiles_n, tile_m = blockIdx.x / p.tiles_n, batch = blockIdx.y;
  const int64_t row0 = tile_m * kBlock, col0 = tile_n * kBlock, col = col0 + tx * 8;
  const char* x = static_cast<const char*>(p.x) + batch * p.x_batch * dtype_size(DTYPE);
  uint8_t* codes = p.codes + batch * p.code_batch;
  float* scales = p.scales + batch * p.scale_batch;
  const int n = int(max(int64_t(0), min(int64_t(8), p.cols - col)));

  Values8<DTYPE, GATED> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + ty * 8 + i;
    v[i].load_row(p, x, row, col, row < p.rows ? n : 0);
  }
  for (int i = tid; i < (COLUMN ? kBlock : 1); i += 256) amax[i] = 0;
  __syncthreads();
  if (COLUMN) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i].get(k)) & 0x7FFFFFFFu);
      a = max(a, uint32_t(__shfl_xor(int(a), 16, 64)));  // the wave's four row groups
      a = max(a, uint32_t(__shfl_xor(int(a), 32, 64)));
      if ((tid & 48) == 0) atomicMax(&amax[COLUMN ? tx * 8 + k : 0], a);
    }
  } else {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) a = max(a, __float_as_uint(v[i].get(k)) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 32; d; d >>= 1) a = max(a, uint32_t(__shfl_xor(int(a), d, 64)));
    if ((tid & 63) == 0) atomicMax(&amax[0], a);
  }
  __syncthreads();
  if (TRANSPOSE) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Scale s = scale_of(amax[COLUMN ? tx * 8 + k : 0]);
      const uint64_t lo = code4(s, v[0].get(k), v[1].get(k), v[2].get(k), v[3].get(k));
      const uint64_t hi = code4(s, v[4].get(k), v[5].get(k), v[6].get(k), v[7].get(k));
      *reinterpret_cast<uint64_t*>(&turn[(tx * 8 + k) * kPitch + ty * 8]) = hi << 32 | lo;
    }
    __syncthreads();
    // output rows col0.., eight bytes a lane
    const int m = int(max(int64_t(0), min(int64_t(8), p.rows - row0 - tx * 8)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 16 + ty;
      if (col0 + c >= p.cols) continue;
      const uint64_t w = *reinterpret_cast<const uint64_t*>(&turn[c * kPitch + tx * 8]);
      store_codes(codes + (col0 + c) * p.code_stride + row0 + tx * 8, uint32_t(w), uint32_t(w >> 32), m);
    }
    if (COLUMN) {
      if (tid < kBlock && col0 + tid < p.cols)
        scales[(col0 + tid) * p.scale_stride + tile_m] = scale_of(amax[COLUMN ? tid : 0]).scale;
    } else if (tid == 0) {
      scales[tile_n * p.scale_stride + tile_m] = scale_of(amax[0]).scale;
    }
  } else {
    const Scale s = scale_of(amax[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + ty * 8 + i;
      if (row < p.rows)
        store_codes(codes + row * p.code_stride + col, code4(s, v[i].get(0), v[i].get(1), v[i].get(2), v[i].get(3)),
                    code4(s, v[i].get(4), v[i].get(5), v[i].get(6), v[i].get(7)), n);
    }
    if (tid == 0) scales[tile_m * p.scale_stride + tile_n] = s.scale;
  }
}

template <int DTYPE, bool GATED>
void quant_tiles(const QuantArgs& p, bool column, bool transpose, int64_t batch, hipStream_t stream) {
  const dim3 grid(uint32_t(p.tiles_m * p.tiles_n), uint32_t(batch));
  if (column) rs_quant_tile_kernel<DTYPE, GATED, true, true><<<grid, 256, 0, stream>>>(p);
  else if (transpose) rs_quant_tile_kernel<DTYPE, GATED, false, true><<<grid, 256, 0, stream>>>(p);
  else rs_quant_tile_kernel<DTYPE, GATED, false, false><<<grid, 256, 0, stream>>>(p);
}

// --------------------------------------------------------------------------
// Product.  One v_mfma_f32_16x16x128_f8f6f4 multiplies a 16 x 16 tile over
// exactly one scale block of 128, so its result times a_scale * b_scale is
// added to the float32 accumulators in the vector units.  b is the
// instruction's row operand: a lane then holds one row of c (lane % 16) and
// four neighbouring columns.  Both operands number the 128 products alike, so
// their order within the block is free: lane quarter q takes the 16-byte
// chunks q and q + 4 of a row.
// --------------------------------------------------------------------------

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct MatmulArgs {
  const uint8_t* a;
  const float* sa;
  const int32_t* index;
  const uint8_t* b;
  const float* sb;
  const int32_t* offsets;
  void* c;
  int64_t m, a_rows, lda, ldsa, ldb, ldsb, b_group, sb_group, ldc;
  int32_t n, k, n_groups, kblocks, n_tiles, split, split_blocks, out_dtype, b_rows;
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma128(const ou32x4 a0, const ou32x4 a1, const ou32x4 b0, const ou32x4 b1) {
  const i32x8 a = {int(a0[0]), int(a0[1]), int(a0[2]), int(a0[3]), int(a1[0]), int(a1[1]), int(a1[2]), int(a1[3])};
  const i32x8 b = {int(b0[0]), int(b0[1]), int(b0[2]), int(b0[3]), int(b1[0]), int(b1[1]), int(b1[2]), int(b1[3])};
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// The same product with exact terms: the FP8 matrix path lines eight
// neighbouring products up with the largest and cuts them 13 bits below it
// (measured; 1.4e-5 of the rms result on normal values, 5e-5 with a column in 128
// a hundred times the others).  That is taken for a bf16 c, whose own rounding
// is 2^-8, and not for f16 or float32: the bfloat16 path sums products of E4M3
// values to 1e-8, at half the rate.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
struct Wide {
  bf16x8 v[4];
};
__device__ __forceinline__ Wide widen(const ou32x4 lo, const ou32x4 hi) {
  return Wide{{widen(lo[0], lo[1]), widen(lo[2], lo[3]), widen(hi[0], hi[1]), widen(hi[2], hi[3])}};
}
__device__ __forceinline__ f32x4 mfma128_exact(const Wide& a, const Wide& b) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[s], b.v[s], d, 0, 0, 0);
  return d;
}

// The groups' row tiles (of tile_m rows), sixty-four groups at a time, a group
// a lane; every wave finds its tile for itself.
struct GroupTiles {
  int64_t lo, hi;  // this lane's group's rows
  int count, sum;  // its tiles, and those up to it among the sixty-four
};
__device__ __forceinline__ GroupTiles group_tiles(const MatmulArgs& p, int g0, int tile_m) {
  const int lane = threadIdx.x & 63, g = g0 + lane;
  GroupTiles t{0, 0, 0, 0};
  if (p.n_groups == 0) return t;
  if (g < p.n_groups) {
    t.lo = max(int64_t(0), min(p.m, int64_t(p.offsets[g])));
    t.hi = max(t.lo, min(p.m, int64_t(p.offsets[g + 1])));
  }
  t.count = t.sum = int((t.hi - t.lo + tile_m - 1) / tile_m);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(t.sum, d, 64);
    if (lane >= d) t.sum += o;
  }
  return t;
}

// All row tiles, of which `first` are the first sixty-four groups'.  (Offsets
// that descend could name a row twice; the launch has `most` tiles' workgroups
// at the most.)
__device__ __forceinline__ int count_tiles(const MatmulArgs& p, const GroupTiles& first, int tile_m, int most) {
  if (p.n_groups == 0) return most;
  int total = __shfl(first.sum, 63, 64);
  for (int g0 = 64; g0 < p.n_groups; g0 += 64) total += __shfl(group_tiles(p, g0, tile_m).sum, 63, 64);
  return min(total, most);
}

// Rows [begin, end) of c and the group of row tile `tile`.  False: there is no
// such tile (or the sums of offsets that descend passed 32 bits).
__device__ __forceinline__ bool find_tile(const MatmulArgs& p, const GroupTiles& first, int tile, int tile_m, int* group,
                                          int64_t* begin, int64_t* end) {
  if (p.n_groups == 0) {
    *group = 0;
    *begin = int64_t(tile) * tile_m;
    *end = min(p.m, *begin + tile_m);
    return *begin < p.m;
  }
  GroupTiles t = first;
  int seen = 0;
  for (int g0 = 0;;) {
    const uint64_t past = __ballot(seen + t.sum > tile);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      const int before = seen + __shfl(t.sum, at, 64) - __shfl(t.count, at, 64);
      const int64_t from = __shfl(int(t.lo), at, 64), to = __shfl(int(t.hi), at, 64);
      *group = g0 + at;
      *begin = from + int64_t(tile - before) * tile_m;
      *end = min(to, *begin + tile_m);
      return *begin >= from && *begin < to;
    }
    seen += __shfl(t.sum, 63, 64);
    g0 += 64;
    if (g0 >= p.n_groups) return false;
    t = group_tiles(p, g0, tile_m);
  }
}

// Row of b's scales for row n of b.
__device__ __forceinline__ int b_block(const MatmulArgs& p, int n) {
  if (p.b_rows == 1) return n;
  return n < p.split ? n >> 7 : p.split_blocks + ((n - p.split) >> 7);
}

// Sixteen bytes of a row at column k; bytes from column `limit` on are zero.
__device__ __forceinline__ ou32x4 chunk16(const uint8_t* row, int k, int limit) {
  ou32x4 v = {0, 0, 0, 0};
  if (k >= limit) return v;
  v = *reinterpret_cast<const ou32x4*>(row + k);
  const int left = limit - k;
  if (left < 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bytes = left - 4 * i;
      v[i] = bytes <= 0 ? 0 : bytes >= 4 ? v[i] : v[i] & ((1u << (8 * bytes)) - 1);
    }
  }
  return v;
}

// --- few rows --------------------------------------------------------------
//
// MT x 16 rows of c by NT x 16 columns per workgroup, whose W waves share
// out the scale blocks of k (wave w takes blocks w, w + W, ...) and add their
// sums at the end, in the order of the waves.  b is read once, straight into
// the registers of the one wave that multiplies it, so there is no LDS
// staging and no barrier before the end: with few rows the time is that of
// reading b, and many waves with several blocks each in flight hide it.
//
// EACH: the scales of b are looked up row by row, since a tile's 16 rows need
// not share one.

template <int MT, int NT, int U, int W, bool EACH, bool EXACT>
__global__ __launch_bounds__(W * 64) void rs_matmul_stream_kernel(MatmulArgs p) {
  __shared__ f32x4 part[W][MT * NT * 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = int(blockIdx.x % p.n_tiles) * NT * 16;
  int g;
  int64_t begin, end;
  if (!find_tile(p, group_tiles(p, 0, MT * 16), int(blockIdx.x / p.n_tiles), MT * 16, &g, &begin, &end)) return;
  const uint8_t* b = p.b + g * p.b_group;
  const float* sb = p.sb + g * p.sb_group;

  // Rows behind the tile's last are read from the last, gathered rows outside
  // a from row 0, columns behind c's last from the last; none is stored.
  const uint8_t *arow[MT], *brow[NT];
  const float *sarow[MT], *sbrow[NT][EACH ? 4 : 1];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t r = min(begin + i * 16 + (lane & 15), end - 1);
    if (p.index) r = p.index[r];
    if (r < 0 || r >= p.a_rows) r = 0;
    arow[i] = p.a + r * p.lda;
    sarow[i] = p.sa + r * p.ldsa;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    brow[j] = b + int64_t(min(n0 + j * 16 + (lane & 15), p.n - 1)) * p.ldb;
#pragma unroll
    for (int q = 0; q < (EACH ? 4 : 1); ++q)
      sbrow[j][q] = sb + int64_t(b_block(p, min(n0 + j * 16 + (EACH ? (lane >> 4) * 4 + q : 0), p.n - 1))) * p.ldsb;
  }
  f32x4 acc[MT][NT] = {};
  const int whole = p.k / kBlock, kblocks = p.a_rows > 0 ? p.kblocks : 0;
  const int at0 = (lane >> 4) * 16, at1 = at0 + 64;
  for (int k0 = wave; k0 < kblocks; k0 += W * U) {
    ou32x4 fa[U][MT][2], fb[U][NT][2];
    float pa[U][MT], pb[U][NT][EACH ? 4 : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * W;
      if (kb >= kblocks) continue;
      const int k = kb * kBlock;
      if (kb < whole) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          fb[u][j][0] = *reinterpret_cast<const ou32x4*>(brow[j] + k + at0);
          fb[u][j][1] = *reinterpret_cast<const ou32x4*>(brow[j] + k + at1);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          fa[u][i][0] = *reinterpret_cast<const ou32x4*>(arow[i] + k + at0);
          fa[u][i][1] = *reinterpret_cast<const ou32x4*>(arow[i] + k + at1);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) fb[u][j][0] = chunk16(brow[j], k + at0, p.k), fb[u][j][1] = chunk16(brow[j], k + at1, p.k);
#pragma unroll
        for (int i = 0; i < MT; ++i) fa[u][i][0] = chunk16(arow[i], k + at0, p.k), fa[u][i][1] = chunk16(arow[i], k + at1, p.k);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) pa[u][i] = sarow[i][kb];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < (EACH ? 4 : 1); ++q) pb[u][j][q] = sbrow[j][q][kb];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * W >= kblocks) continue;
      Wide wa[MT];
      if (EXACT) {
#pragma unroll
        for (int i = 0; i < MT; ++i) wa[i] = widen(fa[u][i][0], fa[u][i][1]);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Wide wb;
        if (EXACT) wb = widen(fb[u][j][0], fb[u][j][1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const f32x4 d = EXACT ? mfma128_exact(wb, wa[i]) : mfma128(fb[u][j][0], fb[u][j][1], fa[u][i][0], fa[u][i][1]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] += pa[u][i] * pb[u][j][EACH ? q : 0] * d[q];
        }
      }
    }
  }
  // a lane's four columns of tile (i, j) lie at [i][row lane % 16][j][lane / 16]
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][((i * 16 + (lane & 15)) * NT + j) * 4 + (lane >> 4)] = acc[i][j];
  __syncthreads();
  for (int e = tid; e < MT * NT * 64; e += W * 64) {
    f32x4 v = part[0][e];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const f32x4 o = part[w][e];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += o[q];
    }
    const int64_t row = begin + e / (NT * 4);
    const int n = n0 + (e % (NT * 4)) * 4;
    if (row >= end) continue;
    if (p.index) {
      const int64_t from = p.index[row];
      if (from < 0 || from >= p.a_rows) v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < p.n) store1(p.c, p.out_dtype, row * p.ldc + n + q, v[q]);
  }
}

// Four values of c in 16 bits: bf16, or f16 where the sums are exact.
template <bool F16>
__device__ __forceinline__ uint64_t pack4(f32x4 v) {
  uint64_t w = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) w |= uint64_t(F16 ? float_f16(v[q]) : float_bf16(v[q])) << (16 * q);
  return w;
}

// --- large tiles -----------------------------------------------------------
//
// BM x BN values of c per workgroup of eight waves: WM of them along the rows,
// KG along k, the others along the columns.  A wave's columns lie within one
// 128-row block of b, so that one b scale serves it per k block (EACH: one
// each).  Blocks of both operands go from memory straight into S stages of
// LDS, the loads of later blocks under way while one is multiplied.
//
// A stage holds a block's rows of 128 bytes, 16-byte chunk c of row r in place
// c ^ (r % 8): a load puts a wave's chunks down in the order of its lanes, so
// each lane fetches the chunk that belongs in its place, and the sixteen rows
// that a quarter wave reads one chunk of lie in all banks (8192 x 8192 x 8192:
// 1.6e6 conflict cycles, 4.6e7 in the plain order).
//
// 8192 x 8192 x 8192: 490 us, 2,240 TFLOP/s (f16 or float32 c, by the bfloat16
// path: 880 to 890 us).  A copy of the kernel without its loads takes 437 us, one that
// does not scale either 344 to 360: matrix instructions with the LDS reads that
// feed them bound it, scaling (four vector FMAs a matrix instruction) and
// loads each add what the schedule does not hide.  256 x 256 tiles read least
// from LDS and L2 for a product; 128 x 256 take 600 us, 64 x 256 798, 64 x 128
// 809, 64 x 64 1,547: those are for shapes with too few tiles to fill the chip.

typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return uint32_t(uintptr_t((const lds_u8*)p));
}

// Sixteen (four) bytes per lane from base + off straight into LDS at `to` +
// 16 (4) * lane, if kb < end.  The compiler does not see these loads: what
// waits for them is wait_loads().  (It sets m0 itself right where it needs
// it, so nothing of its own is lost there.)  Nor does it see the branch: a visible
// one in the middle of the main loop costs it the registers that the loop
// needs (21 to 135 spilled).
__device__ __forceinline__ void load_lds16(uint32_t to, const void* base, uint32_t off, int kb, int end) {
  asm volatile(
      "s_cmp_ge_i32 %3, %4\n\t"
      "s_cbranch_scc1 .Lskip%=\n\t"
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2\n"
      ".Lskip%=:" ::"s"(to), "v"(off), "s"(base), "s"(kb), "s"(end)
      : "memory", "scc");
}
__device__ __forceinline__ void load_lds4(uint32_t to, const void* base, uint32_t off, int kb, int end) {
  asm volatile(
      "s_cmp_ge_i32 %3, %4\n\t"
      "s_cbranch_scc1 .Lskip%=\n\t"
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2\n"
      ".Lskip%=:" ::"s"(to), "v"(off), "s"(base), "s"(kb), "s"(end)
      : "memory", "scc");
}
// The same from addresses that a 32-bit offset does not reach.
__device__ __forceinline__ void load_lds16(uint32_t to, const void* base, uint64_t off, int kb, int end) {
  asm volatile(
      "s_cmp_ge_i32 %2, %3\n\t"
      "s_cbranch_scc1 .Lskip%=\n\t"
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off\n"
      ".Lskip%=:" ::"s"(to), "v"(reinterpret_cast<uint64_t>(base) + off), "s"(kb), "s"(end)
      : "memory", "scc");
}
__device__ __forceinline__ void load_lds4(uint32_t to, const void* base, uint64_t off, int kb, int end) {
  asm volatile(
      "s_cmp_ge_i32 %2, %3\n\t"
      "s_cbranch_scc1 .Lskip%=\n\t"
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, off\n"
      ".Lskip%=:" ::"s"(to), "v"(reinterpret_cast<uint64_t>(base) + off), "s"(kb), "s"(end)
      : "memory", "scc");
}
// Waits until at most N of this wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The same for 0, 2, 8 or 9, without a branch that the compiler sees.
__device__ __forceinline__ void wait_loads_at_most(int n) {
  asm volatile(
      "s_cmp_lt_i32 %0, 9\n\t"
      "s_cbranch_scc0 .Lnine%=\n\t"
      "s_cmp_lt_i32 %0, 8\n\t"
      "s_cbranch_scc0 .Leight%=\n\t"
      "s_cmp_lt_i32 %0, 2\n\t"
      "s_cbranch_scc0 .Ltwo%=\n\t"
      "s_waitcnt vmcnt(0)\n\t"
      "s_branch .Ldone%=\n"
      ".Lnine%=:\n\t"
      "s_waitcnt vmcnt(9)\n\t"
      "s_branch .Ldone%=\n"
      ".Leight%=:\n\t"
      "s_waitcnt vmcnt(8)\n\t"
      "s_branch .Ldone%=\n"
      ".Ltwo%=:\n\t"
      "s_waitcnt vmcnt(2)\n"
      ".Ldone%=:" ::"s"(n)
      : "memory", "scc");
}

// All waves' LDS reads and writes so far are done.  (__syncthreads() would
// also wait for the loads that are to stay under way.)
__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Workgroup -> tile: each XCD (blockIdx modulo 8) takes a contiguous range,
// in bands of four row tiles walked column tile by column tile, so the tiles
// running on one XCD share rows of a and b in its L2.  The ranges divide the
// tiles that there are: with groups the launch may have more workgroups, and
// those are left over on every XCD alike.
__device__ __forceinline__ bool tile_of(uint32_t id, uint32_t row_tiles, uint32_t n_tiles, uint32_t* mt, uint32_t* nt) {
  constexpr uint32_t kXcds = 8, kBand = 4;
  const uint32_t total = row_tiles * n_tiles, x = id % kXcds, each = total / kXcds, more = total % kXcds;
  if (id / kXcds >= each + (x < more)) return false;
  id = x * each + min(x, more) + id / kXcds;
  const uint32_t band = id / (kBand * n_tiles), in = id % (kBand * n_tiles);
  const uint32_t rows = min(kBand, row_tiles - band * kBand);
  *mt = band * kBand + in % rows;
  *nt = in / rows;
  return true;
}

// FAR: load offsets of 64 bits.
template <int BM, int BN, int WM, int S, int KG, bool EACH, bool EXACT, bool FAR = false>
struct Tile {
  using Offset = std::conditional_t<FAR, uint64_t, uint32_t>;
  // Two stages: the two waves of a SIMD (w and w + 4) take turns at reading
  // LDS and multiplying; see the loops.
  static constexpr bool kTurns = S == 2 && KG == 1 && !EXACT;
  static constexpr int kStage = (BM + BN) * 128, kScales = (BM + BN) * 4, kScaleStages = kTurns ? 3 : S * KG;
  static constexpr int kLds = S * KG * kStage + kScaleStages * kScales;
  static __device__ __forceinline__ void run(const MatmulArgs& p, uint8_t* lds, uint8_t* absent, int g, int64_t begin,
                                             int64_t end, int n0);
};

// Rows [begin, end) of group g, columns from n0.  absent[r]: gathered row r lies
// outside a.
template <int BM, int BN, int WM, int S, int KG, bool EACH, bool EXACT, bool FAR>
__device__ __forceinline__ void Tile<BM, BN, WM, S, KG, EACH, EXACT, FAR>::run(const MatmulArgs& p, uint8_t* lds,
                                                                               uint8_t* absent, int g, int64_t begin,
                                                                               int64_t end, int n0) {
  constexpr int WN = 8 / WM / KG, MT = BM / WM / 16, NT = BN / WN / 16;   // 16 x 16 tiles per wave: MT x NT
  constexpr int LA = BM / 64, LB = BN / 64;                          // 16-byte loads per lane and stage
  static_assert(!kTurns || (WN * 128 == BN && NT == 8), "a wave's first four column tiles lie in b's even pieces");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint8_t* abase = p.index ? p.a : p.a + begin * p.lda;
  const uint8_t* bbase = p.b + g * p.b_group + int64_t(n0) * p.ldb;
  const float* sabase = p.index ? p.sa : p.sa + begin * p.ldsa;
  const float* sbbase = p.sb + g * p.sb_group;

  // This lane's share of the loads.  Rows behind the tile's last are read
  // from the last, gathered rows outside a from row 0; neither is stored.
  const auto a_row = [&](int r) {
    const int64_t i = min(begin + r, end - 1);
    if (!p.index) return Offset(i - begin);
    const int64_t at = p.index[i];
    return Offset(at >= 0 && at < p.a_rows ? at : 0);
  };
  if (p.index && tid < BM) {
    const int64_t at = p.index[min(begin + tid, end - 1)];
    absent[tid] = at < 0 || at >= p.a_rows;
  }
  const int chunk = (lane & 7) ^ (lane >> 3);
  Offset aoff[LA], boff[LB], soff = 0;
#pragma unroll
  for (int i = 0; i < LA; ++i) aoff[i] = a_row(i * 64 + wave * 8 + (lane >> 3)) * Offset(p.lda) + chunk * 16;
#pragma unroll
  for (int i = 0; i < LB; ++i) boff[i] = Offset(min(i * 64 + wave * 8 + (lane >> 3), p.n - 1 - n0)) * Offset(p.ldb) + chunk * 16;
  const bool sa_wave = wave < LA, sb_wave = wave >= 4 && wave < 4 + (EACH ? LB : 1);
  static_assert(LA <= 4 && LB <= 4, "one wave's load per 64 scales");
  const int scale_end = __builtin_amdgcn_readfirstlane(sa_wave || sb_wave ? INT32_MAX : 0);
  if (sa_wave) soff = a_row(wave * 64 + lane) * Offset(p.ldsa) * 4;
  else if (sb_wave) soff = Offset(b_block(p, min(n0 + (EACH ? (wave - 4) * 64 + lane : (lane & 1) * 128), p.n - 1))) * Offset(p.ldsb) * 4;

  const uint32_t lds0 = lds_address(lds);
  // The loads of block kb < to_kb, in two parts: a, b's even 64-row pieces and
  // the scales, then b's odd pieces.  Chunks beyond k are read from the
  // block's first instead.
  const auto issue = [&](int kb, int stage, int scale_stage, bool first, bool second, int to_kb) {
    const uint32_t to = lds0 + stage * kStage + wave * 1024;
    const uint32_t cut = kb * 128 + chunk * 16 < p.k ? 0 : chunk * 16;
    const uint8_t *ak = abase + kb * 128, *bk = bbase + kb * 128;
#pragma unroll
    for (int i = 0; i < LA; ++i)
      if (first) load_lds16(to + i * 8192, ak, aoff[i] - cut, kb, to_kb);
#pragma unroll
    for (int i = 0; i < LB; ++i)
      if (i % 2 ? second : first) load_lds16(to + BM * 128 + i * 8192, bk, boff[i] - cut, kb, to_kb);
    if (!first) return;
    const uint32_t sto = lds0 + S * KG * kStage + scale_stage * kScales;
    const uint32_t sat = sa_wave ? wave * 256 : BM * 4 + (wave - 4) * 256;
    load_lds4(sto + sat, (sa_wave ? sabase : sbbase) + kb, soff, kb, min(to_kb, scale_end));
  };

  const int wm = (wave % WM) * (BM / WM), wn = (wave / WM % WN) * (BN / WN), kg = wave / (WM * WN);
  const int key = lane & 7, c0 = ((lane >> 4) ^ key) * 16, c1 = c0 ^ 64;
  const int arow = (wm + (lane & 15)) * 128, brow = BM * 128 + (wn + (lane & 15)) * 128;
  f32x4 acc[MT][NT] = {};

  const uint8_t* here = lds;    // the stage and scales read from
  const float* scales = nullptr;
  const auto read_from = [&](int stage, int scale_stage) {
    here = lds + stage * kStage;
    scales = reinterpret_cast<const float*>(lds + S * KG * kStage + scale_stage * kScales);
  };
  float pa[MT];
  constexpr int kRing = kTurns ? NT / 2 : 3;  // column tiles of b in registers
  ou32x4 fa[MT][2], fb[kRing][2];
  f32x4 d[2][MT], pb[2];
  const auto read_b = [&](int j) {
    fb[j % kRing][0] = *reinterpret_cast<const ou32x4*>(here + brow + j * 2048 + c0);
    fb[j % kRing][1] = *reinterpret_cast<const ou32x4*>(here + brow + j * 2048 + c1);
  };
  const auto read_a = [&] {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      fa[i][0] = *reinterpret_cast<const ou32x4*>(here + arow + i * 2048 + c0);
      fa[i][1] = *reinterpret_cast<const ou32x4*>(here + arow + i * 2048 + c1);
    }
    const float sb = EACH ? 1.0f : scales[BM + (wn >> 7)];
#pragma unroll
    for (int i = 0; i < MT; ++i) pa[i] = scales[wm + i * 16 + (lane & 15)] * sb;
  };
  const auto read_pb = [&](int j) {
    pb[j & 1] = *reinterpret_cast<const f32x4*>(scales + BM + wn + j * 16 + (lane >> 4) * 4);
  };
  // Column tiles from..to - 1, of which `upto` are there to be read.  Tile j
  // multiplies while the sums of tile j - 1 are scaled and added: the vector
  // units work on results that are there already.
  const auto multiply = [&](auto from, auto to, auto upto) {
    if constexpr (EXACT) {
      Wide wa[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) wa[i] = widen(fa[i][0], fa[i][1]);
#pragma unroll
      for (int j = from; j < to; ++j) {
        if (j + 2 < upto) read_b(j + 2);
        if (EACH) pb[0] = *reinterpret_cast<const f32x4*>(scales + BM + wn + j * 16 + (lane >> 4) * 4);
        const Wide wb = widen(fb[j % kRing][0], fb[j % kRing][1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const f32x4 e = mfma128_exact(wb, wa[i]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] += (EACH ? pa[i] * pb[0][q] : pa[i]) * e[q];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int j = from; j < to + (to == NT); ++j) {
        if (j + 2 < upto) read_b(j + 2);
        if (EACH && !kTurns && j < NT) read_pb(j);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if (j < NT) d[j & 1][i] = mfma128(fb[j % kRing][0], fb[j % kRing][1], fa[i][0], fa[i][1]);
          if (j > 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              acc[i][j - 1][q] += (EACH ? pa[i] * pb[(j - 1) & 1][q] : pa[i]) * d[(j - 1) & 1][i][q];
          }
        }
        if (EACH && kTurns && j + 1 < NT) read_pb(j + 1);
        if (j > 0 && j < NT) {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);              // one matrix instruction,
            __builtin_amdgcn_sched_group_barrier(0x002, EACH ? 8 : 4, 0);   // one tile's scaling
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  constexpr std::integral_constant<int, 0> kFirst;
  constexpr std::integral_constant<int, NT / 2> kHalf;
  constexpr std::integral_constant<int, NT> kAll;
  const int whole = p.k / kBlock;

  if constexpr (kTurns) {
    // A block goes in four phases with a barrier before each: read a and half
    // of b, multiply, read the other half, multiply.  Waves 4..7 are one phase
    // behind waves 0..3, so that on every SIMD one wave multiplies while the
    // other reads.  Block m is in stage m % 2.  Its first part (a, b's even
    // pieces) is read in phases 4 m and 4 m + 1 (waves 4..7), its second in
    // 4 m + 2 and 4 m + 3; so in either wave's second reading the first part
    // of block m + 2 may follow into its stage, and in the first reading of
    // block m + 1 the second part.  Each has five phases to arrive.  (Scales
    // are read until phase 4 m + 4: three stages.)  A wave that multiplies comes
    // before one that reads where each row of b has its own scale (8192 x 8192 x
    // 8192: 570 us, 585 without); otherwise it makes no difference.
    const int late = wave >> 2;
    const int first_loads = LA + LB / 2 + (scale_end ? 1 : 0), second_loads = LB / 2;
    const auto phase = [&] {
      __builtin_amdgcn_sched_barrier(0);
      barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    issue(0, 0, 0, true, false, p.kblocks);
    issue(0, 0, 0, false, true, p.kblocks);
    issue(1, 1, 1, true, false, p.kblocks);
    wait_loads_at_most(p.kblocks > 1 ? second_loads + first_loads : second_loads);
    if (late) barrier();
    for (int m = 0, s3 = 0; m < whole; ++m) {
      const int stage = m & 1, next3 = s3 == 2 ? 0 : s3 + 1, after3 = next3 == 2 ? 0 : next3 + 1;
      phase();
      read_from(stage, s3);
      read_a();
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) read_b(j);
      if (EACH) read_pb(0);
      issue(m + 1, stage ^ 1, next3, false, true, p.kblocks);
      wait_loads_at_most(m + 1 < p.kblocks ? first_loads + second_loads : 0);  // block m's second part is there
      phase();
      if (EACH) __builtin_amdgcn_s_setprio(1);
      multiply(kFirst, kHalf, kFirst);
      if (EACH) __builtin_amdgcn_s_setprio(0);
      phase();
#pragma unroll
      for (int j = NT / 2; j < NT; ++j) read_b(j);
      issue(m + 2, stage, after3, true, false, p.kblocks);
      // block m + 1's first part is there
      wait_loads_at_most(m + 2 < p.kblocks ? second_loads + first_loads : m + 1 < p.kblocks ? second_loads : 0);
      phase();
      if (EACH) __builtin_amdgcn_s_setprio(1);
      multiply(kHalf, kAll, kFirst);
      if (EACH) __builtin_amdgcn_s_setprio(0);
      s3 = next3;
    }
    if (!late) barrier();
  } else {
    // KG blocks go at a time, one for each group of 8 / KG waves, whose sums
    // are added at the end.  Step t is in stage t % S; the loads of the S - 2
    // steps after the one that is read may stay under way.
    const auto issue_step = [&](int t, int stage) {
#pragma unroll
      for (int u = 0; u < KG; ++u) issue(t * KG + u, stage * KG + u, stage * KG + u, true, true, p.kblocks);
    };
    const int steps = (whole + KG - 1) / KG;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue_step(i, i);
    for (int t = 0, stage = 0; t < steps; ++t, stage = stage + 1 == S ? 0 : stage + 1) {
      if (S > 2 && (t + S - 1) * KG <= whole) {
        if (scale_end) wait_loads<(S - 2) * KG * (LA + LB + 1)>();
        else wait_loads<(S - 2) * KG * (LA + LB)>();
      } else {
        wait_loads<0>();
      }
      barrier();
      read_from(stage * KG + kg, stage * KG + kg);
      read_b(0);
      read_a();
      read_b(1);
      const int next = stage == 0 ? S - 1 : stage - 1;  // the stage read last, free behind the barrier
      issue_step(t + S - 1, next);
      if (KG == 1 || t * KG + kg < whole) multiply(kFirst, kAll, kAll);
    }
  }
  if (p.k % kBlock) {
    // The columns behind the last whole block were loaded like a block of
    // their own; what lies behind k is made zero in LDS.
    constexpr int kSlots = S * KG;
    const int slot = whole % kSlots;
    wait_loads<0>();
    barrier();
    const int tail = p.k % kBlock;
    for (int e = tid; e < (BM + BN) * 8; e += 512) {
      const int r = e >> 3, c = e & 7, left = tail - c * 16;
      if (left >= 16) continue;
      ou32x4* at = reinterpret_cast<ou32x4*>(lds + slot * kStage + r * 128 + (c ^ (r & 7)) * 16);
      ou32x4 v = {0, 0, 0, 0};
      if (left > 0) {
        v = *at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int bytes = left - 4 * i;
          v[i] = bytes <= 0 ? 0 : bytes >= 4 ? v[i] : v[i] & ((1u << (8 * bytes)) - 1);
        }
      }
      *at = v;
    }
    barrier();
    read_from(slot, whole % kScaleStages);
    read_a();
    if constexpr (kTurns) {
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) read_b(j);
      if (EACH) read_pb(0);
      multiply(kFirst, kHalf, kFirst);
#pragma unroll
      for (int j = NT / 2; j < NT; ++j) read_b(j);
      multiply(kHalf, kAll, kFirst);
    } else {
      read_b(0);
      read_b(1);
      if (KG == 1 || kg == 0) multiply(kFirst, kAll, kAll);
    }
  }
  if constexpr (KG > 1) {  // the groups' sums to the first one's, in the order of the groups
    barrier();
    f32x4* parts = reinterpret_cast<f32x4*>(lds);
    const auto part = [&](int group, int i, int j) -> f32x4& {
      return parts[(((group * WM * WN + wave % (WM * WN)) * MT + i) * NT + j) * 64 + lane];
    };
    static_assert(KG * BM * BN * 4 <= S * KG * kStage, "the groups' sums fit the stages");
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part(kg, i, j) = acc[i][j];
    }
    barrier();
    if (kg > 0) return;
#pragma unroll
    for (int u = 1; u < KG; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const f32x4 v = part(u, i, j);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] += v[q];
        }
  }

  // Sixteen rows at a time through this wave's part of LDS, so that the
  // wave's columns of a row are stored at once.  (Groups behind the first
  // have ended, and the sums read above are not touched: turn lies in group
  // 0's place.)
  if (KG == 1) barrier();
  const auto store = [&](auto size) {
    constexpr int kSize = size, kPitch = NT * 16 * kSize + 16;
    uint8_t* turn = lds + wave * 16 * kPitch;
    static_assert(KG == 1 || WM * WN * 16 * kPitch <= BM * BN * 4, "turn stays clear of the groups' sums");
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 v = acc[i][j];
        uint8_t* at = turn + (lane & 15) * kPitch + (j * 16 + (lane >> 4) * 4) * kSize;
        if (kSize == 4) *reinterpret_cast<f32x4*>(at) = v;
        else *reinterpret_cast<uint64_t*>(at) = pack4<EXACT>(v);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      constexpr int kVec = 16 / kSize, kLanes = NT * 16 / kVec;  // values a store, lanes a row
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += 64 / kLanes) {
        const int r = r0 + lane / kLanes, col = (lane % kLanes) * kVec, n = n0 + wn + col;
        const int64_t row = begin + wm + i * 16 + r;
        ou32x4 v = *reinterpret_cast<const ou32x4*>(turn + r * kPitch + col * kSize);
        if (row >= end) continue;
        if (p.index && absent[wm + i * 16 + r]) v = ou32x4{0, 0, 0, 0};
        uint8_t* to = static_cast<uint8_t*>(p.c) + (row * p.ldc + n) * kSize;
        if (n + kVec <= p.n) {
          *reinterpret_cast<ou32x4_2*>(to) = v;
        } else {
#pragma unroll
          for (int q = 0; q < kVec; ++q) {
            if (n + q >= p.n) break;
            if (kSize == 4) reinterpret_cast<uint32_t*>(to)[q] = v[q];
            else reinterpret_cast<uint16_t*>(to)[q] = uint16_t(v[q / 2] >> (16 * (q & 1)));
          }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  };
  if (!EXACT || p.out_dtype == RS_F16) store(std::integral_constant<int, 2>());
  else store(std::integral_constant<int, 4>());
}

// A group's last tile has half its rows or fewer in half of the cases: then it
// goes as one of half the height, which takes two thirds of the time.
template <int BM, int BN, int WM, int S, int KG, bool EACH, bool EXACT, bool FAR>
__global__ __launch_bounds__(512, BM * BN > 128 * 128 || KG > 1 || FAR ? 2 : 4) void rs_matmul_tile_kernel(MatmulArgs p, uint32_t row_tiles) {
  using Whole = Tile<BM, BN, WM, S, KG, EACH, EXACT, FAR>;
  using Half = Tile<128, 256, 2, 3, 1, EACH, EXACT>;
  constexpr bool kHalves = BM == 256;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kHalves && Half::kLds > Whole::kLds ? Half::kLds : Whole::kLds];
  __shared__ uint8_t absent[BM];
  uint32_t mt, nt;
  const GroupTiles tiles = group_tiles(p, 0, BM);
  row_tiles = __builtin_amdgcn_readfirstlane(count_tiles(p, tiles, BM, int(row_tiles)));
  if (!tile_of(blockIdx.x, row_tiles, p.n_tiles, &mt, &nt)) return;
  int g;
  int64_t begin, end;
  if (!find_tile(p, tiles, int(mt), BM, &g, &begin, &end)) return;
  g = __builtin_amdgcn_readfirstlane(g);
  begin = __builtin_amdgcn_readfirstlane(int(begin));
  end = __builtin_amdgcn_readfirstlane(int(end));
  if constexpr (kHalves) {
    if (end - begin <= 128) return Half::run(p, lds, absent, g, begin, end, int(nt) * BN);
  }
  Whole::run(p, lds, absent, g, begin, end, int(nt) * BN);
}

// A launch holds fewer than 2^32 threads.
inline bool too_many(int64_t workgroups, int64_t threads) { return workgroups * threads > int64_t(UINT32_MAX); }

template <int BM, int BN, int WM, int S, int KG, bool FAR = false>
hipError_t launch_tile(MatmulArgs p, bool each, bool exact, int64_t row_tiles, hipStream_t stream) {
  p.n_tiles = (p.n + BN - 1) / BN;
  if (too_many(row_tiles * p.n_tiles, 512)) return hipErrorInvalidConfiguration;
  const uint32_t tiles = uint32_t(row_tiles);
  const dim3 grid(tiles * p.n_tiles);
  if (each && exact) rs_matmul_tile_kernel<BM, BN, WM, S, KG, true, true, FAR><<<grid, 512, 0, stream>>>(p, tiles);
  else if (each) rs_matmul_tile_kernel<BM, BN, WM, S, KG, true, false, FAR><<<grid, 512, 0, stream>>>(p, tiles);
  else if (exact) rs_matmul_tile_kernel<BM, BN, WM, S, KG, false, true, FAR><<<grid, 512, 0, stream>>>(p, tiles);
  else rs_matmul_tile_kernel<BM, BN, WM, S, KG, false, false, FAR><<<grid, 512, 0, stream>>>(p, tiles);
  return hipGetLastError();
}

template <int MT, int NT, int U, int W>
hipError_t launch_stream(MatmulArgs p, bool each, bool exact, int64_t row_tiles, hipStream_t stream) {
  constexpr int kThreads = W * 64;
  p.n_tiles = (p.n + NT * 16 - 1) / (NT * 16);
  if (too_many(row_tiles * p.n_tiles, kThreads)) return hipErrorInvalidConfiguration;
  const dim3 grid(uint32_t(row_tiles * p.n_tiles));
  if (each && exact) rs_matmul_stream_kernel<MT, NT, U, W, true, true><<<grid, kThreads, 0, stream>>>(p);
  else if (each) rs_matmul_stream_kernel<MT, NT, U, W, true, false><<<grid, kThreads, 0, stream>>>(p);
  else if (exact) rs_matmul_stream_kernel<MT, NT, U, W, false, true><<<grid, kThreads, 0, stream>>>(p);
  else rs_matmul_stream_kernel<MT, NT, U, W, false, false><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantise(const rs_fp8_quant& q, const void* x, const int32_t* row_count, uint8_t* codes,
                           float* scales, hipStream_t stream) {
  QuantArgs p{x, row_count, codes, scales, q.rows, q.cols, q.x_stride, q.x_batch_stride, q.code_stride,
              q.code_batch_stride, q.scale_stride, q.scale_batch_stride, blocks128(q.rows), blocks128(q.cols), 0};
  p.magic = ~uint64_t(0) / uint64_t(p.tiles_n) + 1;
  const auto run = [&](auto dtype, auto gated) {
    constexpr int kType = decltype(dtype)::value;
    constexpr bool kGated = decltype(gated)::value;
    if (q.block_rows == 1 && !q.transpose) quant_rows<kType, kGated>(p, q.batch, stream);
    else quant_tiles<kType, kGated>(p, q.block_rows == 1, q.transpose, q.batch, stream);
  };
  const auto typed = [&](auto dtype) { q.gated ? run(dtype, std::true_type()) : run(dtype, std::false_type()); };
  if (q.dtype == RS_BF16) typed(std::integral_constant<int, RS_BF16>());
  else if (q.dtype == RS_F16) typed(std::integral_constant<int, RS_F16>());
  else typed(std::integral_constant<int, RS_F32>());
  return hipGetLastError();
}

hipError_t launch_matmul(const rs_fp8_matmul& mm, const uint8_t* a, const float* a_scales,
                         const int32_t* a_index, const uint8_t* b, const float* b_scales,
                         const int32_t* offsets, void* c, hipStream_t stream) {
  MatmulArgs p{a, a_scales, a_index, b, b_scales, offsets, c, mm.m, mm.a_rows, mm.a_stride, mm.a_scale_stride,
               mm.b_stride, mm.b_scale_stride, mm.b_group_stride, mm.b_scale_group_stride, mm.c_stride,
               int32_t(mm.n), int32_t(mm.k), mm.n_groups, int32_t(blocks128(mm.k)), 0,
               int32_t(mm.b_split ? mm.b_split : mm.n), int32_t(blocks128(mm.b_split)), mm.out_dtype, mm.b_block_rows};
  const bool each = mm.b_block_rows == 1 || mm.b_split % kBlock != 0, exact = mm.out_dtype != RS_BF16;
  const auto row_tiles = [&](int64_t rows) {
    return mm.m / rows + (mm.n_groups ? min(int64_t(mm.n_groups), mm.m) : (mm.m % rows != 0));
  };
  switch (matmul_shape(mm, a_index != nullptr)) {
    case MatmulShape::kStream16x64: return launch_stream<1, 4, 2, 4>(p, each, exact, row_tiles(16), stream);
    case MatmulShape::kStream16x16: return launch_stream<1, 1, 4, 8>(p, each, exact, row_tiles(16), stream);
    case MatmulShape::kStream32x32: return launch_stream<2, 2, 2, 8>(p, each, exact, row_tiles(32), stream);
    case MatmulShape::kFar64x256: return launch_tile<64, 256, 1, 3, 1, true>(p, each, exact, row_tiles(64), stream);
    case MatmulShape::k256x256: return launch_tile<256, 256, 4, 2, 1>(p, each, exact, row_tiles(256), stream);
    case MatmulShape::k128x256: return launch_tile<128, 256, 2, 3, 1>(p, each, exact, row_tiles(128), stream);
    case MatmulShape::k64x256: return launch_tile<64, 256, 1, 3, 1>(p, each, exact, row_tiles(64), stream);
    case MatmulShape::k64x128: return launch_tile<64, 128, 2, 3, 1>(p, each, exact, row_tiles(64), stream);
    case MatmulShape::k64x64: return launch_tile<64, 64, 1, 2, 4>(p, each, exact, row_tiles(64), stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace rs
