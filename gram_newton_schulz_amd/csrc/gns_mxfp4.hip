// Microscaled 4-bit floating point (MXFP4), written for CDNA4 (gfx950): a value
// is a code of {0, 1/2, 1, 3/2, 2, 3, 4, 6} and sign times the power of two of its
// block of 32.
//
// * mx_quantize   -- codes and scales of a matrix, of its transpose, or of both
//                    from one read of it.  HBM-bound: 8192 x 16384 bf16 both
//                    ways in 90 us (4.6 TB/s).
// * mx_dequantize -- the values back.  HBM-bound.
// * mx_gemm       -- C = A B^T of two quantised matrices by scaled MFMA.  Where it is
//                    large the matrix cores are busy 57% of the time at the clock
//                    that the power leaves, 1.63 GHz (8192^3: 272 us, 4.0 PFLOP/s);
//                    codes of zero take 190 us at a higher clock and about the same
//                    share.
// * mx_join       -- the sum of such a product's parts of the contraction.
// * mx_thin       -- C = A B^T of few rows of A: bound by the bytes of B.  It can
//                    quantise A itself.
//
// Codes lie two to a byte, rows of whole 128 columns; the scales of 32 rows and
// 128 columns are 128 consecutive bytes, a word of four per row.  Both are padded
// with zeros, so that no product looks at where a contraction ends.  Sums are fp32
// in a fixed order, rounded once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gns_elem.h"
#include "gns_kernels.h"

namespace gns {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));   // anywhere
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// quantisation
// ---------------------------------------------------------------------------
// Scale byte of a block whose largest magnitude has these bits: the exponent
// of the largest value less 2, which puts it into [4, 8) of the grid.  With
// noise, one more where it would be above 6, the largest value of the grid.
__device__ __forceinline__ uint32_t scale_byte(uint32_t largest, bool unclipped) {
  const uint32_t e = largest >> 23;
  if (e == 255) return 255;
  if (e < 2) return 0;
  return e - 2 + (unclipped && (largest & 0x7fffff) > 0x400000 ? 1 : 0);
}
// 2^(s - 127) as fp32 (subnormal for s = 0)
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x400000u); }
// 2^(127 - s), s <= 254
__device__ __forceinline__ float inverse_scale(uint32_t s) {
  return __uint_as_float(s < 254 ? (254 - s) << 23 : 0x400000u);
}

// x rounded up with its probability (t = |x| / scale <= 6, exactly)
__device__ __forceinline__ uint32_t noisy_code(float x, float inverse, uint32_t noise) {
  const float t = fabsf(x) * inverse;
  const float steps = t < 2.0f ? 2.0f * t : t < 4.0f ? t + 2.0f : 0.5f * t + 4.0f;
  const float whole = floorf(steps);
  const uint32_t up = (steps - whole) * 256.0f > static_cast<float>(noise) + 0.5f ? 1 : 0;
  return (static_cast<uint32_t>(whole) + up) | (__float_as_uint(x) >> 31 << 3);
}

// Eight consecutive values of a row, as they lie in memory.
template <class T>
struct Octet {
  static constexpr bool k16 = sizeof(typename T::S) == 2;
  uint32_t w[k16 ? 4 : 8];

  // `left` of them are there, the others are zero.  (16-byte accesses need no
  // alignment beyond the element's.)
  __device__ __forceinline__ void load(const typename T::S *src, int left, bool once = false) {
    if (left >= 8) {
      if (once) {
#pragma unroll
        for (int i = 0; i < (k16 ? 4 : 8); i += 4) {
          const u32x4_any t = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(src) + i / 4);
          w[i] = t[0], w[i + 1] = t[1], w[i + 2] = t[2], w[i + 3] = t[3];
        }
      } else {
        __builtin_memcpy(w, src, sizeof(w));
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < (k16 ? 4 : 8); ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      if (i >= left) break;
      if constexpr (k16) w[i / 2] |= static_cast<uint32_t>(src[i]) << (16 * (i & 1));
      else w[i] = __float_as_uint(src[i]);
    }
  }
  // bits of the largest magnitude, as a float's
  __device__ __forceinline__ uint32_t largest() const {
    if constexpr (k16) {
      u16x2 m{0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
      return __float_as_uint(T::ld(max(m[0], m[1])));
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    }
  }
};

// The value of another lane of 16, where values are equal within the groups
// that it spans: lane ^ 1, ^ 2 (quads), ^ 4 (mirrored halves) or ^ 8 (mirrored
// rows of 16 lanes).
template <int D>
__device__ __forceinline__ uint32_t other_lane(uint32_t v) {
  constexpr int kControl = D == 1 ? 0xb1 : D == 2 ? 0x4e : D == 4 ? 0x141 : 0x140;
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kControl, 0xf, 0xf, true));
}

// Two codes into byte SEL of old: the conversion divides by the scale, rounds
// to nearest with ties to even and cuts off at 6.
template <class T, int SEL>
__device__ __forceinline__ uint32_t two_codes(uint32_t old, uint32_t low, uint32_t high, float scale) {
  if constexpr (T::code == DT_F32) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __uint_as_float(low), __uint_as_float(high), scale, SEL);
  } else {
    const uint32_t pair = __builtin_amdgcn_perm(high, low, 0x05040100u);   // their low halves
    if constexpr (T::code == DT_BF16)
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, pair), scale, SEL);
    else
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2_t, pair), scale, SEL);
  }
}

// Eight codes of values given by their bits (16-bit ones in the low half).
template <class T, bool NOISE>
__device__ __forceinline__ uint32_t eight_codes(const uint32_t *bits, const uint32_t *noise, uint32_t s) {
  uint32_t word = 0;
  if constexpr (NOISE) {
    const float inverse = inverse_scale(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v;
      if constexpr (T::code == DT_F32) v = __uint_as_float(bits[i]);
      else v = T::ld(static_cast<typename T::S>(bits[i]));
      word |= noisy_code(v, inverse, noise[i]) << (4 * i);
    }
  } else {
    const float scale = scale_of(s);
    word = two_codes<T, 0>(word, bits[0], bits[1], scale);
    word = two_codes<T, 1>(word, bits[2], bits[3], scale);
    word = two_codes<T, 2>(word, bits[4], bits[5], scale);
    word = two_codes<T, 3>(word, bits[6], bits[7], scale);
  }
  return s == 255 ? 0 : word;
}

struct MxQuantize {
  const void *x;
  int64_t pitch, batch_stride;
  const uint8_t *noise;
  int64_t rows, cols;
  MxMatrix by_rows, by_columns;
  int64_t batch;
  int tiles_r, tiles_c;
  int once;                     // x is read with the streaming hint
  int dealt;                    // XCDs take squares of four tiles
};
// A matrix that fills the last-level cache has the hint, so that its codes stay
// there for the product (the layer gradients of 8192 x 16384 bf16: 704 -> 693 us,
// quantising 4096 x 16384 fp32 both ways and back 157 -> 140); a smaller one may
// still lie there itself (8192 x 4096 bf16 through a layer: 304 us, 308 with it).
constexpr int64_t kLastLevelCache = int64_t(256) << 20;
// Half of a line of codes belongs to each of two neighbouring tiles, in both
// orders.  Squares of four tiles go to one XCD, whose L2 joins the halves, where
// there are many tiles (both ways: 8192 x 16384 bf16 103 -> 90 us, 32768 x 4096 bf16
// 93 -> 82, 16389 x 8330 bf16 129 -> 113, 4096 x 16384 fp32 76.5 -> 74.6); fewer
// are spread over the GPU one by one (8192 x 4096 bf16 by rows: 15.4 us, 16.7 in
// squares).
constexpr int64_t kDealtTiles = 4096, kMaxDealt = int64_t(1) << 22;   // (a grid holds 2^24 workgroups)

// A workgroup per tile of 128 rows and kCols columns.  Along the rows a thread
// takes eight values, and four neighbours share a block.  Along the columns the
// tile lies in LDS, and a thread takes 32 rows of one column (of two
// neighbouring ones of a 16-bit type); the four threads of a column are
// neighbours, so that they write its 64 bytes of codes together.  A row of LDS
// has its 16-byte pieces exchanged by its block of 32 rows, which puts those
// four threads on different banks.
// kCols is 128, the extent of a word of scales, but for fp32 matrices of few
// tiles, where tiles of 64 make twice the workgroups (both ways, 3 x 257 x 1531
// with noise: 16.5 -> 9.8 us; 4096 x 16384: 71 -> 87, as its rows of codes are
// written in halves).  Both ways, 8192 x 16384 bf16 take 90 us (4.6 TB/s).  With
// noise the arithmetic bounds it, twice the vector instructions: 185 us there, 136
// against 76 for 4096 x 16384 fp32.  With
// 32 rows of four columns per thread in registers instead of LDS, fp32 4096 x
// 16384 took 166: its stores along the columns are scattered.
template <class T, bool ROWS, bool COLS, bool NOISE, int kCols>
__global__ void __launch_bounds__(256) mx_quantize(MxQuantize p) {
  using S = typename T::S;
  constexpr bool k16 = sizeof(S) == 2;
  constexpr int kRowWords = kCols * sizeof(S) / 4;           // of LDS
  constexpr int kLanes = kCols / 8, kRows = 256 / kLanes;    // threads to a row, rows at a time
  constexpr int kNoiseWords = kCols / 4;
  __shared__ __attribute__((aligned(16))) uint32_t tile[COLS ? 128 * kRowWords : 4];
  __shared__ __attribute__((aligned(16))) uint32_t noises[COLS && NOISE ? 128 * kNoiseWords : 4];
  const int tid = threadIdx.x, lane = tid & 63;
  int64_t tile_index = blockIdx.x;
  int tiles_r = p.tiles_r, tiles_c = p.tiles_c;
  if (p.dealt) {
    tile_index = static_cast<int64_t>(blockIdx.x / 32) * 8 + blockIdx.x % 8;   // of the square
    tiles_r = (tiles_r + 1) / 2;
    tiles_c = (tiles_c + 1) / 2;
  }
  const int64_t per_matrix = static_cast<int64_t>(tiles_r) * tiles_c;
  const int64_t mat = tile_index / per_matrix;
  const int in = static_cast<int>(tile_index - mat * per_matrix);
  int tile_r = in / tiles_c, tile_c = in % tiles_c;
  if (p.dealt) {
    const int corner = blockIdx.x / 8 % 4;
    tile_r = tile_r * 2 + corner / 2;
    tile_c = tile_c * 2 + corner % 2;
    if (mat >= p.batch || tile_r >= p.tiles_r || tile_c >= p.tiles_c) return;
  }
  const int64_t row0 = static_cast<int64_t>(tile_r) * 128, col0 = static_cast<int64_t>(tile_c) * kCols;
  const S *x = static_cast<const S *>(p.x) + mat * p.batch_stride;
  const uint8_t *noise = NOISE ? p.noise + mat * p.rows * p.cols : nullptr;
  const int r_in = tid / kLanes, c_in = (tid % kLanes) * 8;
  const int64_t col = col0 + c_in;
  const int left = static_cast<int>(min<int64_t>(8, p.cols - col));       // of the eight
  const int64_t groups = p.by_rows.groups(), row_blocks = p.by_rows.row_blocks();

  constexpr int kAhead = 4;
  const int64_t last = COLS ? row0 + 128 : min<int64_t>(row0 + 128, (p.rows + 31) / 32 * 32);
  for (int k0 = 0; k0 < 128 && row0 + k0 < last; k0 += kRows * kAhead) {
    Octet<T> v[kAhead];
    uint32_t r[kAhead][2];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t row = row0 + k0 + kRows * a + r_in;
      const int here = row < p.rows ? left : 0;
      v[a].load(x + row * p.pitch + col, here, p.once);
      r[a][0] = r[a][1] = 0;
      if constexpr (NOISE) {
        const uint8_t *from = noise + row * p.cols + col;
        if (here >= 8) {
          __builtin_memcpy(r[a], from, 8);
        } else {
#pragma unroll
          for (int i = 0; i < 7; ++i)
            if (i < here) r[a][i / 4] |= static_cast<uint32_t>(from[i]) << (8 * (i & 3));
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int in_tile = k0 + kRows * a + r_in;
      const int64_t row = row0 + in_tile;
      if constexpr (COLS) {
        // (piece of 16 bytes ^ 4 x block of 32 rows)
        uint4 *to = reinterpret_cast<uint4 *>(tile + in_tile * kRowWords);
        const int turn = (in_tile >> 5) << 2;
#pragma unroll
        for (int i = 0; i < (k16 ? 1 : 2); ++i)
          to[((tid % kLanes) * (k16 ? 1 : 2) + i) ^ turn] = *reinterpret_cast<const uint4 *>(v[a].w + 4 * i);
        if constexpr (NOISE)
          *reinterpret_cast<uint2 *>(noises + in_tile * kNoiseWords +
                                     ((2 * (tid % kLanes)) ^ ((in_tile >> 5) * (kNoiseWords / 4)))) = make_uint2(r[a][0], r[a][1]);
      }
      if constexpr (ROWS) {
        uint32_t largest = v[a].largest();
        largest = max(largest, other_lane<1>(largest));
        largest = max(largest, other_lane<2>(largest));
        const uint32_t s = scale_byte(largest, NOISE);
        uint32_t bits[8], bytes[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          bits[i] = k16 ? v[a].w[i / 2] >> (16 * (i & 1)) & 0xffff : v[a].w[k16 ? 0 : i];
          bytes[i] = NOISE ? r[a][i / 4] >> (8 * (i & 3)) & 0xff : 0;
        }
        const uint32_t word = eight_codes<T, NOISE>(bits, bytes, s);
        // a row's scales of this tile: a word, or half of one
        uint32_t scales = s << (8 * (tid % kLanes / 4));
        scales |= other_lane<4>(scales);
        if constexpr (kCols == 128) scales |= other_lane<8>(scales);
        if (row < p.rows) {
          *reinterpret_cast<uint32_t *>(p.by_rows.codes + (mat * p.rows + row) * (groups * 64) + (col0 + c_in) / 2) = word;
        } else {
          scales = 0;
        }
        if (tid % kLanes == 0 && row < row_blocks * 32) {
          uint8_t *to = p.by_rows.scales + (((mat * row_blocks + row / 32) * groups + col0 / 128) * 32 + row % 32) * 4;
          if constexpr (kCols == 128) *reinterpret_cast<uint32_t *>(to) = scales;
          else *reinterpret_cast<uint16_t *>(to + col0 % 128 / 32) = static_cast<uint16_t>(scales);
        }
      }
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    const int64_t t_groups = p.by_columns.groups(), t_blocks = p.by_columns.row_blocks();
    const int rb = lane & 3, turn = rb << 4;
    constexpr int kSub = k16 ? 2 : 1;                        // columns of a thread at a time
#pragma unroll 1
    for (int it = 0; it < kRowWords / 64; ++it) {
      const int c = (lane >> 2) + 16 * (tid >> 6) + 64 * it; // column, or pair of columns
      uint32_t raw[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) raw[i] = tile[(32 * rb + i) * kRowWords + (c ^ turn)];
#pragma unroll
      for (int h = 0; h < kSub; ++h) {
        const int64_t column = col0 + c * kSub + h;
        uint32_t bits[32], bytes[32], largest = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          bits[i] = k16 ? raw[i] >> (16 * h) & 0xffff : raw[i];
          largest = max(largest, bits[i] & (k16 ? 0x7fffu : 0x7fffffffu));
          const int b = c * kSub + h;                        // its byte of noise
          bytes[i] = NOISE ? noises[(32 * rb + i) * kNoiseWords + ((b >> 2) ^ (rb * (kNoiseWords / 4)))] >> (8 * (b & 3)) & 0xff : 0;
        }
        if constexpr (k16) largest = __float_as_uint(T::ld(static_cast<S>(largest)));
        const uint32_t s = scale_byte(largest, NOISE);
        uint4 word;
        word.x = eight_codes<T, NOISE>(bits, bytes, s);
        word.y = eight_codes<T, NOISE>(bits + 8, bytes + 8, s);
        word.z = eight_codes<T, NOISE>(bits + 16, bytes + 16, s);
        word.w = eight_codes<T, NOISE>(bits + 24, bytes + 24, s);
        uint32_t scales = s << (8 * rb);
        scales |= other_lane<1>(scales);
        scales |= other_lane<2>(scales);
        if (column < p.cols) {
          *reinterpret_cast<uint4 *>(p.by_columns.codes + (mat * p.cols + column) * (t_groups * 64) + row0 / 2 + rb * 16) =
              word;
        } else {
          scales = 0;
        }
        if (rb == 0 && column < t_blocks * 32)
          *reinterpret_cast<uint32_t *>(p.by_columns.scales + (((mat * t_blocks + column / 32) * t_groups + row0 / 128) * 32 +
                                                               column % 32) * 4) = scales;
      }
    }
  }
}

// The values of a tile of 64 rows and 256 columns, eight per thread: whole lines
// of codes (4096 x 16384: 39 us, 4.4 TB/s; 41 in tiles of 128 columns).
constexpr int64_t kTilesX = int64_t(1) << 23;   // of a grid's first dimension
template <class T>
__global__ void __launch_bounds__(256) mx_dequantize(MxMatrix q, typename T::S *out, int tiles_r, int tiles_c) {
  using S = typename T::S;
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const int tid = threadIdx.x;
  const int64_t per_matrix = static_cast<int64_t>(tiles_r) * tiles_c, tile = blockIdx.y * kTilesX + blockIdx.x,
                mat = tile / per_matrix;
  if (mat >= q.batch) return;
  const int in = static_cast<int>(tile - mat * per_matrix);
  const int64_t row0 = static_cast<int64_t>(in / tiles_c) * 64, groups = q.groups();
  const int64_t col = static_cast<int64_t>(in % tiles_c) * 256 + (tid & 31) * 8, group = col / 128;
  if (col >= q.cols) return;
  uint32_t words[8], bytes[8];                               // (all loads before the first store)
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t row = min(row0 + 8 * k + (tid >> 5), q.rows - 1);
    words[k] = *reinterpret_cast<const uint32_t *>(q.codes + (mat * q.rows + row) * q.pitch() + col / 2);
    bytes[k] = q.scales[(((mat * q.row_blocks() + row / 32) * groups + group) * 32 + row % 32) * 4 + ((tid >> 2) & 3)];
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t row = row0 + 8 * k + (tid >> 5);
    if (row >= q.rows) return;
    const uint32_t w = words[k], s = bytes[k];
    const float scale = s == 255 ? __uint_as_float(0x7fc00000u) : scale_of(s);
    float v[8];
    const auto two = [&](int i, f32x2 x) {
      // (a scale of NaN by itself: the conversion takes its exponent only)
      v[i] = s == 255 ? scale : x[0];
      v[i + 1] = s == 255 ? scale : x[1];
    };
    two(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0));
    two(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1));
    two(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2));
    two(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3));
    S *to = out + (mat * q.rows + row) * q.cols + col;
    if (col + 8 <= q.cols) {
      // (16-byte accesses need no alignment beyond the element's)
      if constexpr (sizeof(S) == 4) {
        __builtin_memcpy(to, v, 32);
      } else {
        const uint32_t pairs[4] = {T::st2(v[0], v[1]), T::st2(v[2], v[3]), T::st2(v[4], v[5]), T::st2(v[6], v[7])};
        __builtin_memcpy(to, pairs, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < q.cols) to[i] = T::st(v[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
template <class F>
hipError_t with_type(int dtype, F &&f) {
  if (dtype == DT_F32) return f(EF32{});
  if (dtype == DT_BF16) return f(EBF16{});
  return f(EF16{});
}

template <class F>
hipError_t with_flag(bool on, F &&f) {
  return on ? f(std::true_type{}) : f(std::false_type{});
}

__device__ __forceinline__ i32x8 fp4_operand(uint4 v) {
  return i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
}

// C = A B^T in tiles of TM x TN by WGM x WGN waves.  An MFMA multiplies 32 x 64
// codes by 32 x 64: lane l holds one block of 32 codes of row l % 32 of either
// factor, 16 bytes, and its scale.  A stage of the contraction is 128 columns:
// 64 bytes of codes of every row, as four 16-byte chunks, and one word of
// scales of every row.  Both come from HBM or L2 straight into LDS (LDS-DMA)
// into a ring of stages.  The fragments of B are the instruction's rows, so
// that a lane's accumulators are runs of four consecutive columns of C.
template <int TM_, int TN_, int WGM_, int WGN_, int STAGES_>
struct MxTile {
  static constexpr int TM = TM_, TN = TN_, WGM = WGM_, WGN = WGN_, STAGES = STAGES_;
  static constexpr int NW = WGM * WGN, THREADS = 64 * NW;
  static constexpr int WTM = TM / WGM, WTN = TN / WGN;
  static constexpr int NBM = WTM / 32, NBN = WTN / 32;           // 32 x 32 blocks of a wave
  static constexpr int CODES_A = TM * 64, CODES_B = TN * 64;     // bytes of codes in a stage
  static constexpr int PIECES_A = TM / 32, PIECES_B = TN / 32;   // 128-byte pieces of scales
  static constexpr int STAGE = CODES_A + CODES_B + (PIECES_A + PIECES_B) * 128;
  static constexpr int LDS = STAGES * STAGE;
  static constexpr int LOADS_A = TM / 16 / NW, LOADS_B = TN / 16 / NW;         // of 1 KiB, per wave
  static constexpr int PAIRS = (PIECES_A + PIECES_B) / 2;                      // of pieces: a load of scales each
  static constexpr int LOADS_S = (PAIRS + NW - 1) / NW;
  static constexpr int LOADS = LOADS_A + LOADS_B + LOADS_S;      // of a wave per stage
  static_assert(LOADS_A * NW * 16 == TM && LOADS_B * NW * 16 == TN && PIECES_A % 2 == 0, "whole loads");
  static_assert(LDS <= 160 * 1024 && TM * (TN + 8) * 2 <= LDS, "LDS");
};

struct MxGemm {
  MxMatrix a, b;
  MxOutput o;
  int tiles_m, tiles_n;
  int run;             // consecutive tiles dealt to one XCD
  int parts;           // of the contraction
  int64_t part_stride; // elements from one part's results to the next's
  int once;            // results that are there are read with the streaming hint
};

// chunk c of row r lies at chunk c ^ swizzle(r): rows that share a bank have
// different chunks in the same place
__device__ __forceinline__ int swizzle(int row) { return ((row >> 1) ^ (row >> 2)) & 3; }

__device__ __forceinline__ i32x4 buffer_of(const uint8_t *at, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(at);
  return i32x4{__builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a))),
               __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a >> 32) & 0xffff)),
               __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000};
}

template <class TO, class L>
__global__ void __launch_bounds__((L::THREADS)) mx_gemm(MxGemm p) {
  using S = typename TO::S;
  __shared__ __attribute__((aligned(16))) unsigned char lds[L::LDS];

  // Workgroup -> tile: runs of tiles go to the XCDs in turn (workgroups do one
  // by one), and within a run 4 x 8 tiles share their panels.
  int64_t t = blockIdx.x;
  {
    const int64_t g8 = gridDim.x & ~7u;
    if (t < g8) {
      const int64_t slot = t >> 3;
      t = ((slot / p.run) * 8 + (t & 7)) * p.run + slot % p.run;
    }
  }
  const int64_t per_matrix = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  const int part = static_cast<int>(t / (per_matrix * p.a.batch));
  t -= part * per_matrix * p.a.batch;
  const int64_t mat = t / per_matrix;
  int ti, tj;
  {
    constexpr int kBand = 4;
    const int r = static_cast<int>(t - mat * per_matrix), band = r / (kBand * p.tiles_n);
    const int high = min(p.tiles_m - band * kBand, kBand), in = r - band * kBand * p.tiles_n;
    ti = band * kBand + in % high;
    tj = in / high;
  }

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, lh = lane >> 5;
  const int wr = (wave / L::WGN) * L::WTM, wc = (wave % L::WGN) * L::WTN;

  const int groups = __builtin_amdgcn_readfirstlane(static_cast<int>(p.a.groups())), pitch = groups * 64;
  const int per_part = (groups + p.parts - 1) / p.parts;
  const int first = __builtin_amdgcn_readfirstlane(part * per_part);
  const int stages = min(groups - first, per_part);

  // this tile's rows of codes and scales; what lies past the last row reads as zero
  // (the range check counts the scalar offset, too)
  auto panel = [&](const MxMatrix &q, int64_t row, int high, i32x4 *codes, i32x4 *scales) {
    const int64_t blocks = q.row_blocks();
    *codes = buffer_of(q.codes + (mat * q.rows + row) * pitch, min<int64_t>(high, q.rows - row) * pitch);
    *scales = buffer_of(q.scales + (mat * blocks + row / 32) * groups * 128,
                        min<int64_t>(high / 32, blocks - row / 32) * groups * 128);
  };
  const int64_t row0 = static_cast<int64_t>(ti) * L::TM, col0 = static_cast<int64_t>(tj) * L::TN;
  i32x4 ca, cb, sa, sb;
  panel(p.a, row0, L::TM, &ca, &sa);
  panel(p.b, col0, L::TN, &cb, &sb);
  const uint32_t lds_base =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char *)(lds)));

  // (A load into LDS needs a wait state after a write of m0, its address; inside
  // a block of assembly the compiler inserts none.)
  // Lane l of a load of codes fills 16 bytes of row l / 4 of its 16 rows, at
  // chunk l % 4; a load of scales fills two pieces, a word per lane.
  const int dma_row = lane >> 2;
  const int code_at = dma_row * pitch + ((lane & 3) ^ swizzle(dma_row)) * 16;
  const int scale_at = lh * groups * 128 + lr * 4;
  auto fetch = [&](int stage, int slot) {
    // stages past the last one go through an empty range: every stage has the
    // same number of loads, and these fetch nothing
    const bool live = stage < stages;
    const int at = first + (live ? stage : 0);
    const uint32_t to = lds_base + static_cast<uint32_t>(slot * L::STAGE);
    i32x4 a = ca, b = cb;
    if (!live) a[2] = b[2] = 0;
#pragma unroll
    for (int q = 0; q < L::LOADS_A; ++q) {
      const int blk = wave + q * L::NW;
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to + blk * 1024), "v"(code_at),
                   "s"(a), "s"(blk * 16 * pitch + at * 64)
                   : "memory", "m0");
    }
#pragma unroll
    for (int q = 0; q < L::LOADS_B; ++q) {
      const int blk = wave + q * L::NW;
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to + L::CODES_A + blk * 1024),
                   "v"(code_at), "s"(b), "s"(blk * 16 * pitch + at * 64)
                   : "memory", "m0");
    }
#pragma unroll
    for (int q = 0; q < L::LOADS_S; ++q) {
      // (a wave with no pair left repeats the last one: the same bytes to the same place)
      const int pair = min(wave + q * L::NW, L::PAIRS - 1);
      const bool of_a = pair < L::PIECES_A / 2;
      i32x4 x = of_a ? sa : sb;
      if (!live) x[2] = 0;
      const int piece = 2 * pair - (of_a ? 0 : L::PIECES_A);
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                   ::"s"(to + L::CODES_A + L::CODES_B + pair * 256), "v"(scale_at), "s"(x),
                   "s"(piece * groups * 128 + at * 128)
                   : "memory", "m0");
    }
  };

  f32x16 acc[L::NBN][L::NBM];
#pragma unroll
  for (int j = 0; j < L::NBN; ++j)
#pragma unroll
    for (int i = 0; i < L::NBM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

  const int sw = swizzle(lr);
  uint4 fa[2][L::NBM], fb[2][L::NBN];
  int xa[L::NBM], xb[L::NBN];
  // Fragments of a stage: half h of slice s is chunk 2 s + h.  Shifted by h
  // bytes, a row's word has the scales of its slices in bytes 0 and 2.
  auto read = [&](int slot) {
    const unsigned char *at = lds + slot * L::STAGE;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int chunk = ((2 * s + lh) ^ sw) * 16;
#pragma unroll
      for (int i = 0; i < L::NBM; ++i)
        fa[s][i] = *reinterpret_cast<const uint4 *>(at + (wr + 32 * i + lr) * 64 + chunk);
#pragma unroll
      for (int j = 0; j < L::NBN; ++j)
        fb[s][j] = *reinterpret_cast<const uint4 *>(at + L::CODES_A + (wc + 32 * j + lr) * 64 + chunk);
    }
    const unsigned char *words = at + L::CODES_A + L::CODES_B + lr * 4;
#pragma unroll
    for (int i = 0; i < L::NBM; ++i)
      xa[i] = *reinterpret_cast<const uint32_t *>(words + (wr / 32 + i) * 128) >> (8 * lh);
#pragma unroll
    for (int j = 0; j < L::NBN; ++j)
      xb[j] = *reinterpret_cast<const uint32_t *>(words + (L::PIECES_A + wc / 32 + j) * 128) >> (8 * lh);
  };
  auto multiply = [&]() {
#pragma unroll
    for (int j = 0; j < L::NBN; ++j)
#pragma unroll
      for (int i = 0; i < L::NBM; ++i)
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(fb[0][j]), fp4_operand(fa[0][i]),
                                                                   acc[j][i], 4, 4, 0, xb[j], 0, xa[i]);
#pragma unroll
    for (int j = 0; j < L::NBN; ++j)
#pragma unroll
      for (int i = 0; i < L::NBM; ++i)
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(fb[1][j]), fp4_operand(fa[1][i]),
                                                                   acc[j][i], 4, 4, 2, xb[j], 2, xa[i]);
  };

#pragma unroll
  for (int i = 0; i < L::STAGES - 1; ++i) fetch(i, i);
  constexpr int kWait = L::LOADS * (L::STAGES - 2);      // this wave's loads of later stages
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kWait) : "memory");
  __syncthreads();
  // Stage i + STAGES - 1 goes to the place of stage i - 1, which every wave has
  // finished reading.
  int slot = 0, next = L::STAGES - 1;
  if constexpr (L::NW == 8) {
    // The two waves of a SIMD are one barrier apart: one multiplies while the
    // other reads.
    const bool second = wave >= 4;
    if (second) __syncthreads();
    for (int i = 0; i < stages; ++i) {
      read(slot);
      fetch(i + L::STAGES - 1, next);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kWait) : "memory");
      __syncthreads();
      __builtin_amdgcn_s_setprio(1);
      multiply();
      __builtin_amdgcn_s_setprio(0);
      __syncthreads();
      next = slot;
      slot = slot == L::STAGES - 1 ? 0 : slot + 1;
    }
    if (!second) __syncthreads();
  } else {
    for (int i = 0; i < stages; ++i) {
      read(slot);
      fetch(i + L::STAGES - 1, next);
      multiply();
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kWait) : "memory");
      __syncthreads();
      next = slot;
      slot = slot == L::STAGES - 1 ? 0 : slot + 1;
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // Results leave in whole rows, which takes a way through LDS: 16-bit ones of the
  // whole workgroup (8192 x 4096 by 16384 x 4096: 312 us with the quantisation, 325
  // straight from registers), fp32 ones and those that are added to what is there
  // 32 rows of a wave at a time (4096 x 8192 by 16384 x 8192 into fp32 285 us,
  // added 332; straight from registers 341 and 373, as a lane has four columns).
  // Tiles of four waves, whose results are small, store the latter straight from
  // registers (1000 x 777 x 513: 25.9 us for both gradients, 27.6 through LDS).
  // Accesses of 16 bytes need no alignment beyond the element's.
  S *const out = static_cast<S *>(p.o.out) + part * p.part_stride + mat * p.o.batch_stride;
  const int64_t rows = p.a.rows, cols = p.b.rows;
  if constexpr (sizeof(S) == 2) {
    if (!p.o.accumulate) {
      constexpr int kPitch = L::TN + 8;
      S *const staged = reinterpret_cast<S *>(lds);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < L::NBN; ++j)
#pragma unroll
        for (int i = 0; i < L::NBM; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<uint2 *>(staged + (wr + 32 * i + lr) * kPitch + wc + 32 * j + 8 * g + 4 * lh) =
                make_uint2(TO::st2(acc[j][i][4 * g], acc[j][i][4 * g + 1]),
                           TO::st2(acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]));
      __syncthreads();
#pragma unroll 4
      for (int k = tid; k < L::TM * L::TN / 8; k += L::THREADS) {
        const int r = k / (L::TN / 8), c = k % (L::TN / 8) * 8;
        const int64_t row = row0 + r, col = col0 + c;
        if (row >= rows || col >= cols) continue;
        const S *from = staged + r * kPitch + c;
        S *to = out + row * p.o.pitch + col;
        if (col + 8 <= cols) {
          const uint4 v = *reinterpret_cast<const uint4 *>(from);
          // (the streaming hint keeps the factors' panels in the L2: 317 -> 304 us)
          __builtin_nontemporal_store(u32x4_any{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_any *>(to));
        } else {
          for (int e = 0; col + e < cols; ++e) to[e] = from[e];
        }
      }
      return;
    }
  }
  if constexpr (L::NW == 8) {
    constexpr int kPitch = L::WTN + 4, kLanes = L::WTN / 4, kAt = 64 / kLanes, kSteps = 32 / kAt;
    static_assert(L::NW * 32 * kPitch * 4 <= L::LDS, "LDS");
    float *const staged = reinterpret_cast<float *>(lds) + wave * 32 * kPitch;
    const int c = lane % kLanes * 4;
    const int64_t col = col0 + wc + c;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < L::NBM; ++i) {
      const int64_t first_row = row0 + wr + 32 * i + lane / kLanes;
      uint32_t old[kSteps][sizeof(S)] = {};                  // four values each
      if (p.o.accumulate) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int64_t row = first_row + k * kAt;
          const S *from = out + row * p.o.pitch + col;
          if (row < rows && col + 4 <= cols) {
            // (results of 256 MiB, whose streaming hint leaves the L2 to the factors'
            // panels: the layer gradients of that product 667 -> 654 us)
            using W = std::conditional_t<sizeof(S) == 4, f32x4_any, u32x2_any>;
            const W v = p.once ? __builtin_nontemporal_load(reinterpret_cast<const W *>(from))
                               : *reinterpret_cast<const W *>(from);
            __builtin_memcpy(old[k], &v, sizeof(v));
          } else if (row < rows) {
            S few[4] = {};
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (col + e < cols) few[e] = from[e];
            __builtin_memcpy(old[k], few, sizeof(few));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < L::NBN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float4 *>(staged + lr * kPitch + 32 * j + 8 * g + 4 * lh) =
              make_float4(acc[j][i][4 * g], acc[j][i][4 * g + 1], acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int64_t row = first_row + k * kAt;
        const float4 v = *reinterpret_cast<const float4 *>(staged + (k * kAt + lane / kLanes) * kPitch + c);
        const float x[4] = {v.x, v.y, v.z, v.w};
        S before[4], sum[4];
        __builtin_memcpy(before, old[k], sizeof(before));
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = TO::st(p.o.accumulate ? TO::ld(before[e]) + x[e] : x[e]);
        S *to = out + row * p.o.pitch + col;
        if (row < rows && col + 4 <= cols) {
          if constexpr (sizeof(S) == 4) {
            __builtin_nontemporal_store(f32x4_any{sum[0], sum[1], sum[2], sum[3]}, reinterpret_cast<f32x4_any *>(to));
          } else {
            u32x2_any v;
            __builtin_memcpy(&v, sum, sizeof(v));
            __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any *>(to));
          }
        } else if (row < rows) {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (col + e < cols) to[e] = sum[e];
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    return;
  }
  // (all loads before the first sum: 27.0 us one by one)
  uint32_t old[L::NBM][L::NBN][4][sizeof(S)] = {};           // four values each
  if (p.o.accumulate) {
#pragma unroll
    for (int i = 0; i < L::NBM; ++i)
#pragma unroll
      for (int j = 0; j < L::NBN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int64_t row = row0 + wr + 32 * i + lr, col = col0 + wc + 32 * j + 8 * g + 4 * lh;
          const S *from = out + row * p.o.pitch + col;
          if (row < rows && col + 4 <= cols) {
            __builtin_memcpy(old[i][j][g], from, sizeof(old[i][j][g]));
          } else if (row < rows) {
            S few[4] = {};
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (col + e < cols) few[e] = from[e];
            __builtin_memcpy(old[i][j][g], few, sizeof(few));
          }
        }
  }
#pragma unroll
  for (int i = 0; i < L::NBM; ++i) {
    const int64_t row = row0 + wr + 32 * i + lr;
    if (row >= rows) continue;
    S *const to = out + row * p.o.pitch;
#pragma unroll
    for (int j = 0; j < L::NBN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t col = col0 + wc + 32 * j + 8 * g + 4 * lh;
        S before[4], sum[4];
        __builtin_memcpy(before, old[i][j][g], sizeof(before));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = acc[j][i][4 * g + e];
          sum[e] = TO::st(p.o.accumulate ? TO::ld(before[e]) + x : x);
        }
        if (col + 4 <= cols) {
          __builtin_memcpy(to + col, sum, sizeof(sum));
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (col + e < cols) to[col + e] = sum[e];
        }
      }
  }
}

// out (+)= the sum of the parts of a contraction, in order; four columns per thread.
template <class TO>
__global__ void __launch_bounds__(256)
mx_join(const float *parts, int n_parts, int64_t part_stride, int64_t rows_all, int64_t m, int64_t n, int64_t pitch,
        MxOutput o) {
  using S = typename TO::S;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = at / (pitch / 4),
                col = (at - row * (pitch / 4)) * 4;
  if (row >= rows_all) return;
  const float *from = parts + row * pitch + col;
  float4 sum = *reinterpret_cast<const float4 *>(from);
#pragma unroll 4
  for (int k = 1; k < n_parts; ++k) {
    const float4 v = *reinterpret_cast<const float4 *>(from + k * part_stride);
    sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
  }
  const int64_t mat = row / m;
  S *to = static_cast<S *>(o.out) + mat * o.batch_stride + (row - mat * m) * o.pitch + col;
  const float x[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + e < n) to[e] = TO::st(o.accumulate ? TO::ld(to[e]) + x[e] : x[e]);
}

// Few rows of A, as when single tokens are answered: what counts is reading B
// once.  A workgroup takes 16 rows of B (16 x 16 x 128 MFMA, B's fragments as
// the instruction's rows) and its W waves share the contraction, their sums
// joined in LDS in order; a wave has eight steps of 128 columns in flight, 8
// KiB of codes.  MB: blocks of 16 rows of A.
// With QUANTIZE the workgroup quantises A itself, as mx_quantize would, which
// saves a launch, while the first loads of B are on their way.
constexpr int kThinRows = 32;               // of A
constexpr int kThinValues = 64 * 1024;      // of A that a workgroup quantises at most: 34 KiB of LDS

struct MxThin {
  MxMatrix a, b;                            // a: without codes where x is quantised here
  MxOutput o;
  const void *x;
  int64_t x_pitch, x_batch_stride;
};

template <class TX, class TO, int MB, int W, bool QUANTIZE>
__global__ void __launch_bounds__(64 * W) mx_thin(MxThin p) {
  constexpr int kSteps = 8;
  __shared__ __attribute__((aligned(16))) f32x4 sums[W][MB][64];
  __shared__ __attribute__((aligned(16))) uint8_t codes[QUANTIZE ? kThinValues / 2 + 16 * 16 : 16];
  __shared__ __attribute__((aligned(16))) uint32_t scales[QUANTIZE ? kThinValues / kMxGroup : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t blocks = (p.b.rows + 15) / 16, mat = blockIdx.x / blocks;
  const int64_t row0 = (blockIdx.x - mat * blocks) * 16;
  const int groups = static_cast<int>(p.b.groups()), m = static_cast<int>(p.a.rows);
  const int lr = lane & 15, chunk = lane >> 4;
  const int64_t n = row0 + lr;
  const bool real = n < p.b.rows;
  const uint8_t *bc = p.b.codes + (mat * p.b.rows + (real ? n : row0)) * (groups * 64) + chunk * 16;
  const uint8_t *bs = p.b.scales + ((mat * p.b.row_blocks() + n / 32) * groups * 32 + n % 32) * 4;
  const int per = (groups + W - 1) / W, begin = wave * per, end = min(begin + per, groups);

  uint4 fb[kSteps];
  uint32_t xb[kSteps];
  auto load = [&](int at) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      fb[i] = make_uint4(0, 0, 0, 0);
      xb[i] = 0;
      if (at + i < end && real) {
        fb[i] = *reinterpret_cast<const uint4 *>(bc + static_cast<int64_t>(at + i) * 64);
        xb[i] = *reinterpret_cast<const uint32_t *>(bs + static_cast<int64_t>(at + i) * 128);
      }
    }
  };
  load(begin);

  const int lds_pitch = groups * 64 + 16;     // (rows on different banks)
  if constexpr (QUANTIZE) {
    using S = typename TX::S;
    constexpr bool k16 = sizeof(S) == 2;
    const S *x = static_cast<const S *>(p.x) + mat * p.x_batch_stride;
    for (int u = tid; u < m * groups * 16; u += 64 * W) {
      const int row = u / (groups * 16), at = u - row * groups * 16;
      const int64_t col = static_cast<int64_t>(at) * 8;
      Octet<TX> v;
      v.load(x + row * p.x_pitch + col, static_cast<int>(min<int64_t>(8, p.b.cols - col)));
      uint32_t largest = v.largest();
      largest = max(largest, other_lane<1>(largest));
      largest = max(largest, other_lane<2>(largest));
      const uint32_t s = scale_byte(largest, false);
      uint32_t bits[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) bits[i] = k16 ? v.w[i / 2] >> (16 * (i & 1)) & 0xffff : v.w[k16 ? 0 : i];
      *reinterpret_cast<uint32_t *>(codes + row * lds_pitch + at * 4) = eight_codes<TX, false>(bits, nullptr, s);
      if ((at & 3) == 0) reinterpret_cast<uint8_t *>(scales)[row * groups * 4 + at / 4] = static_cast<uint8_t>(s);
    }
    __syncthreads();
  }

  f32x4 acc[MB];
#pragma unroll
  for (int j = 0; j < MB; ++j) acc[j] = f32x4{0, 0, 0, 0};
  for (int at = begin; at < end; at += kSteps) {
    if (at > begin) load(at);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (at + i >= end) break;
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const int row = 16 * j + lr;
        uint4 fa = make_uint4(0, 0, 0, 0);
        uint32_t xa = 0;
        if (row < m) {
          if constexpr (QUANTIZE) {
            fa = *reinterpret_cast<const uint4 *>(codes + row * lds_pitch + (at + i) * 64 + chunk * 16);
            xa = scales[row * groups + at + i];
          } else {
            fa = *reinterpret_cast<const uint4 *>(p.a.codes + (mat * m + row) * (static_cast<int64_t>(groups) * 64) +
                                                  static_cast<int64_t>(at + i) * 64 + chunk * 16);
            xa = *reinterpret_cast<const uint32_t *>(
                p.a.scales + (((mat * p.a.row_blocks() + row / 32) * groups + at + i) * 32 + row % 32) * 4);
          }
        }
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(fb[i]), fp4_operand(fa), acc[j], 4, 4, 0,
                                                                 xb[i] >> (8 * chunk), 0, xa >> (8 * chunk));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < MB; ++j) sums[wave][j][lane] = acc[j];
  __syncthreads();
  // thread: row lane % 16 of A's block, four rows of B from 4 (lane / 16)
  for (int k = tid; k < MB * 256; k += 64 * W) {
    const int row = k / 16, col = k % 16, j = row / 16, from = (col / 4) * 16 + row % 16;
    if (row >= m || row0 + col >= p.b.rows) continue;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += reinterpret_cast<const float *>(&sums[w][j][from])[col % 4];
    typename TO::S *to = static_cast<typename TO::S *>(p.o.out) + mat * p.o.batch_stride + row * p.o.pitch + row0 + col;
    *to = TO::st(p.o.accumulate ? TO::ld(*to) + sum : sum);
  }
}

template <class TX, class TO, int MB, bool QUANTIZE>
hipError_t run_thin(const MxThin &p, hipStream_t s) {
  // about 4096 waves, at most 16 to a workgroup (one row, 16 waves and four: 4096 x
  // 4096 4.6 and 6.3 us, 4096 x 16384 10.1 and 16.7, 8192 x 16384 20.1 and 22.4; where
  // a compute unit has more than one workgroup, between 256 and 512 of them, short
  // contractions lose: 8192 x 4096 7.4 and 7.3, 8192 x 2048 5.7 and 5.0; beyond all do:
  // 16384 x 4096 12.8 and 9.6)
  const int64_t grid = p.b.batch * ((p.b.rows + 15) / 16);
  if (grid <= 512 && p.b.groups() >= 16) mx_thin<TX, TO, MB, 16, QUANTIZE><<<dim3(grid), dim3(1024), 0, s>>>(p);
  else mx_thin<TX, TO, MB, 4, QUANTIZE><<<dim3(grid), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxInput &in, int64_t batch, int64_t rows, int64_t cols, const MxMatrix &by_rows,
                              const MxMatrix &by_columns, hipStream_t s) {
  MxQuantize p{in.x, in.pitch, in.batch_stride, in.noise, rows, cols, by_rows, by_columns,
               batch, static_cast<int>((rows + 127) / 128), static_cast<int>((cols + 127) / 128),
               batch * rows * cols * dtype_size(in.dtype) >= kLastLevelCache, 0};
  int64_t tiles = batch * p.tiles_r * p.tiles_c;
  if (tiles >= kDealtTiles && tiles <= kMaxDealt && std::min(p.tiles_r, p.tiles_c) >= 8) {
    p.dealt = 1;
    tiles = (batch * ((p.tiles_r + 1) / 2) * ((p.tiles_c + 1) / 2) + 7) / 8 * 32;
  }
  const bool narrow = in.dtype == DT_F32 && tiles < 512;
  if (narrow) p.tiles_c *= 2;
  return with_type(in.dtype, [&](auto t) {
    using T = decltype(t);
    return with_flag(in.noise != nullptr, [&](auto noise) {
      constexpr bool N = decltype(noise)::value;
      auto run = [&](auto wide) {
        constexpr int kCols = decltype(wide)::value;
        const dim3 grid(static_cast<unsigned>(tiles * (128 / kCols)));
        if (!by_columns.codes) mx_quantize<T, true, false, N, kCols><<<grid, dim3(256), 0, s>>>(p);
        else if (!by_rows.codes) mx_quantize<T, false, true, N, kCols><<<grid, dim3(256), 0, s>>>(p);
        else mx_quantize<T, true, true, N, kCols><<<grid, dim3(256), 0, s>>>(p);
        return hipGetLastError();
      };
      if constexpr (T::code == DT_F32) {
        if (narrow) return run(std::integral_constant<int, 64>{});
      }
      return run(std::integral_constant<int, 128>{});
    });
  });
}

hipError_t launch_mx_dequantize(const MxMatrix &q, void *out, int dtype, hipStream_t s) {
  const int tiles_r = static_cast<int>((q.rows + 63) / 64), tiles_c = static_cast<int>((q.cols + 255) / 256);
  const int64_t tiles = q.batch * tiles_r * tiles_c;
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    mx_dequantize<T><<<dim3(std::min(tiles, kTilesX), (tiles + kTilesX - 1) / kTilesX), dim3(256), 0, s>>>(q, static_cast<typename T::S *>(out), tiles_r, tiles_c);
    return hipGetLastError();
  });
}

// How a product runs that mx_thin does not take.
struct MxPlan {
  enum Tile { T256, T128, T64 } tile;
  int parts;                  // of the contraction
};

MxPlan mx_plan(int64_t batch, int64_t m, int64_t n, int64_t k) {
  auto tiles = [&](int64_t tm, int64_t tn) { return batch * ((m + tm - 1) / tm) * ((n + tn - 1) / tn); };
  // Few rows of A take a tile that wastes less of them, if it fills the GPU
  // (64 matrices of 48 x 7168 by 2048 x 7168: 109 us, against 118 with 256 x 256.
  // 48 x 4096 by 50257 x 4096, 197 tiles: 31.0 us, 32.2 with 256- and 32.1 with
  // 128-edge ones; 48 x 2048 by 63000 x 2048: 20.2, 21.9 and 21.3; 48 x 4096 by 32768 x
  // 4096, 128 tiles: 27.0, 28.1 and 18.5).
  if (m <= 64 && tiles(64, 256) >= 192) return {MxPlan::T64, 1};
  // Many tiles of 256 x 256 keep the GPU busy (k = 4096: 2048 x 6144 in 192 of them
  // 32.2 us, 36.4 with 128-edge ones; 4096 x 4096 in 256 39.6 and 47.9).  The bound
  // is on the safe side: 128 of them are 512 of the others, which fit at once (2048
  // x 4096: 28.7 and 26.4), 160 would gain already (2560 x 4096: 29.5 and 35.6), 272
  // start a second round that is nearly empty (4096 x 4352: 61.6 and 55.6).
  // (A grid holds fewer than 2^32 threads: of these tiles, 512 to one, half as
  // many as the calls let through of the smaller ones.)
  if (tiles(256, 256) >= 192 && tiles(256, 256) < int64_t(1) << 23) return {MxPlan::T256, 1};
  // Where tiles of 128 leave compute units idle, a long contraction may be cut
  // into parts.  A stage takes 0.27 us of a workgroup; joining the parts takes a
  // launch, 5 us, and their results written and read at about 5 TB/s.  (48 x
  // 16384 by 4096 x 16384: 41.5 us whole, 22.4 in 16 parts; 1500 x 5000 by 1500 x
  // 5000: 26 whole, 33 in three.)
  const int64_t t = tiles(128, 128), stages = (k + kMxGroup - 1) / kMxGroup;
  int parts = 1;
  double best = 0.27 * stages;
  for (int p = 2; p <= 16 && t * p <= 512 && p <= stages; p *= 2) {
    const double us = 0.27 * stages / p + 5.0 + static_cast<double>(p) * batch * m * n * 8.0 / 5e6;
    if (us < best) {
      best = us;
      parts = p;
    }
  }
  const int64_t each = (stages + parts - 1) / parts;       // (no part without stages)
  return {MxPlan::T128, parts == 1 ? 1 : static_cast<int>((stages + each - 1) / each)};
}

int64_t join_pitch(int64_t n) { return (n + 3) / 4 * 4; }

// Whether mx_thin takes a product: up to 16 rows of A, and up to kThinRows by a
// B of up to 2^25 values.  Beyond those its workgroups' reads of A cost more
// than the others' tiles waste (32 x 4096 by 4096 x 4096: 12.8 us, in tiles 16.7;
// 32 x 16384 by 16384 x 16384: 54 and 33.  16 x 8192 by 16384 x 8192: 23.3 and 24.0; 16 x
// 16384 by 16384 x 16384, the largest, 43.5 and 37.6).  (A grid holds 2^24 workgroups
// of 256 threads.)
bool thin(int64_t batch, int64_t m, int64_t n, int64_t k) {
  return m <= kThinRows && batch < (int64_t(1) << 24) / ((n + 15) / 16 + 1) &&
         (m <= 16 || k == 0 || batch * n <= (int64_t(1) << 25) / k);
}

// Whether the product quantises A: each of its workgroups of 16 rows of B does
// then, which costs more than the launch that it saves where rows and workgroups
// are many.  (us in the product and before it, captured, K = 4096, bf16:
//     rows of A by  1024         4096         16384        65536        131072
//     1             3.7   6.2    5.1   7.8    9.5  12.5    30   37      55   65
//     2             4.1   6.2    5.3   7.9    10.8 12.5    36   38      67   67
//     4             4.6   6.4    6.0   8.1    13.5 12.8    45   40      84   70
//     8             6.0   6.5    7.5   8.3    19.0 13.2    64   42      118  74
//     16            9.0   6.9    10.8  8.9    29.6 14.5    102  46      190  84
// Calls that are not captured pay the host for both launches, 11.5 us whatever the
// size: 16 by 4096 take 10.2 and 11.3, 8 x 8192 by 4096 x 8192 12.7 and 11.5, 12 x
// 2048 by 8192 x 2048 9.5 and 11.4.)
bool mx_linear_quantizes(int64_t batch, int64_t m, int64_t n, int64_t k) {
  const int64_t values = m * ((k + kMxGroup - 1) / kMxGroup) * kMxGroup;
  if (!thin(batch, m, n, k) || m > 16 || values > kThinValues) return false;
  return m == 1 || values * batch * ((n + 15) / 16) <= int64_t(1) << (m == 2 ? 25 : 24);
}

size_t mx_matmul_bytes(int64_t batch, int64_t m, int64_t n, int64_t k) {
  if (thin(batch, m, n, k)) return 0;
  const int parts = mx_plan(batch, m, n, k).parts;
  return parts > 1 ? static_cast<size_t>(parts) * batch * m * join_pitch(n) * 4 : 0;
}

hipError_t launch_mx_linear(const MxInput &in, int64_t m, const MxMatrix &w, const MxOutput &out, hipStream_t s) {
  const MxThin p{MxMatrix{nullptr, nullptr, w.batch, m, w.cols}, w, out, in.x, in.pitch, in.batch_stride};
  return with_type(in.dtype, [&](auto tx) {
    return with_type(out.dtype, [&](auto to) { return run_thin<decltype(tx), decltype(to), 1, true>(p, s); });
  });
}

template <class T, class L>
hipError_t run_gemm(const MxMatrix &a, const MxMatrix &b, const MxOutput &out, int parts, hipStream_t s) {
  MxGemm p{a, b, out, static_cast<int>((a.rows + L::TM - 1) / L::TM), static_cast<int>((b.rows + L::TN - 1) / L::TN), 1,
           parts, a.batch * out.batch_stride,
           static_cast<int64_t>(sizeof(typename T::S)) * a.batch * a.rows * b.rows >= kLastLevelCache};
  const int64_t tiles = a.batch * p.tiles_m * p.tiles_n * parts;
  // runs of up to 32 tiles, in whole runs per XCD
  const int64_t each = tiles / 8;
  for (int r = 32; r > 1; --r)
    if (each % r == 0 && each > 0) {
      p.run = r;
      break;
    }
  mx_gemm<T, L><<<dim3(tiles), dim3(L::THREADS), 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_mx_matmul(const MxMatrix &a, const MxMatrix &b, const MxOutput &out, void *workspace, hipStream_t s) {
  return with_type(out.dtype, [&](auto t) {
    using T = decltype(t);
    if (thin(a.batch, a.rows, b.rows, a.cols)) {
      const MxThin p{a, b, out, nullptr, 0, 0};
      return a.rows <= 16 ? run_thin<EF32, T, 1, false>(p, s) : run_thin<EF32, T, 2, false>(p, s);
    }
    const MxPlan plan = mx_plan(a.batch, a.rows, b.rows, a.cols);
    if (plan.tile == MxPlan::T64) return run_gemm<T, MxTile<64, 256, 1, 4, 3>>(a, b, out, 1, s);
    if (plan.tile == MxPlan::T256) return run_gemm<T, MxTile<256, 256, 4, 2, 4>>(a, b, out, 1, s);
    if (plan.parts == 1) return run_gemm<T, MxTile<128, 128, 2, 2, 4>>(a, b, out, 1, s);
    const int64_t pitch = join_pitch(b.rows);
    const MxOutput each{workspace, DT_F32, pitch, a.rows * pitch, false};
    const hipError_t e = run_gemm<EF32, MxTile<128, 128, 2, 2, 4>>(a, b, each, plan.parts, s);
    if (e != hipSuccess) return e;
    const int64_t rows = a.batch * a.rows;
    mx_join<T><<<dim3((rows * (pitch / 4) + 255) / 256), dim3(256), 0, s>>>(
        static_cast<const float *>(workspace), plan.parts, rows * pitch, rows, a.rows, b.rows, pitch, out);
    return hipGetLastError();
  });
}

}  // namespace gns
