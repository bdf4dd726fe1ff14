// Microscaled 4-bit floating point (MXFP4) on CDNA4: quantisation, its
// inverse, and the product of two quantised matrices.
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

// A thread per block of 32: elements along `along`, blocks of one line, lines
// `across` apart.  Also the blocks that only pad a line, and the scales of
// lines that only pad the last 32.
template <class T>
__global__ void __launch_bounds__(256)
mx_quantize_blocks(const typename T::S *x, int64_t sb, int64_t along, int64_t across, const uint8_t *noise,
                   int64_t noise_along, int64_t noise_across, int64_t batch, int64_t lines, int64_t length,
                   uint8_t *codes, uint8_t *scales) {
  const int64_t groups = (length + kMxGroup - 1) / kMxGroup, blocks = groups * 4;
  const int64_t line_blocks = (lines + 31) / 32;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= batch * line_blocks * 32 * blocks) return;
  const int64_t blk = at % blocks, line = at / blocks % (line_blocks * 32), b = at / blocks / (line_blocks * 32);
  uint8_t *scale_at = scales + (((b * line_blocks + line / 32) * groups + blk / 4) * 32 + line % 32) * 4 + blk % 4;
  if (line >= lines) {
    *scale_at = 0;
    return;
  }
  const typename T::S *src = x + b * sb + line * across;
  float v[32];
  uint32_t largest = 0;
  for (int i = 0; i < 32; ++i) {
    const int64_t k = blk * 32 + i;
    v[i] = k < length ? T::ld(src[k * along]) : 0.0f;
    largest = max(largest, __float_as_uint(v[i]) & 0x7fffffffu);
  }
  const uint32_t s = scale_byte(largest, noise != nullptr);
  uint32_t word[4] = {0, 0, 0, 0};
  if (s != 255) {
    for (int i = 0; i < 32; i += 2) {
      uint32_t pair;
      if (noise) {
        const uint8_t *r = noise + b * lines * length + line * noise_across;
        const int64_t k = blk * 32 + i;
        const uint32_t r0 = k < length ? r[k * noise_along] : 0, r1 = k + 1 < length ? r[(k + 1) * noise_along] : 0;
        pair = noisy_code(v[i], inverse_scale(s), r0) | noisy_code(v[i + 1], inverse_scale(s), r1) << 4;
      } else {
        pair = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[i], v[i + 1], scale_of(s), 0) & 0xff;
      }
      word[i / 8] |= pair << (4 * (i % 8));
    }
  }
  *reinterpret_cast<uint4 *>(codes + ((b * lines + line) * groups * 64) + blk * 16) =
      make_uint4(word[0], word[1], word[2], word[3]);
  *scale_at = static_cast<uint8_t>(s);
}

template <class T>
__global__ void __launch_bounds__(256) mx_dequantize_values(MxMatrix q, typename T::S *out) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t groups = q.groups();
  if (at >= q.batch * q.rows * groups * 4) return;
  const int64_t blk = at % (groups * 4), row = at / (groups * 4) % q.rows, b = at / (groups * 4) / q.rows;
  const uint4 w = *reinterpret_cast<const uint4 *>(q.codes + (b * q.rows + row) * q.pitch() + blk * 16);
  const uint32_t s = q.scales[(((b * q.row_blocks() + row / 32) * groups + blk / 4) * 32 + row % 32) * 4 + blk % 4];
  const uint32_t word[4] = {w.x, w.y, w.z, w.w};
  typename T::S *dst = out + (b * q.rows + row) * q.cols;
  for (int i = 0; i < 32; ++i) {
    const int64_t k = blk * 32 + i;
    if (k >= q.cols) break;
    const uint32_t c = word[i / 8] >> (4 * (i % 8)) & 15;
    const uint32_t m = c & 7;
    const float t = m < 4 ? 0.5f * m : m < 6 ? static_cast<float>(m) - 2.0f : 2.0f * m - 8.0f;
    const float val = s == 255 ? __uint_as_float(0x7fc00000u) : (c & 8 ? -t : t) * scale_of(s);
    dst[k] = T::st(val);
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

__device__ __forceinline__ i32x8 fp4_operand(uint4 v) {
  return i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
}

// C = A B^T in tiles of TILE x TILE, with 8 waves (256) in a 4 x 2 grid of 64 x
// 128 wave tiles or 4 waves (128) in a 2 x 2 grid of 64 x 64.  An MFMA
// multiplies 32 x 64 codes by 32 x 64: lane l holds one block of 32 codes of
// row l % 32 of either factor, 16 bytes, and its scale.  A stage of the
// contraction is 128 columns: 64 bytes of codes of every row, as four 16-byte
// chunks, and one word of scales of every row.  Both come from HBM or L2
// straight into LDS (LDS-DMA) into a ring of four stages.  The fragments of B
// are the instruction's rows, so that a lane's accumulators are runs of four
// consecutive columns of C.
template <int TILE>
struct MxTile {
  static constexpr int WGM = TILE == 256 ? 4 : 2, WGN = 2;       // waves along rows, columns
  static constexpr int NW = WGM * WGN, THREADS = 64 * NW;
  static constexpr int WTM = TILE / WGM, WTN = TILE / WGN;
  static constexpr int NBM = WTM / 32, NBN = WTN / 32;           // 32 x 32 blocks of a wave
  static constexpr int CODES = TILE * 64;                        // bytes of one factor's codes in a stage
  static constexpr int PIECES = TILE / 32;                       // 128-byte pieces of one factor's scales
  static constexpr int STAGE = 2 * CODES + 2 * PIECES * 128;
  static constexpr int STAGES = 4;
  static constexpr int CODE_LOADS = TILE / 16 / NW;              // of 1 KiB, per wave and factor
  static constexpr int LOADS = 2 * CODE_LOADS + 1;               // of a wave per stage
  static_assert(CODE_LOADS * NW * 16 == TILE && 2 * NW == 2 * PIECES, "the waves' loads cover a stage");
  static_assert(STAGES * STAGE <= 160 * 1024, "LDS");
};

struct MxGemm {
  MxMatrix a, b;
  MxOutput o;
  int tiles_m, tiles_n;
  int run;             // consecutive tiles dealt to one XCD
  int parts;           // of the contraction
  int64_t part_stride; // elements of o from one part's results to the next's
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

template <class TO, int TILE>
__global__ void __launch_bounds__((MxTile<TILE>::THREADS)) mx_gemm(MxGemm p) {
  using L = MxTile<TILE>;
  using S = typename TO::S;
  __shared__ __attribute__((aligned(16))) unsigned char lds[L::STAGES * L::STAGE];

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
  auto panel = [&](const MxMatrix &q, int tile, i32x4 *codes, i32x4 *scales) {
    const int64_t row = static_cast<int64_t>(tile) * TILE, blocks = q.row_blocks();
    *codes = buffer_of(q.codes + (mat * q.rows + row) * pitch, min<int64_t>(TILE, q.rows - row) * pitch);
    *scales = buffer_of(q.scales + (mat * blocks + row / 32) * groups * 128,
                        min<int64_t>(L::PIECES, blocks - row / 32) * groups * 128);
  };
  i32x4 ca, cb, sa, sb;
  panel(p.a, ti, &ca, &sa);
  panel(p.b, tj, &cb, &sb);
  const uint32_t lds_base =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char *)(lds)));

  // Lane l of a load of codes fills 16 bytes of row l / 4 of its 16 rows, at
  // chunk l % 4; a load of scales fills two pieces, a word per lane.
  const int dma_row = lane >> 2;
  const int code_at = dma_row * pitch + ((lane & 3) ^ swizzle(dma_row)) * 16;
  const int scale_at = lh * groups * 128 + lr * 4;
  const bool scales_of_a = wave < L::NW / 2;
  const int scale_piece = 2 * (scales_of_a ? wave : wave - L::NW / 2);
  const i32x4 sx = scales_of_a ? sa : sb;
  auto fetch = [&](int stage) {
    // stages past the last one go through an empty range: every stage has the
    // same number of loads, and these fetch nothing
    const bool live = stage < stages;
    const int at = first + (live ? stage : 0);
    const uint32_t to = lds_base + static_cast<uint32_t>((stage % L::STAGES) * L::STAGE);
    i32x4 a = ca, b = cb, x = sx;
    if (!live) a[2] = b[2] = x[2] = 0;
#pragma unroll
    for (int q = 0; q < L::CODE_LOADS; ++q) {
      const int blk = wave + q * L::NW, from = blk * 16 * pitch + at * 64;
      asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to + blk * 1024), "v"(code_at),
                   "s"(a), "s"(from)
                   : "memory", "m0");
      asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to + L::CODES + blk * 1024),
                   "v"(code_at), "s"(b), "s"(from)
                   : "memory", "m0");
    }
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(to + 2 * L::CODES + wave * 256),
                 "v"(scale_at), "s"(x), "s"(scale_piece * groups * 128 + at * 128)
                 : "memory", "m0");
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
        fb[s][j] = *reinterpret_cast<const uint4 *>(at + L::CODES + (wc + 32 * j + lr) * 64 + chunk);
    }
    const unsigned char *words = at + 2 * L::CODES + lr * 4;
#pragma unroll
    for (int i = 0; i < L::NBM; ++i)
      xa[i] = *reinterpret_cast<const uint32_t *>(words + (wr / 32 + i) * 128) >> (8 * lh);
#pragma unroll
    for (int j = 0; j < L::NBN; ++j)
      xb[j] = *reinterpret_cast<const uint32_t *>(words + (L::PIECES + wc / 32 + j) * 128) >> (8 * lh);
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
  for (int i = 0; i < L::STAGES - 1; ++i) fetch(i);
  constexpr int kWait = L::LOADS * (L::STAGES - 2);      // this wave's loads of later stages
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kWait) : "memory");
  __syncthreads();
  if constexpr (L::NW == 8) {
    // The two waves of a SIMD are one barrier apart: one multiplies while the
    // other reads.  Stage i + 3 goes to the place of stage i - 1, which both
    // have finished reading.
    const bool second = wave >= 4;
    if (second) __syncthreads();
    for (int i = 0; i < stages; ++i) {
      read(i % L::STAGES);
      fetch(i + L::STAGES - 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kWait) : "memory");
      __syncthreads();
      __builtin_amdgcn_s_setprio(1);
      multiply();
      __builtin_amdgcn_s_setprio(0);
      __syncthreads();
    }
    if (!second) __syncthreads();
  } else {
    for (int i = 0; i < stages; ++i) {
      read(i % L::STAGES);
      fetch(i + L::STAGES - 1);
      multiply();
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kWait) : "memory");
      __syncthreads();
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // Results go through LDS, so that the workgroup stores whole rows, 16 bytes
  // per thread.  Rounded first where they are stored as they are; as fp32
  // where they are added to what is there, half a tile of 256 at a time.
  S *const out = static_cast<S *>(p.o.out) + part * p.part_stride + mat * p.o.batch_stride;
  const int64_t row0 = static_cast<int64_t>(ti) * TILE, col0 = static_cast<int64_t>(tj) * TILE;
  const int64_t rows = p.a.rows, cols = p.b.rows;
  const bool whole_words = p.o.pitch * sizeof(S) % 16 == 0 && p.o.batch_stride * sizeof(S) % 16 == 0 &&
                           reinterpret_cast<uintptr_t>(p.o.out) % 16 == 0;
  constexpr int kPer = 16 / sizeof(S);                   // elements of 16 bytes
  if constexpr (sizeof(S) == 2) {
    if (!p.o.accumulate) {
      constexpr int kPitch = TILE + 8;
      static_assert(TILE * kPitch * 2 <= L::STAGES * L::STAGE, "LDS");
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
      for (int k = tid; k < TILE * TILE / kPer; k += L::THREADS) {
        const int r = k / (TILE / kPer), c = k % (TILE / kPer) * kPer;
        const int64_t row = row0 + r, col = col0 + c;
        if (row >= rows || col >= cols) continue;
        const S *from = staged + r * kPitch + c;
        S *to = out + row * p.o.pitch + col;
        if (whole_words && col + kPer <= cols) {
          *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
        } else {
          for (int e = 0; e < kPer && col + e < cols; ++e) to[e] = from[e];
        }
      }
      return;
    }
  }
  constexpr int kHalves = TILE / 128, kPitch = TILE + 4;
  static_assert(128 * kPitch * 4 <= L::STAGES * L::STAGE, "LDS");
  float *const staged = reinterpret_cast<float *>(lds);
  for (int half = 0; half < kHalves; ++half) {
    __syncthreads();
    if (wr / 128 == half) {
#pragma unroll
      for (int j = 0; j < L::NBN; ++j)
#pragma unroll
        for (int i = 0; i < L::NBM; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<float4 *>(staged + (wr % 128 + 32 * i + lr) * kPitch + wc + 32 * j + 8 * g + 4 * lh) =
                make_float4(acc[j][i][4 * g], acc[j][i][4 * g + 1], acc[j][i][4 * g + 2], acc[j][i][4 * g + 3]);
    }
    __syncthreads();
    for (int k = tid; k < 128 * TILE / 4; k += L::THREADS) {
      const int r = k / (TILE / 4), c = k % (TILE / 4) * 4;
      const int64_t row = row0 + 128 * half + r, col = col0 + c;
      if (row >= rows || col >= cols) continue;
      const float4 v = *reinterpret_cast<const float4 *>(staged + r * kPitch + c);
      S *to = out + row * p.o.pitch + col;
      if (sizeof(S) == 4 && whole_words && col + 4 <= cols) {
        float4 *at = reinterpret_cast<float4 *>(to);
        float4 sum = v;
        if (p.o.accumulate) {
          const float4 old = *at;
          sum = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
        }
        *at = sum;
      } else {
        const float e4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < cols) to[e] = TO::st(p.o.accumulate ? TO::ld(to[e]) + e4[e] : e4[e]);
      }
    }
  }
}

}  // namespace

hipError_t launch_mx_quantize(const MxInput &in, int64_t batch, int64_t rows, int64_t cols, const MxMatrix &by_rows,
                              const MxMatrix &by_columns, hipStream_t s) {
  return with_type(in.dtype, [&](auto t) {
    using T = decltype(t);
    const typename T::S *x = static_cast<const typename T::S *>(in.x);
    auto run = [&](const MxMatrix &q, int64_t along, int64_t across, int64_t na, int64_t nc) {
      const int64_t n = batch * q.row_blocks() * 32 * q.groups() * 4;
      mx_quantize_blocks<T><<<dim3((n + 255) / 256), dim3(256), 0, s>>>(x, in.batch_stride, along, across, in.noise, na,
                                                                       nc, batch, q.rows, q.cols, q.codes, q.scales);
    };
    if (by_rows.codes) run(by_rows, 1, in.pitch, 1, cols);
    if (by_columns.codes) run(by_columns, in.pitch, 1, cols, 1);
    return hipGetLastError();
  });
}

hipError_t launch_mx_dequantize(const MxMatrix &q, void *out, int dtype, hipStream_t s) {
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const int64_t n = q.batch * q.rows * q.groups() * 4;
    mx_dequantize_values<T><<<dim3((n + 255) / 256), dim3(256), 0, s>>>(q, static_cast<typename T::S *>(out));
    return hipGetLastError();
  });
}

size_t mx_matmul_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx_matmul(const MxMatrix &a, const MxMatrix &b, const MxOutput &out, void *, hipStream_t s) {
  return with_type(out.dtype, [&](auto t) {
    using T = decltype(t);
    auto run = [&](auto tile) {
      constexpr int TILE = decltype(tile)::value;
      MxGemm p{a, b, out, static_cast<int>((a.rows + TILE - 1) / TILE), static_cast<int>((b.rows + TILE - 1) / TILE),
               1, 1, 0};
      const int64_t tiles = a.batch * p.tiles_m * p.tiles_n;
      // runs of up to 32 tiles, in whole runs per XCD
      const int64_t each = tiles / 8;
      for (int r = 32; r > 1; --r)
        if (each % r == 0 && each > 0) {
          p.run = r;
          break;
        }
      mx_gemm<T, TILE><<<dim3(tiles), dim3(MxTile<TILE>::THREADS), 0, s>>>(p);
      return hipGetLastError();
    };
    const int64_t big = a.batch * ((a.rows + 255) / 256) * ((b.rows + 255) / 256);
    return big >= 192 ? run(std::integral_constant<int, 256>{}) : run(std::integral_constant<int, 128>{});
  });
}

}  // namespace gns
