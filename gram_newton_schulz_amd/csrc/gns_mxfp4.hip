// Microscaled 4-bit floating point (MXFP4) on CDNA4: quantisation, its
// inverse, and the product of two quantised matrices.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gns_elem.h"
#include "gns_kernels.h"

namespace gns {
namespace {

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

// One wave per 32 x 32 tile.  Lane l of the MFMA holds row l % 32 of either
// factor, 32 consecutive elements (one block) from k + 32 (l / 32), and their
// scale.
template <class TO>
__global__ void __launch_bounds__(64) mx_matmul_wave(MxMatrix a, MxMatrix b, MxOutput o) {
  const int64_t tm = (a.rows + 31) / 32, tn = (b.rows + 31) / 32;
  const int64_t tile = blockIdx.x;
  const int64_t tj = tile % tn, ti = tile / tn % tm, mat = tile / tn / tm;
  const int lane = threadIdx.x, lr = lane & 31, lh = lane >> 5;
  const int64_t i = ti * 32 + lr, j = tj * 32 + lr, groups = a.groups();
  const uint8_t *ca = a.codes + (mat * a.rows + i) * a.pitch(), *cb = b.codes + (mat * b.rows + j) * b.pitch();
  const uint8_t *sa = a.scales + ((mat * a.row_blocks() + ti) * groups * 32 + lr) * 4;
  const uint8_t *sb = b.scales + ((mat * b.row_blocks() + tj) * groups * 32 + lr) * 4;
  f32x16 acc{};
  for (int64_t blk = lh; blk < groups * 4; blk += 2) {
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    if (i < a.rows) va = *reinterpret_cast<const uint4 *>(ca + blk * 16);
    if (j < b.rows) vb = *reinterpret_cast<const uint4 *>(cb + blk * 16);
    const int xa = sa[blk / 4 * 128 + blk % 4], xb = sb[blk / 4 * 128 + blk % 4];
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(va), fp4_operand(vb), acc, 4, 4, 0, xa, 0, xb);
  }
  if (j >= b.rows) return;
  typename TO::S *out = static_cast<typename TO::S *>(o.out) + mat * o.batch_stride + j;
  for (int r = 0; r < 16; ++r) {
    const int64_t row = ti * 32 + 8 * (r / 4) + 4 * lh + r % 4;
    if (row >= a.rows) continue;
    typename TO::S *p = out + row * o.pitch;
    *p = TO::st(o.accumulate ? TO::ld(*p) + acc[r] : acc[r]);
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
    const int64_t tiles = a.batch * a.row_blocks() * b.row_blocks();
    mx_matmul_wave<T><<<dim3(tiles), dim3(64), 0, s>>>(a, b, out);
    return hipGetLastError();
  });
}

}  // namespace gns
