// Device kernels over lists of tensors: global norm, clipping and AdamW.
//
// A list's table (ListEntry, ListChunk) lies in device memory; every kernel
// runs one workgroup per chunk of one entry.  All of them are bound by HBM:
// a handful of operations per element against 2 to 28 bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gns_elem.h"
#include "gns_kernels.h"

namespace gns {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_elem(const void *p, int64_t i, int dtype) {
  if (dtype == DT_F32) return static_cast<const float *>(p)[i];
  const uint16_t h = static_cast<const uint16_t *>(p)[i];
  return dtype == DT_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
}

__device__ __forceinline__ void store_elem(void *p, int64_t i, int dtype, float v) {
  if (dtype == DT_F32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = dtype == DT_BF16 ? f32_to_bf16(v) : f32_to_f16(v);
}

// Calls f(row, column) for every element of chunk c that this thread has.
template <class F>
__device__ __forceinline__ void each_element(const ListEntry &e, uint32_t index, int64_t chunk_units, F f) {
  const int64_t u0 = static_cast<int64_t>(index) * chunk_units;
  const int64_t u1 = u0 + chunk_units < e.units ? u0 + chunk_units : e.units;
  for (int64_t u = u0 + threadIdx.x; u < u1; u += kThreads) {
    const int64_t row = u / e.per_row;
    const int64_t c0 = (u - row * e.per_row) * kListUnit;
    const int64_t c1 = c0 + kListUnit < e.cols ? c0 + kListUnit : e.cols;
    for (int64_t c = c0; c < c1; ++c) f(row, c);
  }
}

// Sum (or maximum) over a workgroup of up to 16 waves, in a fixed order; the
// result is thread 0's.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[16];
  for (int off = 32; off > 0; off >>= 1) x += __shfl_down(x, off, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0)
    for (unsigned w = 1; w < (blockDim.x + 63) / 64; ++w) x += part[w];
  return x;
}
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
  __shared__ uint32_t part[16];
  for (int off = 32; off > 0; off >>= 1) x = max(x, static_cast<uint32_t>(__shfl_down(x, off, 64)));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0)
    for (unsigned w = 1; w < (blockDim.x + 63) / 64; ++w) x = max(x, part[w]);
  return x;
}

// The magnitudes of floats order as their bits without the sign do, with NaN
// above infinity: an integer maximum keeps a NaN.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <bool MAX>
__global__ void __launch_bounds__(kThreads) list_partials(ListView v, uint64_t *partials) {
  const ListChunk ch = v.chunks[blockIdx.x];
  const ListEntry &e = v.entries[ch.entry];
  if constexpr (MAX) {
    uint32_t top = 0;
    each_element(e, ch.index, v.chunk_units, [&](int64_t r, int64_t c) {
      top = max(top, magnitude(load_elem(e.data[0], r * e.pitch[0] + c, e.dtype[0])));
    });
    top = block_max(top);
    if (threadIdx.x == 0) partials[blockIdx.x] = top;
  } else {
    double acc = 0.0;
    each_element(e, ch.index, v.chunk_units, [&](int64_t r, int64_t c) {
      const double x = load_elem(e.data[0], r * e.pitch[0] + c, e.dtype[0]);
      acc += x * x;
    });
    acc = block_sum(acc);
    if (threadIdx.x == 0) partials[blockIdx.x] = __double_as_longlong(acc);
  }
}

// Norm of chunks [first, first + n) (thread 0's).
template <bool MAX>
__device__ __forceinline__ double norm_of(const uint64_t *partials, int64_t first, int64_t n) {
  if constexpr (MAX) {
    uint32_t top = 0;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) top = max(top, static_cast<uint32_t>(partials[first + i]));
    return __uint_as_float(block_max(top));
  } else {
    double acc = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) acc += __longlong_as_double(partials[first + i]);
    return sqrt(block_sum(acc));
  }
}

// Block 0: the norm of everything and the clip factor; block 1 + i: entry i's.
template <bool MAX>
__global__ void __launch_bounds__(kThreads)
list_finish(ListView v, const uint64_t *partials, const float *inv_scale, double max_norm, double eps,
            float *result, float *tensor_norms) {
  const double s = inv_scale ? static_cast<double>(*inv_scale) : 1.0;
  if (blockIdx.x == 0) {
    const double norm = norm_of<MAX>(partials, 0, v.n_chunks) * s;
    if (threadIdx.x == 0) {
      const float n32 = static_cast<float>(norm);
      const double ratio = max_norm / (norm + eps);
      result[0] = n32;
      result[1] = isfinite(norm) ? static_cast<float>(s * (ratio < 1.0 ? ratio : 1.0)) : __builtin_nanf("");
    }
  } else {
    const ListEntry &e = v.entries[blockIdx.x - 1];
    const double norm = norm_of<MAX>(partials, e.first_chunk, e.chunks) * s;
    if (threadIdx.x == 0) tensor_norms[blockIdx.x - 1] = static_cast<float>(norm);
  }
}

__global__ void __launch_bounds__(kThreads) list_scale(ListView v, int dst, const float *factor) {
  const float f = *factor;
  if (!isfinite(f) || (dst == 0 && f == 1.0f)) return;
  const ListChunk ch = v.chunks[blockIdx.x];
  const ListEntry &e = v.entries[ch.entry];
  each_element(e, ch.index, v.chunk_units, [&](int64_t r, int64_t c) {
    const float x = load_elem(e.data[0], r * e.pitch[0] + c, e.dtype[0]);
    store_elem(e.data[dst], r * e.pitch[dst] + c, e.dtype[dst], x * f);
  });
}

__global__ void __launch_bounds__(kThreads)
list_adamw(ListView v, bool copy, AdamwScalars h, const float *grad_scale) {
  const float f = grad_scale ? *grad_scale : 1.0f;
  if (!isfinite(f)) return;
  const ListChunk ch = v.chunks[blockIdx.x];
  const ListEntry &e = v.entries[ch.entry];
  const double eta = h.lr * e.lr_scale;
  const float decay = static_cast<float>(1.0 - eta * (h.weight_decay * e.wd_scale));
  const float rate = static_cast<float>(eta / h.bias1);
  each_element(e, ch.index, v.chunk_units, [&](int64_t r, int64_t c) {
    const float g = f * load_elem(e.data[0], r * e.pitch[0] + c, e.dtype[0]);
    float *p = static_cast<float *>(e.data[1]) + r * e.pitch[1] + c;
    float *m = static_cast<float *>(e.data[2]) + r * e.pitch[2] + c;
    float *s = static_cast<float *>(e.data[3]) + r * e.pitch[3] + c;
    const float m1 = fmaf(h.beta1, *m, h.one_minus_beta1 * g);
    const float s1 = fmaf(h.beta2, *s, h.one_minus_beta2 * (g * g));
    const float p1 = fmaf(-rate, m1 / fmaf(sqrtf(s1), h.inv_sqrt_bias2, h.eps), decay * *p);
    *m = m1;
    *s = s1;
    *p = p1;
    if (copy) store_elem(e.data[4], r * e.pitch[4] + c, e.dtype[4], p1);
  });
}

}  // namespace

hipError_t launch_list_partials(const ListView &v, bool max, uint64_t *partials, hipStream_t s) {
  if (v.n_chunks == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(v.n_chunks));
  if (max) list_partials<true><<<grid, kThreads, 0, s>>>(v, partials);
  else list_partials<false><<<grid, kThreads, 0, s>>>(v, partials);
  return hipGetLastError();
}

hipError_t launch_list_finish(const ListView &v, bool max, const uint64_t *partials, const float *inv_scale,
                              double max_norm, double eps, float *result, float *tensor_norms, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(tensor_norms ? 1 + v.count : 1));
  if (max) list_finish<true><<<grid, kThreads, 0, s>>>(v, partials, inv_scale, max_norm, eps, result, tensor_norms);
  else list_finish<false><<<grid, kThreads, 0, s>>>(v, partials, inv_scale, max_norm, eps, result, tensor_norms);
  return hipGetLastError();
}

hipError_t launch_list_scale(const ListView &v, int dst, const float *factor, hipStream_t s) {
  if (v.n_chunks == 0) return hipSuccess;
  list_scale<<<dim3(static_cast<unsigned>(v.n_chunks)), kThreads, 0, s>>>(v, dst, factor);
  return hipGetLastError();
}

hipError_t launch_list_adamw(const ListView &v, bool copy, const AdamwScalars &h, const float *grad_scale,
                             hipStream_t s) {
  if (v.n_chunks == 0) return hipSuccess;
  list_adamw<<<dim3(static_cast<unsigned>(v.n_chunks)), kThreads, 0, s>>>(v, copy, h, grad_scale);
  return hipGetLastError();
}

}  // namespace gns
