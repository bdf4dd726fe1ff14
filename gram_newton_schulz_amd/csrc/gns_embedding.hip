// Token embedding and its gradient.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gns_elem.h"
#include "gns_kernels.h"

namespace gns {
namespace {

template <class F>
hipError_t with_type(int dtype, F &&f) {
  if (dtype == DT_F32) return f(EF32{});
  if (dtype == DT_BF16) return f(EBF16{});
  return f(EF16{});
}

// A product as fp32 has it.  (Left to itself the compiler rounds a product that
// goes into fp16 once, from its exact value.)
__device__ __forceinline__ float times(float a, float b) {
  float p = a * b;
  asm("" : "+v"(p));
  return p;
}

struct Tokens {
  const void *at;
  int bits;
  __device__ int64_t operator[](int64_t i) const {
    return bits == 32 ? static_cast<const int32_t *>(at)[i] : static_cast<const int64_t *>(at)[i];
  }
};

// A workgroup per token.
template <class TW, class TO>
__global__ void __launch_bounds__(256)
embedding_rows(Tokens tokens, const typename TW::S *weight, int64_t vocab, int64_t width, int64_t weight_pitch,
               float scale, typename TO::S *out, int64_t out_pitch) {
  const int64_t i = blockIdx.x, t = tokens[i];
  const bool real = t >= 0 && t < vocab;
  for (int64_t c = threadIdx.x; c < width; c += 256)
    out[i * out_pitch + c] = TO::st(real ? times(TW::ld(weight[t * weight_pitch + c]), scale) : 0.0f);
}

// A workgroup per row of the table, which looks through all tokens.
template <class TG, class TW>
__global__ void __launch_bounds__(256)
embedding_sums(Tokens tokens, int64_t count, const typename TG::S *grad, int64_t grad_pitch, int64_t width,
               float scale, typename TW::S *grad_weight, int64_t weight_pitch, bool accumulate) {
  __shared__ int64_t found[256];
  const int64_t v = blockIdx.x;
  for (int64_t c0 = 0; c0 < width; c0 += 256) {
    const int64_t c = c0 + threadIdx.x;
    float sum = 0.0f;
    bool any = false;
    for (int64_t i0 = 0; i0 < count; i0 += 256) {
      const int64_t i = i0 + threadIdx.x;
      found[threadIdx.x] = i < count && tokens[i] == v ? i : -1;
      __syncthreads();
      for (int k = 0; k < 256; ++k) {
        if (found[k] < 0) continue;
        any = true;
        if (c < width) sum += TG::ld(grad[found[k] * grad_pitch + c]);
      }
      __syncthreads();
    }
    if (c < width && (any || !accumulate)) {
      typename TW::S *p = grad_weight + v * weight_pitch + c;
      *p = TW::st(accumulate ? TW::ld(*p) + times(scale, sum) : times(scale, sum));
    }
  }
}

}  // namespace

hipError_t launch_embedding(const void *tokens, int token_bits, int64_t count, const TokenRows &weight, int64_t vocab,
                            int64_t width, float scale, const TokenRows &out, hipStream_t s) {
  return with_type(weight.dtype, [&](auto tw) {
    return with_type(out.dtype, [&](auto to) {
      using TW = decltype(tw);
      using TO = decltype(to);
      embedding_rows<TW, TO><<<dim3(count), dim3(256), 0, s>>>(
          Tokens{tokens, token_bits}, static_cast<const typename TW::S *>(weight.data), vocab, width, weight.pitch,
          scale, static_cast<typename TO::S *>(out.data), out.pitch);
      return hipGetLastError();
    });
  });
}

size_t embedding_grad_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_embedding_grad(const void *tokens, int token_bits, int64_t count, const TokenRows &grad,
                                 int64_t vocab, int64_t width, float scale, const TokenRows &grad_weight,
                                 bool accumulate, void *, hipStream_t s) {
  return with_type(grad.dtype, [&](auto tg) {
    return with_type(grad_weight.dtype, [&](auto tw) {
      using TG = decltype(tg);
      using TW = decltype(tw);
      embedding_sums<TG, TW><<<dim3(vocab), dim3(256), 0, s>>>(
          Tokens{tokens, token_bits}, count, static_cast<const typename TG::S *>(grad.data), grad.pitch, width, scale,
          static_cast<typename TW::S *>(grad_weight.data), grad_weight.pitch, accumulate);
      return hipGetLastError();
    });
  });
}

}  // namespace gns
