// Device kernels over lists of tensors: global norm, clipping and AdamW.
//
// A list's table (ListEntry, ListChunk) lies in device memory; every kernel
// runs one workgroup per chunk of one entry.  All of them are bound by HBM:
// a handful of operations per element against 2 to 28 bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gns_elem.h"
#include "gns_kernels.h"

namespace gns {

namespace {

constexpr int kThreads = 256;

// V consecutive elements as they lie in memory.  The addresses are aligned to
// the element only: gfx950 loads and stores 8 and 16 bytes from any address,
// and a wave's accesses are consecutive, so a misaligned tensor costs one more
// cache line per wave and instruction, not another path.
template <int BYTES> struct Raw;
template <> struct Raw<8> {
  typedef uint32_t T __attribute__((ext_vector_type(2), aligned(2)));
  T v[1];
};
template <> struct Raw<16> {
  typedef uint32_t T __attribute__((ext_vector_type(4), aligned(2)));
  T v[1];
};
template <> struct Raw<32> {
  typedef uint32_t T __attribute__((ext_vector_type(4), aligned(2)));
  T v[2];
};
template <class E, int V> using RawOf = Raw<V * static_cast<int>(sizeof(typename E::S))>;

// A tensor's address comes out of the table, where the compiler does not see
// that it is global memory: said here, so that these are no flat accesses.
#define GNS_GLOBAL __attribute__((address_space(1)))
template <class S> __device__ __forceinline__ S ld_one(const S *p) { return *(const GNS_GLOBAL S *)p; }
template <class S> __device__ __forceinline__ void st_one(S *p, S v) { *(GNS_GLOBAL S *)p = v; }

template <class E, int V>
__device__ __forceinline__ RawOf<E, V> ld_raw(const typename E::S *p) {
  using R = RawOf<E, V>;
  R r;
  const GNS_GLOBAL typename R::T *q = (const GNS_GLOBAL typename R::T *)p;
#pragma unroll
  for (unsigned i = 0; i < sizeof(R) / sizeof(typename R::T); ++i) r.v[i] = q[i];
  return r;
}
template <class E, int V>
__device__ __forceinline__ void st_raw(typename E::S *p, const RawOf<E, V> &r) {
  using R = RawOf<E, V>;
  GNS_GLOBAL typename R::T *q = (GNS_GLOBAL typename R::T *)p;
#pragma unroll
  for (unsigned i = 0; i < sizeof(R) / sizeof(typename R::T); ++i) q[i] = r.v[i];
}
template <class R> __device__ __forceinline__ uint32_t word(const R &r, int i) {
  constexpr int W = sizeof(typename R::T) / 4;
  return r.v[i / W][i % W];
}
template <class E, int V>
__device__ __forceinline__ void decode(const RawOf<E, V> &r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (E::code == DT_F32) x[i] = __uint_as_float(word(r, i));
    else x[i] = E::ld(static_cast<uint16_t>(word(r, i / 2) >> (16 * (i & 1))));
  }
}
template <class E, int V>
__device__ __forceinline__ RawOf<E, V> encode(const float (&x)[V]) {
  RawOf<E, V> r;
  constexpr int W = sizeof(typename RawOf<E, V>::T) / 4;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(r)) / 4; ++i) {
    if constexpr (E::code == DT_F32) r.v[i / W][i % W] = __float_as_uint(x[i]);
    else r.v[i / W][i % W] = E::st2(x[2 * i], x[2 * i + 1]);
  }
  return r;
}

// Calls f with a value of the element type that a table names.
template <class F>
__device__ __forceinline__ void with_type(int dtype, F f) {
  if (dtype == DT_BF16) f(EBF16{});
  else if (dtype == DT_F16) f(EF16{});
  else f(EF32{});
}

// A chunk of an entry.  Dense: `n` elements from element `first` of the only
// row.  Otherwise units [u0, u0 + n_units), found row by row.
struct Span {
  int64_t first;
  int n;
  bool dense;
};
__device__ __forceinline__ Span span_of(const ListEntry &e, uint32_t index, int64_t chunk_units) {
  Span s;
  const int64_t u0 = static_cast<int64_t>(index) * chunk_units;
  s.dense = e.units == e.per_row;
  const int64_t left = s.dense ? e.cols - u0 * kListUnit : e.units - u0;
  const int64_t most = s.dense ? chunk_units * kListUnit : chunk_units;
  s.first = s.dense ? u0 * kListUnit : u0;
  s.n = static_cast<int>(left < most ? left : most);
  return s;
}

// A dense chunk by this thread: whole(i) takes the V elements from i (called
// for U pieces at a time by block(i, stride), which can issue all their loads
// first), and one(i) each element of the last, partial piece.
template <int V, int U, class Block, class Whole, class One>
__device__ __forceinline__ void each_dense(int n, Block block, Whole whole, One one) {
  constexpr int step = kThreads * V;
  const int end = n / V * V;
  int i = threadIdx.x * V;
  for (; i + (U - 1) * step < end; i += U * step) block(i, step);
  for (; i < end; i += step) whole(i);
  if (i == end)
    for (int j = end; j < n; ++j) one(j);
}

// A chunk of units by this thread: f(row, column, elements of the unit).
template <class F>
__device__ __forceinline__ void each_unit(const ListEntry &e, const Span &s, F f) {
  const int64_t row0 = s.first / e.per_row;
  const int64_t at0 = s.first - row0 * e.per_row;
  const bool narrow = e.per_row < (int64_t(1) << 30);   // 32-bit division
  for (int u = threadIdx.x; u < s.n; u += kThreads) {
    int64_t r, q;
    if (narrow) {
      const uint32_t at = static_cast<uint32_t>(at0) + u;
      const uint32_t d = at / static_cast<uint32_t>(e.per_row);
      r = row0 + d;
      q = at - d * static_cast<uint32_t>(e.per_row);
    } else {
      const int64_t d = (at0 + u) / e.per_row;
      r = row0 + d;
      q = at0 + u - d * e.per_row;
    }
    const int64_t c = q * kListUnit;
    const int64_t left = e.cols - c;
    f(r, c, static_cast<int>(left < kListUnit ? left : kListUnit));
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

// What one thread has of a chunk's norm: a sum of squares, or the largest
// magnitude.
template <class E, bool MAX> struct NormPart;
template <class E> struct NormPart<E, false> {
  double acc = 0.0, acc2 = 0.0;
  template <int V> __device__ void add(const RawOf<E, V> &r) {
    float x[V];
    decode<E, V>(r, x);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      acc = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), acc);
      acc2 = fma(static_cast<double>(x[i + 1]), static_cast<double>(x[i + 1]), acc2);
    }
  }
  __device__ void add_one(typename E::S v) {
    const double x = E::ld(v);
    acc = fma(x, x, acc);
  }
  __device__ void finish(uint64_t *out) {
    const double t = block_sum(acc + acc2);
    if (threadIdx.x == 0) *out = __double_as_longlong(t);
  }
};
template <class E> struct NormPart<E, true> {
  uint32_t top = 0;
  template <int V> __device__ void add(const RawOf<E, V> &r) {
    float x[V];
    decode<E, V>(r, x);
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, magnitude(x[i]));
  }
  __device__ void add_one(typename E::S v) { top = max(top, magnitude(E::ld(v))); }
  __device__ void finish(uint64_t *out) {
    const uint32_t t = block_max(top);
    if (threadIdx.x == 0) *out = t;
  }
};

template <bool MAX>
__global__ void __launch_bounds__(kThreads) list_partials(ListView v, uint64_t *partials) {
  const ListChunk ch = v.chunks[blockIdx.x];
  const ListEntry &e = v.entries[ch.entry];
  const Span s = span_of(e, ch.index, v.chunk_units);
  with_type(e.dtype[0], [&](auto type) {
    using E = decltype(type);
    using S = typename E::S;
    constexpr int V = 16 / sizeof(S);
    const S *base = static_cast<const S *>(e.data[0]);
    NormPart<E, MAX> part;
    if (s.dense) {
      const S *p = base + s.first;
      each_dense<V, kUnroll>(
          s.n,
          [&](int i, int step) {
            RawOf<E, V> r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) r[u] = ld_raw<E, V>(p + i + u * step);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) part.template add<V>(r[u]);
          },
          [&](int i) { part.template add<V>(ld_raw<E, V>(p + i)); }, [&](int i) { part.add_one(ld_one(p + i)); });
    } else {
      const int64_t pitch = e.pitch[0];
      each_unit(e, s, [&](int64_t r, int64_t c, int n) {
        const S *p = base + r * pitch + c;
        if (n == kListUnit) part.template add<kListUnit>(ld_raw<E, kListUnit>(p));
        else
          for (int j = 0; j < n; ++j) part.add_one(ld_one(p + j));
      });
    }
    part.finish(partials + blockIdx.x);
  });
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
  const Span s = span_of(e, ch.index, v.chunk_units);
  with_type(e.dtype[0], [&](auto from) {
    with_type(e.dtype[dst], [&](auto to) {
      using A = decltype(from);
      using B = decltype(to);
      using SA = typename A::S;
      using SB = typename B::S;
      constexpr int V = sizeof(SA) == 2 && sizeof(SB) == 2 ? 8 : 4;   // 16 bytes on the wider side
      const SA *x = static_cast<const SA *>(e.data[0]);
      SB *y = static_cast<SB *>(e.data[dst]);
      if (s.dense) {
        const SA *p = x + s.first;
        SB *q = y + s.first;
        auto put = [&](int i, const RawOf<A, V> &r) {
          float t[V];
          decode<A, V>(r, t);
#pragma unroll
          for (int j = 0; j < V; ++j) t[j] *= f;
          st_raw<B, V>(q + i, encode<B, V>(t));
        };
        each_dense<V, kUnroll>(
            s.n,
            [&](int i, int step) {
              RawOf<A, V> r[kUnroll];
#pragma unroll
              for (int u = 0; u < kUnroll; ++u) r[u] = ld_raw<A, V>(p + i + u * step);
#pragma unroll
              for (int u = 0; u < kUnroll; ++u) put(i + u * step, r[u]);
            },
            [&](int i) { put(i, ld_raw<A, V>(p + i)); }, [&](int i) { st_one(q + i, B::st(A::ld(ld_one(p + i)) * f)); });
      } else {
        each_unit(e, s, [&](int64_t r, int64_t c, int n) {
          const SA *p = x + r * e.pitch[0] + c;
          SB *q = y + r * e.pitch[dst] + c;
          if (n == kListUnit) {
            float t[kListUnit];
            decode<A, kListUnit>(ld_raw<A, kListUnit>(p), t);
#pragma unroll
            for (int j = 0; j < kListUnit; ++j) t[j] *= f;
            st_raw<B, kListUnit>(q, encode<B, kListUnit>(t));
          } else {
            for (int j = 0; j < n; ++j) st_one(q + j, B::st(A::ld(ld_one(p + j)) * f));
          }
        });
      }
    });
  });
}

// One element's update: m and v in place, the parameter returned.
struct AdamwRule {
  float f, beta1, one_minus_beta1, beta2, one_minus_beta2, inv_sqrt_bias2, eps, decay, rate;
  __device__ float operator()(float p, float g, float &m, float &v) const {
    g *= f;
    m = fmaf(beta1, m, one_minus_beta1 * g);
    v = fmaf(beta2, v, one_minus_beta2 * (g * g));
    return fmaf(-rate, m / fmaf(sqrtf(v), inv_sqrt_bias2, eps), decay * p);
  }
};

template <bool COPY>
__global__ void __launch_bounds__(kThreads) list_adamw(ListView v, AdamwScalars h, const float *grad_scale) {
  const float f = grad_scale ? *grad_scale : 1.0f;
  if (!isfinite(f)) return;
  const ListChunk ch = v.chunks[blockIdx.x];
  const ListEntry &e = v.entries[ch.entry];
  const Span s = span_of(e, ch.index, v.chunk_units);
  const double eta = h.lr * e.lr_scale;
  const AdamwRule rule{f, h.beta1, h.one_minus_beta1, h.beta2, h.one_minus_beta2, h.inv_sqrt_bias2, h.eps,
                       static_cast<float>(1.0 - eta * (h.weight_decay * e.wd_scale)),
                       static_cast<float>(eta / h.bias1)};
  float *P = static_cast<float *>(e.data[1]), *M = static_cast<float *>(e.data[2]),
        *Q = static_cast<float *>(e.data[3]);
  auto body = [&](auto grad, auto copy) {
    using G = decltype(grad);
    using C = decltype(copy);
    const typename G::S *g = static_cast<const typename G::S *>(e.data[0]);
    typename C::S *w = static_cast<typename C::S *>(e.data[4]);
    auto update = [&](auto width, const auto &rp, const auto &rg, const auto &rm, const auto &rq, int64_t ip,
                      int64_t im, int64_t iq, int64_t iw) {
      constexpr int V = decltype(width)::value;
      float p[V], x[V], m[V], q[V];
      decode<EF32, V>(rp, p);
      decode<G, V>(rg, x);
      decode<EF32, V>(rm, m);
      decode<EF32, V>(rq, q);
#pragma unroll
      for (int j = 0; j < V; ++j) p[j] = rule(p[j], x[j], m[j], q[j]);
      st_raw<EF32, V>(P + ip, encode<EF32, V>(p));
      st_raw<EF32, V>(M + im, encode<EF32, V>(m));
      st_raw<EF32, V>(Q + iq, encode<EF32, V>(q));
      if constexpr (COPY) st_raw<C, V>(w + iw, encode<C, V>(p));
    };
    auto one = [&](int64_t ig, int64_t ip, int64_t im, int64_t iq, int64_t iw) {
      float m = ld_one(M + im), q = ld_one(Q + iq);
      const float p = rule(ld_one(P + ip), G::ld(ld_one(g + ig)), m, q);
      st_one(P + ip, p);
      st_one(M + im, m);
      st_one(Q + iq, q);
      if constexpr (COPY) st_one(w + iw, C::st(p));
    };
    if (s.dense) {
      constexpr int V = 4, U = 2;
      auto whole = [&](int i) {
        const int64_t at = s.first + i;
        update(std::integral_constant<int, V>{}, ld_raw<EF32, V>(P + at), ld_raw<G, V>(g + at),
               ld_raw<EF32, V>(M + at), ld_raw<EF32, V>(Q + at), at, at, at, at);
      };
      each_dense<V, U>(
          s.n,
          [&](int i, int step) {
            RawOf<EF32, V> rp[U], rm[U], rq[U];
            RawOf<G, V> rg[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int64_t at = s.first + i + u * step;
              rp[u] = ld_raw<EF32, V>(P + at);
              rg[u] = ld_raw<G, V>(g + at);
              rm[u] = ld_raw<EF32, V>(M + at);
              rq[u] = ld_raw<EF32, V>(Q + at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int64_t at = s.first + i + u * step;
              update(std::integral_constant<int, V>{}, rp[u], rg[u], rm[u], rq[u], at, at, at, at);
            }
          },
          whole, [&](int i) { one(s.first + i, s.first + i, s.first + i, s.first + i, s.first + i); });
    } else {
      each_unit(e, s, [&](int64_t r, int64_t c, int n) {
        const int64_t ig = r * e.pitch[0] + c, ip = r * e.pitch[1] + c, im = r * e.pitch[2] + c,
                      iq = r * e.pitch[3] + c, iw = r * e.pitch[4] + c;
        if (n == kListUnit) {
          constexpr int V = kListUnit;
          update(std::integral_constant<int, V>{}, ld_raw<EF32, V>(P + ip), ld_raw<G, V>(g + ig),
                 ld_raw<EF32, V>(M + im), ld_raw<EF32, V>(Q + iq), ip, im, iq, iw);
        } else {
          for (int j = 0; j < n; ++j) one(ig + j, ip + j, im + j, iq + j, iw + j);
        }
      });
    }
  };
  with_type(e.dtype[0], [&](auto grad) {
    if constexpr (COPY) with_type(e.dtype[4], [&](auto copy) { body(grad, copy); });
    else body(grad, EF32{});
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
  const dim3 grid(static_cast<unsigned>(v.n_chunks));
  if (copy) list_adamw<true><<<grid, kThreads, 0, s>>>(v, h, grad_scale);
  else list_adamw<false><<<grid, kThreads, 0, s>>>(v, h, grad_scale);
  return hipGetLastError();
}

}  // namespace gns
