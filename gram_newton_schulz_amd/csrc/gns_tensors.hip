// Device kernels over lists of tensors: global norm, clipping and AdamW.
//
// A list's table (ListEntry, ListChunk) lies in device memory; every kernel
// runs one workgroup per chunk of one entry.  All of them are bound by HBM:
// a handful of operations per element against 2 to 28 bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gns_elem.h"
#include "gns_kernels.h"

namespace gns {

namespace {

constexpr int kThreads = 256;

// Norms of up to this many chunks are one launch (list_norm_once), where the
// workgroup that ends last adds the partials up: a call is bound by its
// launches there, and one instead of two takes a list of 24 x 1024 fp32 from
// 12.8 to 8.1 us, of 4M elements (512 chunks) from 10.8 to 8.1 (bf16) and 8.8
// (fp32).  Each workgroup pays an atomic and its fences, which line up on one
// address, so there are few, of four chunks each: with 1024 chunks there is
// nothing to gain, 2048 cost 4 us, and with a workgroup for each of 16384
// chunks it was 800 us.
constexpr int64_t kOnceChunks = 512, kOnceEntries = 4096;
// Entries of more chunks have their norm added up by a wave instead of a thread.
constexpr uint32_t kLargeEntry = 16;

// Up to this many partials are added up by every workgroup of the scaling
// itself, which saves the launch between: 3 x 513x777 13.9 -> 11.5 us per
// call, 8 x 512x4096 bf16 (2048 chunks) 18.9 -> 17.5; with 16384 chunks it
// costs 82 us.
constexpr int64_t kScaleChunks = 4096;

// The passes that write cut the chunks into parts of so many units, a
// workgroup each.  The workgroups run in order, so short ones keep all of them
// in a narrow window of every array that moves through memory, where long
// ones each go their own way: AdamW of 268M elements with the norm before it
// takes 1448 us with parts of 16384 elements, 1415 with 8192, 1391 with 4096,
// 1372 with 2048, 1270 with 1024 (one 16-byte piece of each array per thread)
// and 1288 with 512; of 8.9M packed elements 58.4 with 4096, 55.3, 53.3 and 55.0.
// Its streaming hints belong to that: plain loads or stores take it to 1450.
// (All of this is dense chunks.  A part of a strided entry is 128 units for 256
// threads, so half of them have none: the part size was not chosen for those.)
// Grids that walk the parts in a loop instead lose the window again
// (clipping 64 x 2048x7168 bf16: 880 us one by one, 1010 to 1270 in loops).
constexpr int64_t kAdamwUnits = 128;
// Clipping moves fewer bytes per workgroup, so that starting them weighs more
// (940M bf16 elements: 960 us with parts of 8192 units, 915 with 2048, 880 with
// 512, 1010 with 256).  Lists that the last-level cache holds do not gain
// (134 MB fp16 to fp32: 83 us whole, 86 with 512).  In place most steps end
// with nothing to write once training is stable, and then starting the
// workgroups is all that is left: 5 us for the same list with 8192 units, 47
// with 512.
constexpr int64_t kScaleUnits = 512, kScaleInPlaceUnits = 8192;

// V consecutive elements as they lie in memory.  The addresses are aligned to
// the element only: gfx950 loads and stores 8 and 16 bytes from any address,
// and a wave's accesses are consecutive, so a misaligned tensor costs one more
// cache line per wave and instruction, not another path.
template <int BYTES> struct Raw;
template <> struct Raw<4> {
  typedef uint32_t T __attribute__((ext_vector_type(1), aligned(2)));
  T v[1];
};
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

// NT: with the streaming hint, for data that this pass is the last to want.
template <class E, int V, bool NT>
__device__ __forceinline__ RawOf<E, V> ld_raw(const typename E::S *p) {
  using R = RawOf<E, V>;
  R r;
  const GNS_GLOBAL typename R::T *q = (const GNS_GLOBAL typename R::T *)p;
#pragma unroll
  for (unsigned i = 0; i < sizeof(R) / sizeof(typename R::T); ++i) {
    if constexpr (NT) r.v[i] = __builtin_nontemporal_load(q + i);
    else r.v[i] = q[i];
  }
  return r;
}
template <class E, int V, bool NT>
__device__ __forceinline__ void st_raw(typename E::S *p, const RawOf<E, V> &r) {
  using R = RawOf<E, V>;
  GNS_GLOBAL typename R::T *q = (GNS_GLOBAL typename R::T *)p;
#pragma unroll
  for (unsigned i = 0; i < sizeof(R) / sizeof(typename R::T); ++i) {
    if constexpr (NT) __builtin_nontemporal_store(r.v[i], q + i);
    else q[i] = r.v[i];
  }
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

// A unit of n <= kListUnit elements.  A short one is its pieces of four, two
// and one, in x[0..3], x[4..5] and x[6] (the rest of x is zero).
template <class E, int V, bool NT>
__device__ __forceinline__ void ld_piece(const typename E::S *p, float *x) {
  float t[V];
  decode<E, V>(ld_raw<E, V, NT>(p), t);
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = t[j];
}
template <class E, int V, bool NT>
__device__ __forceinline__ void st_piece(typename E::S *p, const float *x) {
  float t[V];
#pragma unroll
  for (int j = 0; j < V; ++j) t[j] = x[j];
  st_raw<E, V, NT>(p, encode<E, V>(t));
}
template <class E, bool NT>
__device__ __forceinline__ void ld_unit(const typename E::S *p, int n, float (&x)[kListUnit]) {
  if (n == kListUnit) {
    ld_piece<E, kListUnit, NT>(p, x);
  } else {
#pragma unroll
    for (int j = 0; j < kListUnit; ++j) x[j] = 0.0f;
    if (n & 4) ld_piece<E, 4, NT>(p, x);
    if (n & 2) ld_piece<E, 2, NT>(p + (n & 4), x + 4);
    if (n & 1) x[6] = E::ld(ld_one(p + (n & 6)));
  }
}
template <class E, bool NT>
__device__ __forceinline__ void st_unit(typename E::S *p, int n, const float (&x)[kListUnit]) {
  if (n == kListUnit) {
    st_piece<E, kListUnit, NT>(p, x);
  } else {
    if (n & 4) st_piece<E, 4, NT>(p, x);
    if (n & 2) st_piece<E, 2, NT>(p + (n & 4), x + 4);
    if (n & 1) st_one(p + (n & 6), E::st(x[6]));
  }
}

// Calls f with a value of the element type that a table names.
template <class F>
__device__ __forceinline__ void with_type(int dtype, F f) {
  if (dtype == DT_BF16) f(EBF16{});
  else if (dtype == DT_F16) f(EF16{});
  else f(EF32{});
}

// A chunk of an entry.  Dense: `n` elements from element `first` of the only
// row.  Otherwise units [first, first + n), found row by row.
//
// Dense chunks are shifted so that array `a` starts on a multiple of kStart
// bytes from element `head` of the chunk on (head > 0 in an entry's first chunk
// only): tensors packed behind one another start anywhere, and stores that end
// inside a cache line leave partial lines behind.  Two lines of 128 bytes,
// so that a 16-bit array at the same offset in its own buffer starts on one.
// Without the shift, with 128 bytes, with 256: AdamW of 200 packed fp32
// tensors (8.9M elements) 57.2, 53.4, 53.2 us; of 60 with bf16 gradients and
// copies (27M) 150, 131, 129; clipping their gradients into fp32 42.3, 39.7,
// 35.4.  Arrays of another phase are accessed across lines.
constexpr int kStart = 256;
static_assert(kStart / 2 <= kThreads, "a thread for every element of a head");
struct Span {
  int64_t first;
  int n, head;
  bool dense;
};
__device__ __forceinline__ Span span_of(const ListEntry &e, uint32_t index, int64_t chunk_units, int a) {
  Span s;
  const int64_t u0 = static_cast<int64_t>(index) * chunk_units;
  s.dense = e.units == e.per_row;
  s.head = 0;
  if (s.dense) {
    const uint32_t size = e.dtype[a] == DT_F32 ? 4 : 2;
    const int shift = static_cast<int>((0u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(e.data[a]))) %
                                       kStart / size);
    const int64_t end = (u0 + chunk_units) * kListUnit + shift;
    s.first = index ? u0 * kListUnit + shift : 0;
    const int64_t n = (end < e.cols ? end : e.cols) - s.first;
    s.n = n > 0 ? static_cast<int>(n) : 0;
    if (!index) s.head = shift < s.n ? shift : s.n;
  } else {
    s.first = u0;
    const int64_t left = e.units - u0;
    s.n = left <= 0 ? 0 : static_cast<int>(left < chunk_units ? left : chunk_units);
  }
  return s;
}

// Which of the kThreads threads that share a chunk this is.
__device__ __forceinline__ int thread_of_chunk() { return threadIdx.x % kThreads; }

// A dense chunk by this thread: block(i, stride) takes U pieces of V elements
// (it can issue all their loads first), whole(i) one piece, and one(i) one
// element, at the two ends.
template <int V, int U, class Block, class Whole, class One>
__device__ __forceinline__ void each_dense(const Span &s, Block block, Whole whole, One one) {
  constexpr int step = kThreads * V;
  const int end = s.head + (s.n - s.head) / V * V;
  int i = s.head + thread_of_chunk() * V;
  for (; i + (U - 1) * step < end; i += U * step) block(i, step);
  for (; i < end; i += step) whole(i);
  const int t = thread_of_chunk();
  if (t < s.head) one(t);
  if (t < s.n - end) one(end + t);
}

// A chunk of units by this thread: f(row, column, elements of the unit).
template <class F>
__device__ __forceinline__ void each_unit(const ListEntry &e, const Span &s, F f) {
  const int64_t row0 = s.first / e.per_row;
  const int64_t at0 = s.first - row0 * e.per_row;
  const bool narrow = e.per_row < (int64_t(1) << 30);   // 32-bit division
  for (int u = thread_of_chunk(); u < s.n; u += kThreads) {
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

// Partials are 64 bits: a sum of squares (fp64), or with MAX the bits of the
// largest magnitude as a float.  Zero bits are zero for both.
template <bool MAX> __device__ __forceinline__ uint64_t join(uint64_t a, uint64_t b) {
  if constexpr (MAX) return max(static_cast<uint32_t>(a), static_cast<uint32_t>(b));
  else return __double_as_longlong(__longlong_as_double(a) + __longlong_as_double(b));
}
template <bool MAX> __device__ __forceinline__ double norm_of_total(uint64_t bits) {
  if constexpr (MAX) return __uint_as_float(static_cast<uint32_t>(bits));
  else return sqrt(__longlong_as_double(bits));
}

// Sum (or maximum) over a wave, in a fixed order; the first lane's.
template <bool MAX>
__device__ __forceinline__ uint64_t wave_total(uint64_t bits) {
  for (int off = 32; off > 0; off >>= 1)
    bits = join<MAX>(bits, __shfl_down(static_cast<unsigned long long>(bits), off, 64));
  return bits;
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
    add_values<V>(x);
  }
  template <int V> __device__ void add_values(const float (&x)[V]) {
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
  __device__ uint64_t bits() const { return __double_as_longlong(acc + acc2); }
};
template <class E> struct NormPart<E, true> {
  uint32_t top = 0;
  template <int V> __device__ void add(const RawOf<E, V> &r) {
    float x[V];
    decode<E, V>(r, x);
    add_values<V>(x);
  }
  template <int V> __device__ void add_values(const float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, magnitude(x[i]));
  }
  __device__ void add_one(typename E::S v) { top = max(top, magnitude(E::ld(v))); }
  __device__ uint64_t bits() const { return top; }
};

// Total of `n` partials, this thread's share as number `t` of `threads`.
template <bool MAX>
__device__ __forceinline__ uint64_t partials_of(const uint64_t *p, int64_t n, int t, int threads) {
  constexpr int kAtOnce = 16;   // loads in flight per thread
  uint64_t total = 0;
  for (int64_t i = t; i < n; i += kAtOnce * threads) {
    uint64_t x[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) x[u] = i + u * threads < n ? p[i + u * threads] : 0;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) total = join<MAX>(total, x[u]);
  }
  return total;
}

// Norm of `n` partials (thread 0's), by the whole workgroup of up to 16 waves.
template <bool MAX>
__device__ __forceinline__ double norm_of(const uint64_t *partials, int64_t n) {
  __shared__ uint64_t part[16];
  uint64_t total = wave_total<MAX>(partials_of<MAX>(partials, n, threadIdx.x, blockDim.x));
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = total;
  __syncthreads();
  if (threadIdx.x == 0)
    for (unsigned w = 1; w < blockDim.x / 64; ++w) total = join<MAX>(total, part[w]);
  return norm_of_total<MAX>(total);
}

// The result's {norm, clip factor} from the norm of the stored gradients.
__device__ __forceinline__ double unscale(const NormArgs &a) {
  return a.inv_scale ? static_cast<double>(*a.inv_scale) : 1.0;
}
__device__ __forceinline__ float2 result_of(const NormArgs &a, double raw) {
  const double s = unscale(a);
  const double norm = raw * fabs(s);
  const double ratio = a.max_norm / (norm + a.eps);
  return make_float2(static_cast<float>(norm),
                     isfinite(norm) ? static_cast<float>(s * (ratio < 1.0 ? ratio : 1.0)) : __builtin_nanf(""));
}
__device__ __forceinline__ void write_result(const NormArgs &a, double raw) {
  const float2 r = result_of(a, raw);
  a.result[0] = r.x;
  a.result[1] = r.y;
}

// This thread's share of chunk c's norm.
template <bool MAX>
__device__ __forceinline__ uint64_t chunk_part(const ListView &v, int64_t c) {
  const ListChunk ch = v.chunks[c];
  const ListEntry &e = v.entries[ch.entry];
  const Span s = span_of(e, ch.index, v.chunk_units, 0);
  uint64_t bits = 0;
  with_type(e.dtype[0], [&](auto type) {
    using E = decltype(type);
    using S = typename E::S;
    constexpr int V = 16 / sizeof(S);
    const S *base = static_cast<const S *>(e.data[0]);
    NormPart<E, MAX> part;
    // Loads with the streaming hint run at 7.0 TB/s against 6.0, but leave
    // nothing in the last-level cache for the pass that takes the gradients
    // next.  So the chunks that fill the cache are read without it: AdamW after
    // the norm of 67M fp32 gradients 383 -> 343 us for both, clipping 268M
    // fp32 gradients 528 -> 516, and a norm alone pays for it with 4 of
    // 164 us (8 x 4096x16384 bf16).
    auto dense = [&](auto once) {
      constexpr bool ONCE = decltype(once)::value;
      const S *p = base + s.first;
      each_dense<V, kUnroll>(
          s,
          [&](int i, int step) {
            RawOf<E, V> r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) r[u] = ld_raw<E, V, ONCE>(p + i + u * step);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) part.template add<V>(r[u]);
          },
          [&](int i) { part.template add<V>(ld_raw<E, V, ONCE>(p + i)); }, [&](int i) { part.add_one(ld_one(p + i)); });
    };
    if (s.dense && c < v.keep_from) dense(std::true_type{});
    else if (s.dense) dense(std::false_type{});
    else {
      // without the hint, whatever the size: neighbouring threads end and begin
      // in the same cache line, which has to stay for the second of them.  With
      // it 3 slices of 777 columns take 43.1 us (norm and AdamW) against 34.7, 47
      // of 15 columns 51.9 against 41.6, and what it gains is 2 of 90 us for the
      // norm of 3 x 8192x5120 fp32 alone.
      const int64_t pitch = e.pitch[0];
      each_unit(e, s, [&](int64_t r, int64_t c, int n) {
        float x[kListUnit];
        ld_unit<E, false>(base + r * pitch + c, n, x);
        part.template add_values<kListUnit>(x);
      });
    }
    bits = part.bits();
  });
  return bits;
}

// partials[c] of chunk c, one workgroup per chunk.
template <bool MAX>
__global__ void __launch_bounds__(kThreads) list_partials(ListView v, uint64_t *partials) {
  __shared__ uint64_t part[kThreads / 64];
  const uint64_t bits = wave_total<MAX>(chunk_part<MAX>(v, blockIdx.x));
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = bits;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint64_t total = part[0];
    for (int w = 1; w < kThreads / 64; ++w) total = join<MAX>(total, part[w]);
    partials[blockIdx.x] = total;
  }
}

// Whether a factor changes anything: not finite, nothing is written; one, an
// array in place is what it should be.
__device__ __forceinline__ bool scales(float f, int dst) { return isfinite(f) && (dst != 0 || f != 1.0f); }

// Array dst <- f * array 0 in part `part` of `parts` of chunk c.
__device__ __forceinline__ void scale_chunk(const ListView &v, int dst, float f, int64_t c, unsigned part,
                                            unsigned parts) {
  const ListChunk ch = v.chunks[c];
  const ListEntry &e = v.entries[ch.entry];
  const Span s = span_of(e, ch.index * parts + part, v.chunk_units / parts, dst);
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
          st_raw<B, V, true>(q + i, encode<B, V>(t));
        };
        each_dense<V, kUnroll>(
            s,
            [&](int i, int step) {
              RawOf<A, V> r[kUnroll];
#pragma unroll
              for (int u = 0; u < kUnroll; ++u) r[u] = ld_raw<A, V, true>(p + i + u * step);
#pragma unroll
              for (int u = 0; u < kUnroll; ++u) put(i + u * step, r[u]);
            },
            [&](int i) { put(i, ld_raw<A, V, true>(p + i)); },
            [&](int i) { st_one(q + i, B::st(A::ld(ld_one(p + i)) * f)); });
      } else {
        each_unit(e, s, [&](int64_t r, int64_t c, int n) {
          const SA *p = x + r * e.pitch[0] + c;
          SB *q = y + r * e.pitch[dst] + c;
          // each width on its own, from load to store: a wave then waits for the
          // ends of rows while the stores of the whole units are on their way.
          // With the hint, as the dense chunks: norm and clipping of 3 slices
          // 16384x5120 bf16 299 us against 353 without, of 5121 columns into fp32
          // 460 against 513; 12 slices 80x20000 bf16 into fp32 are the other way
          // round, 38.5 against 34.3.
          auto piece = [&](auto width, int at) {
            constexpr int W = decltype(width)::value;
            float t[W];
            decode<A, W>(ld_raw<A, W, true>(p + at), t);
#pragma unroll
            for (int j = 0; j < W; ++j) t[j] *= f;
            st_raw<B, W, true>(q + at, encode<B, W>(t));
          };
          if (n == kListUnit) {
            piece(std::integral_constant<int, kListUnit>{}, 0);
          } else {
            if (n & 4) piece(std::integral_constant<int, 4>{}, 0);
            if (n & 2) piece(std::integral_constant<int, 2>{}, n & 4);
            if (n & 1) st_one(q + (n & 6), B::st(A::ld(ld_one(p + (n & 6))) * f));
          }
        });
      }
    });
  });
}

// A norm in one launch, for lists of few chunks: kGroups chunks to a
// workgroup, and the workgroup that ends last adds the partials up
// (in the order of the chunks) and writes the result and the entries' norms.
// It leaves *arrived at zero, as it found it.
//
// CLIP (lists of up to kGroups chunks, one workgroup): then array dst <- clip
// factor * array 0.  One launch instead of two takes clipping 8192 to 32768
// elements from 10.8 to 8.1 us per call; with a second round of chunks, 16 of
// them, it was 23 us against 11.
constexpr int kGroups = 4;
template <bool MAX, bool CLIP>
__global__ void __launch_bounds__(kGroups * kThreads)
list_norm_once(ListView v, uint64_t *partials, uint32_t *arrived, NormArgs args, float *tensor_norms, int dst) {
  constexpr int kWaves = kGroups * kThreads / 64;
  static_assert(kOnceChunks <= kGroups * kThreads, "a thread for every partial");
  __shared__ uint64_t part[kWaves];
  const int t = threadIdx.x, wave = t / 64, n = static_cast<int>(v.n_chunks);
  const int c0 = blockIdx.x * kGroups, c = c0 + t / kThreads;
  const uint64_t bits = wave_total<MAX>(c < n ? chunk_part<MAX>(v, c) : 0);
  if (t % 64 == 0) part[wave] = bits;
  __syncthreads();
  // one thread stores all of them, so that its release below covers them
  if (t == 0) {
    for (int g = 0; g < kGroups && c0 + g < n; ++g) {
      uint64_t total = part[g * (kWaves / kGroups)];
      for (int w = 1; w < kWaves / kGroups; ++w) total = join<MAX>(total, part[g * (kWaves / kGroups) + w]);
      __hip_atomic_store(partials + c0 + g, total, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  __shared__ bool last;
  if (t == 0)
    last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __shared__ uint64_t all[kOnceChunks];
  __shared__ uint32_t large[kOnceChunks / kLargeEntry], n_large;
  __shared__ float factor;
  uint64_t mine = 0;
  if (t < n) mine = all[t] = __hip_atomic_load(partials + t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (t == 0) n_large = 0;
  mine = wave_total<MAX>(mine);
  if (t % 64 == 0) part[wave] = mine;
  __syncthreads();
  if (t == 0) {
    uint64_t total = part[0];
    for (int w = 1; w < kWaves; ++w) total = join<MAX>(total, part[w]);
    const float2 r = result_of(args, norm_of_total<MAX>(total));
    args.result[0] = r.x;
    args.result[1] = factor = r.y;
    __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if constexpr (CLIP) {
    __syncthreads();
    if (c < n && scales(factor, dst)) scale_chunk(v, dst, factor, c, 0, 1);
  }
  if (!tensor_norms) return;
  // entries of few chunks by a thread, the others by a wave
  const double s = fabs(unscale(args));
  for (int64_t i = t; i < v.count; i += kGroups * kThreads) {
    const uint32_t first = v.entries[i].first_chunk, count = v.entries[i].chunks;
    if (count > kLargeEntry) {
      large[atomicAdd(&n_large, 1u)] = static_cast<uint32_t>(i);
      continue;
    }
    uint64_t total = 0;
    for (uint32_t c = first; c < first + count; ++c) total = join<MAX>(total, all[c]);
    tensor_norms[i] = static_cast<float>(norm_of_total<MAX>(total) * s);
  }
  __syncthreads();
  for (uint32_t k = wave; k < n_large; k += kWaves) {
    const ListEntry &e = v.entries[large[k]];
    uint64_t total = 0;
    for (uint32_t c = t % 64; c < e.chunks; c += 64) total = join<MAX>(total, all[e.first_chunk + c]);
    total = wave_total<MAX>(total);
    if (t % 64 == 0) tensor_norms[large[k]] = static_cast<float>(norm_of_total<MAX>(total) * s);
  }
}

// The second launch of a norm: block 0 writes the result; the others write
// the entries' own norms, a block or (per_wave) a wave to each.
template <bool MAX>
__global__ void __launch_bounds__(1024)
list_finish(ListView v, const uint64_t *partials, NormArgs args, float *tensor_norms, bool per_wave) {
  if (blockIdx.x == 0) {
    const double norm = norm_of<MAX>(partials, v.n_chunks);
    if (threadIdx.x == 0) write_result(args, norm);
    return;
  }
  const double s = fabs(unscale(args));
  if (!per_wave) {
    const ListEntry &e = v.entries[blockIdx.x - 1];
    const double norm = norm_of<MAX>(partials + e.first_chunk, e.chunks) * s;
    if (threadIdx.x == 0) tensor_norms[blockIdx.x - 1] = static_cast<float>(norm);
    return;
  }
  const int64_t i = (blockIdx.x - 1) * static_cast<int64_t>(blockDim.x / 64) + threadIdx.x / 64;
  if (i >= v.count) return;
  const ListEntry &e = v.entries[i];
  const uint64_t total =
      wave_total<MAX>(partials_of<MAX>(partials + e.first_chunk, e.chunks, threadIdx.x % 64, 64));
  if (threadIdx.x % 64 == 0) tensor_norms[i] = static_cast<float>(norm_of_total<MAX>(total) * s);
}

// Clipping after the norm's partials, one workgroup for each of `parts` parts
// of a chunk.  The factor is the result's, or with PARTIALS every workgroup's
// own sum of the partials (all in the same order, so all the same), of which
// the first writes the result.
template <bool PARTIALS, bool MAX>
__global__ void __launch_bounds__(kThreads)
list_scale(ListView v, int dst, const uint64_t *partials, NormArgs args, unsigned parts) {
  float f;
  if constexpr (PARTIALS) {
    __shared__ float2 found;
    const double norm = norm_of<MAX>(partials, v.n_chunks);
    if (threadIdx.x == 0) {
      found = result_of(args, norm);
      if (blockIdx.x == 0) {
        args.result[0] = found.x;
        args.result[1] = found.y;
      }
    }
    __syncthreads();
    f = found.y;
  } else {
    f = args.result[1];
  }
  if (scales(f, dst)) scale_chunk(v, dst, f, blockIdx.x / parts, blockIdx.x % parts, parts);
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

// Counts a step on the GPU and leaves its bias factors (fp64 powers, rounded
// as the host's are) for the update.  A launch of its own, since every
// workgroup of the update reads what it writes: AdamW of 48 x 1024 fp32 takes
// 8.8 us per call with it and 3.9 without, of 268M elements 1112 and 1109.
__global__ void adamw_count(int64_t *count, double beta1, double beta2, const float *grad_scale, AdamwBias *bias) {
  if (grad_scale && !isfinite(*grad_scale)) return;
  const int64_t step = *count + 1;
  *count = step;
  const double t = static_cast<double>(step);
  bias->bias1 = 1.0 - pow(beta1, t);
  bias->inv_sqrt_bias2 = static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, t)));
}

template <bool COPY>
__global__ void __launch_bounds__(kThreads)
list_adamw(ListView v, AdamwScalars h, const AdamwBias *counted, const float *grad_scale, unsigned parts) {
  const float f = grad_scale ? *grad_scale : 1.0f;
  if (!isfinite(f)) return;
  const ListChunk ch = v.chunks[blockIdx.x / parts];
  const ListEntry &e = v.entries[ch.entry];
  const Span s = span_of(e, ch.index * parts + blockIdx.x % parts, v.chunk_units / parts, 1);
  const double eta = h.lr * e.lr_scale;
  const AdamwBias bias = counted ? *counted : h.bias;
  const AdamwRule rule{f, h.beta1, h.one_minus_beta1, h.beta2, h.one_minus_beta2, bias.inv_sqrt_bias2, h.eps,
                       static_cast<float>(1.0 - eta * (h.weight_decay * e.wd_scale)),
                       static_cast<float>(eta / bias.bias1)};
  float *P = static_cast<float *>(e.data[1]), *M = static_cast<float *>(e.data[2]),
        *Q = static_cast<float *>(e.data[3]);
  auto body = [&](auto grad, auto copy) {
    using G = decltype(grad);
    using C = decltype(copy);
    const typename G::S *g = static_cast<const typename G::S *>(e.data[0]);
    typename C::S *w = static_cast<typename C::S *>(e.data[4]);
    if (s.dense) {
      constexpr int V = 4;
      auto whole = [&](int i) {
        const int64_t at = s.first + i;
        const auto rp = ld_raw<EF32, V, true>(P + at), rm = ld_raw<EF32, V, true>(M + at),
                   rq = ld_raw<EF32, V, true>(Q + at);
        const auto rg = ld_raw<G, V, true>(g + at);
        float p[V], x[V], m[V], q[V];
        decode<EF32, V>(rp, p);
        decode<G, V>(rg, x);
        decode<EF32, V>(rm, m);
        decode<EF32, V>(rq, q);
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = rule(p[j], x[j], m[j], q[j]);
        st_raw<EF32, V, true>(P + at, encode<EF32, V>(p));
        st_raw<EF32, V, true>(M + at, encode<EF32, V>(m));
        st_raw<EF32, V, true>(Q + at, encode<EF32, V>(q));
        if constexpr (COPY) st_raw<C, V, true>(w + at, encode<C, V>(p));
      };
      each_dense<V, 1>(s, [&](int i, int) { whole(i); }, whole, [&](int i) {
        const int64_t at = s.first + i;
        float m = ld_one(M + at), q = ld_one(Q + at);
        const float p = rule(ld_one(P + at), G::ld(ld_one(g + at)), m, q);
        st_one(P + at, p);
        st_one(M + at, m);
        st_one(Q + at, q);
        if constexpr (COPY) st_one(w + at, C::st(p));
      });
    } else {
      // without the hint, which only wide slices of whole units gain from (norm
      // and AdamW of 3 x 8192x5120 with bf16 gradients and copies 757 us, 737 with
      // it): the ends of rows share cache lines with the next thread's.  3 x
      // 2130x777 34.7 against 48.5 with it, 47 x 2643x15 41.6 against 58.0, AdamW
      // alone of 3 x 8192x5121 825 against 850.
      each_unit(e, s, [&](int64_t r, int64_t c, int n) {
        const int64_t ig = r * e.pitch[0] + c, ip = r * e.pitch[1] + c, im = r * e.pitch[2] + c,
                      iq = r * e.pitch[3] + c, iw = r * e.pitch[4] + c;
        float p[kListUnit], x[kListUnit], m[kListUnit], q[kListUnit];
        ld_unit<EF32, false>(P + ip, n, p);
        ld_unit<G, false>(g + ig, n, x);
        ld_unit<EF32, false>(M + im, n, m);
        ld_unit<EF32, false>(Q + iq, n, q);
#pragma unroll
        for (int j = 0; j < kListUnit; ++j) p[j] = rule(p[j], x[j], m[j], q[j]);
        st_unit<EF32, false>(P + ip, n, p);
        st_unit<EF32, false>(M + im, n, m);
        st_unit<EF32, false>(Q + iq, n, q);
        if constexpr (COPY) st_unit<C, false>(w + iw, n, p);
      });
    }
  };
  with_type(e.dtype[0], [&](auto grad) {
    if constexpr (COPY) with_type(e.dtype[4], [&](auto copy) { body(grad, copy); });
    else body(grad, EF32{});
  });
}

// Into how many parts of `units` units a pass cuts every chunk (a power of
// two, as the chunk is); no more than a grid holds.
unsigned parts_of(const ListView &v, int64_t units) {
  int64_t parts = std::max<int64_t>(1, v.chunk_units / units);
  while (parts > 1 && v.n_chunks * parts > (int64_t(1) << 23)) parts /= 2;
  return static_cast<unsigned>(parts);
}

hipError_t launch_partials(const ListView &v, bool max, uint64_t *partials, hipStream_t s) {
  if (v.n_chunks == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(v.n_chunks));
  if (max) list_partials<true><<<grid, kThreads, 0, s>>>(v, partials);
  else list_partials<false><<<grid, kThreads, 0, s>>>(v, partials);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_list_norm(const ListView &v, bool max, uint64_t *partials, uint32_t *arrived, const NormArgs &a,
                            float *tensor_norms, hipStream_t s) {
  if (v.n_chunks > 0 && v.n_chunks <= kOnceChunks && (!tensor_norms || v.count <= kOnceEntries)) {
    const dim3 grid(static_cast<unsigned>((v.n_chunks + kGroups - 1) / kGroups));
    if (max) list_norm_once<true, false><<<grid, kGroups * kThreads, 0, s>>>(v, partials, arrived, a, tensor_norms, 0);
    else list_norm_once<false, false><<<grid, kGroups * kThreads, 0, s>>>(v, partials, arrived, a, tensor_norms, 0);
    return hipGetLastError();
  }
  hipError_t e = launch_partials(v, max, partials, s);
  if (e != hipSuccess) return e;
  const unsigned threads = v.n_chunks > 256 ? 1024 : 256;
  const bool per_wave = v.count > 256;
  const int64_t each = per_wave ? threads / 64 : 1;
  const dim3 blocks(static_cast<unsigned>(tensor_norms ? 1 + (v.count + each - 1) / each : 1));
  if (max) list_finish<true><<<blocks, threads, 0, s>>>(v, partials, a, tensor_norms, per_wave);
  else list_finish<false><<<blocks, threads, 0, s>>>(v, partials, a, tensor_norms, per_wave);
  return hipGetLastError();
}

hipError_t launch_list_clip(const ListView &v, int dst, bool max, uint64_t *partials, uint32_t *arrived,
                            const NormArgs &a, float *tensor_norms, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(v.n_chunks));
  if (v.n_chunks > 0 && v.n_chunks <= kGroups && v.count <= kOnceEntries) {
    if (max) list_norm_once<true, true><<<1, kGroups * kThreads, 0, s>>>(v, partials, arrived, a, tensor_norms, dst);
    else list_norm_once<false, true><<<1, kGroups * kThreads, 0, s>>>(v, partials, arrived, a, tensor_norms, dst);
    return hipGetLastError();
  }
  if (v.n_chunks == 0 || v.n_chunks > kScaleChunks || tensor_norms) {
    hipError_t e = launch_list_norm(v, max, partials, arrived, a, tensor_norms, s);
    if (e != hipSuccess || v.n_chunks == 0) return e;
    const unsigned parts = v.keep_from == 0 ? 1 : parts_of(v, dst ? kScaleUnits : kScaleInPlaceUnits);
    list_scale<false, false><<<grid.x * parts, kThreads, 0, s>>>(v, dst, nullptr, a, parts);
    return hipGetLastError();
  }
  hipError_t e = launch_partials(v, max, partials, s);
  if (e != hipSuccess) return e;
  if (max) list_scale<true, true><<<grid, kThreads, 0, s>>>(v, dst, partials, a, 1);
  else list_scale<true, false><<<grid, kThreads, 0, s>>>(v, dst, partials, a, 1);
  return hipGetLastError();
}

hipError_t launch_adamw_count(int64_t *count, double beta1, double beta2, const float *grad_scale, AdamwBias *bias,
                              hipStream_t s) {
  adamw_count<<<1, 1, 0, s>>>(count, beta1, beta2, grad_scale, bias);
  return hipGetLastError();
}

hipError_t launch_list_adamw(const ListView &v, bool copy, const AdamwScalars &h, const AdamwBias *bias,
                             const float *grad_scale, hipStream_t s) {
  if (v.n_chunks == 0) return hipSuccess;
  const unsigned parts = parts_of(v, kAdamwUnits);
  const dim3 grid(static_cast<unsigned>(v.n_chunks) * parts);
  if (copy) list_adamw<true><<<grid, kThreads, 0, s>>>(v, h, bias, grad_scale, parts);
  else list_adamw<false><<<grid, kThreads, 0, s>>>(v, h, bias, grad_scale, parts);
  return hipGetLastError();
}

}  // namespace gns
