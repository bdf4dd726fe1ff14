// Token embedding and its gradient, written for CDNA4 (gfx950).
//
// * embedding_rows   -- out[i] = scale weight[tokens[i]]: HBM-bound, 8
//                       elements per thread in 16-byte accesses.
// * token_sort_once, token_count, token_scan, token_scatter
//                    -- a stable sort of the tokens by radix, with the
//                       position of each: up to 6144 tokens in one workgroup,
//                       more of them in three launches per digit.
// * embedding_sums   -- the sorted tokens are cut into pieces of equal length,
//                       whatever their runs: a group of threads adds the
//                       gradient rows of one piece up and writes the rows of
//                       the table whose runs lie within it.  A run that
//                       reaches over the end of a piece leaves partial sums.
//                       Rows that no token names are cleared beside it.
// * embedding_join   -- the partial sums of such runs, added up in order.
//
// Every sum has an order that the tokens decide, and no atomic adds a value.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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

// Workgroups in two dimensions: one holds 2^24 of them (2^32 threads).
dim3 grid_of(int64_t groups) {
  const int64_t x = std::min<int64_t>(groups, int64_t(1) << 20);
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>((groups + x - 1) / x));
}
__device__ __forceinline__ int64_t group_index() {
  return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

struct Tokens {
  const void *at;
  int bits;
  __device__ __forceinline__ int64_t operator[](int64_t i) const {
    return bits == 32 ? static_cast<const int32_t *>(at)[i] : static_cast<const int64_t *>(at)[i];
  }
  // the token, or vocab for padding
  __device__ __forceinline__ uint32_t key(int64_t i, uint32_t vocab) const {
    const int64_t t = (*this)[i];
    return t >= 0 && t < static_cast<int64_t>(vocab) ? static_cast<uint32_t>(t) : vocab;
  }
};

// ---------------------------------------------------------------------------
// rows of a table or of gradients, eight elements per thread
// ---------------------------------------------------------------------------
// Threads work in groups of `lanes` (a power of two up to 256) on one row, and
// a thread has eight columns of a block of 8 lanes:
//   OCTETS   eight consecutive ones: both arrays have 16 bits
//   QUADS    twice four consecutive ones, so that neighbours' 16-byte accesses
//            of an fp32 array meet
// Accesses of 16 bytes need no alignment beyond the element's; rows of odd
// widths take them too (20000 x 1531 bf16 gradients: 73 us, against 106 with an
// element per access).
enum Spread { QUADS, OCTETS };
constexpr int kColumns = 8;
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

struct Columns {
  int first, lanes, width;
  __device__ __forceinline__ Columns(Spread m, int64_t block, int lane, int lanes_, int64_t width_)
      : first(static_cast<int>(block) * lanes_ * kColumns + lane * (m == OCTETS ? 8 : 4)), lanes(lanes_),
        width(static_cast<int>(width_)) {}
  template <Spread M>
  __device__ __forceinline__ int at(int k) const {
    return M == OCTETS ? first + k : first + k / 4 * 4 * lanes + k % 4;
  }
};

// (a row's last piece may be short; the others take one access each)
template <class T, Spread M>
__device__ __forceinline__ void load_columns(const typename T::S *row, const Columns &c, float *v) {
  using S = typename T::S;
  constexpr int N = M == OCTETS ? 8 : 4;                       // of one access
#pragma unroll
  for (int k = 0; k < kColumns; k += N) {
    const int at = c.at<M>(k);
    if (at + N <= c.width) {
      if constexpr (sizeof(S) == 4) {
#pragma unroll
        for (int q = 0; q < N; q += 4) {
          __builtin_memcpy(v + k + q, row + at + q, 16);
        }
      } else {
        uint32_t a[4];
        __builtin_memcpy(a, row + at, 2 * N);
#pragma unroll
        for (int q = 0; q < N; q += 2) {
          v[k + q] = T::ld(static_cast<S>(a[q / 2] & 0xffff));
          v[k + q + 1] = T::ld(static_cast<S>(a[q / 2] >> 16));
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < N; ++q) v[k + q] = at + q < c.width ? T::ld(row[at + q]) : 0.0f;
    }
  }
}

// ONCE: fp32 rows that are not read again here have the streaming hint (32768 x
// 4096 fp32 rows of a gradient, mostly cleared: 210 us with it, 227 without).
template <class T, Spread M, bool ONCE = false>
__device__ __forceinline__ void store_columns(typename T::S *row, const Columns &c, const float *v) {
  using S = typename T::S;
  constexpr int N = M == OCTETS ? 8 : 4;
#pragma unroll
  for (int k = 0; k < kColumns; k += N) {
    const int at = c.at<M>(k);
    if (at + N <= c.width) {
      if constexpr (sizeof(S) == 4) {
#pragma unroll
        for (int q = 0; q < N; q += 4) {
          const f32x4_any a{v[k + q], v[k + q + 1], v[k + q + 2], v[k + q + 3]};
          if constexpr (ONCE) __builtin_nontemporal_store(a, reinterpret_cast<f32x4_any *>(row + at + q));
          else *reinterpret_cast<f32x4_any *>(row + at + q) = a;
        }
      } else {
        uint32_t a[4];
#pragma unroll
        for (int q = 0; q < N; q += 2) a[q / 2] = T::st2(v[k + q], v[k + q + 1]);
        __builtin_memcpy(row + at, a, 2 * N);
      }
    } else {
#pragma unroll
      for (int q = 0; q < N; ++q)
        if (at + q < c.width) row[at + q] = T::st(v[k + q]);
    }
  }
}

// Threads to a row: enough for its columns, at most `most`.
int lanes_for(int64_t width, int most = 256) {
  int lanes = 1;
  while (lanes < most && lanes * kColumns < width) lanes *= 2;
  return lanes;
}

int64_t blocks_of(int64_t width, int lanes) {
  const int64_t each = static_cast<int64_t>(lanes) * kColumns;
  return (width + each - 1) / each;
}

Spread spread_of(const TokenRows &a, const TokenRows &b) {
  return a.dtype != DT_F32 && b.dtype != DT_F32 ? OCTETS : QUADS;
}

// f(the spread as a constant)
template <class F>
hipError_t with_spread(Spread m, F &&f) {
  if (m == OCTETS) return f(std::integral_constant<Spread, OCTETS>{});
  return f(std::integral_constant<Spread, QUADS>{});
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
template <class TW, class TO, Spread M>
__global__ void __launch_bounds__(256)
embedding_rows(Tokens tokens, int64_t count, const typename TW::S *weight, int64_t vocab, int64_t width,
               int64_t weight_pitch, float scale, typename TO::S *out, int64_t out_pitch, int lanes, int64_t blocks) {
  const int groups = 256 / lanes, lane = threadIdx.x % lanes;
  const int64_t unit = group_index() * groups + threadIdx.x / lanes;
  const int64_t i = unit / blocks;
  if (i >= count) return;
  const int64_t t = tokens[i];
  const Columns c(M, unit % blocks, lane, lanes, width);
  float v[kColumns] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (t >= 0 && t < vocab) {
    load_columns<TW, M>(weight + t * weight_pitch, c, v);
#pragma unroll
    for (int k = 0; k < kColumns; ++k) v[k] = times(v[k], scale);
  }
  store_columns<TO, M>(out + i * out_pitch, c, v);
}

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
constexpr int kOnce = 6;               // tokens per thread of 1024: of the sort in one workgroup, at most
constexpr int kEach = 2;               // ... and of a tile
constexpr int kTile = kEach * 1024;
constexpr int kFewTiles = 32;          // so few are summed by every workgroup itself
constexpr int kMaxBits = 10;           // of a digit: one thread per value

// Rank of each of a workgroup's tokens among those of its digit.  A wave holds
// 64 N consecutive tokens, 64 at a time in order, so ranks keep the order.
// before[w * bins + d] becomes the number of digit d in earlier waves, *total
// (thread d) that of the whole tile.
template <int N>
__device__ __forceinline__ void tile_ranks(const uint32_t *digit, const bool *live, int bits, uint16_t *before,
                                           uint32_t *rank, uint32_t *total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = 1 << bits;
  for (int k = tid; k < 16 * bins / 2; k += 1024) reinterpret_cast<uint32_t *>(before)[k] = 0;
  __syncthreads();
  volatile uint16_t *mine = before + wave * bins;
  const uint64_t lower = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    uint64_t same = __ballot(live[j]);
#pragma unroll
    for (int b = 0; b < kMaxBits; ++b) {
      if (b >= bits) break;
      const int32_t one = static_cast<int32_t>(digit[j] << (31 - b)) >> 31;   // the bit, in every place
      const uint64_t with = __ballot(one), flip = ~static_cast<uint64_t>(static_cast<int64_t>(one));
      same &= with ^ flip;
    }
    if (live[j]) {
      const uint32_t so_far = mine[digit[j]];
      rank[j] = so_far + __popcll(same & lower);
      __builtin_amdgcn_wave_barrier();
      if ((same & lower) == 0) mine[digit[j]] = static_cast<uint16_t>(so_far + __popcll(same));
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  uint32_t sum = 0;
  if (tid < bins) {
    for (int w = 0; w < 16; ++w) {
      const uint32_t n = before[w * bins + tid];
      before[w * bins + tid] = static_cast<uint16_t>(sum);
      sum += n;
    }
  }
  *total = sum;
}

// Exclusive sum over the 1024 threads of a workgroup.  parts: 16 words.
__device__ __forceinline__ uint32_t scan_1024(uint32_t v, uint32_t *parts, uint32_t *all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t run = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t below = __shfl_up(run, d);
    if (lane >= d) run += below;
  }
  __syncthreads();                      // (parts of an earlier call are read)
  if (lane == 63) parts[wave] = run;
  __syncthreads();
  uint32_t base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    const uint32_t n = parts[w];
    base += w < wave ? n : 0;
    sum += n;
  }
  *all = sum;
  return base + run - v;
}

__device__ __forceinline__ int64_t first_not_below(const uint32_t *keys, int64_t n, uint32_t v) {
  int64_t low = 0, high = n;
  while (low < high) {
    const int64_t mid = (low + high) / 2;
    if (keys[mid] < v) low = mid + 1;
    else high = mid;
  }
  return low;
}

// Up to 1024 N tokens: all digits in one workgroup.  (4739 tokens into 2420 x 42:
// 30.0 us, 33.9 by the launches below; 8192 tokens into 32768 x 128: 35.2 and 33.9.)
template <int N>
__global__ void __launch_bounds__(1024)
token_sort_once(Tokens tokens, int count, uint32_t vocab, int passes, int bits, uint32_t *keys, uint32_t *places,
                uint32_t *joins) {
  if (threadIdx.x < 2) joins[threadIdx.x] = 0;
  __shared__ uint16_t before[16 << kMaxBits];
  __shared__ uint32_t first[1 << kMaxBits], parts[16];
  __shared__ uint32_t key_at[1024 * N];
  __shared__ uint16_t place_at[1024 * N];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int mine = wave * 64 * N + lane;
  uint32_t key[N], place[N];
  bool live[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int i = mine + 64 * j;
    live[j] = i < count;
    key[j] = live[j] ? tokens.key(i, vocab) : 0;
    place[j] = i;
  }
  for (int pass = 0; pass < passes; ++pass) {
    uint32_t digit[N], rank[N], total, all;
#pragma unroll
    for (int j = 0; j < N; ++j) digit[j] = key[j] >> (pass * bits) & ((1u << bits) - 1);
    tile_ranks<N>(digit, live, bits, before, rank, &total);
    const uint32_t at = scan_1024(tid < (1 << bits) ? total : 0, parts, &all);
    if (tid < (1 << bits)) first[tid] = at;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!live[j]) continue;
      const uint32_t to = first[digit[j]] + before[(wave << bits) + digit[j]] + rank[j];
      key_at[to] = key[j];
      place_at[to] = static_cast<uint16_t>(place[j]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!live[j]) continue;
      key[j] = key_at[mine + 64 * j];
      place[j] = place_at[mine + 64 * j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (!live[j]) continue;
    keys[mine + 64 * j] = key[j];
    places[mine + 64 * j] = place[j];
  }
}

// A pass over one digit of many tokens: how often it has each value in every
// tile (counts[value][tile]) ...
__global__ void __launch_bounds__(1024)
token_count(Tokens tokens, const uint32_t *keys, int64_t count, uint32_t vocab, int shift, int bits, uint32_t *counts) {
  __shared__ uint32_t n[1 << kMaxBits];
  const int tid = threadIdx.x;
  n[tid] = 0;
  __syncthreads();
  for (int j = 0; j < kEach; ++j) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kTile + j * 1024 + tid;
    if (i < count) atomicAdd(&n[(keys ? keys[i] : tokens.key(i, vocab)) >> shift & ((1u << bits) - 1)], 1u);
  }
  __syncthreads();
  if (tid < (1 << bits)) counts[static_cast<int64_t>(tid) * gridDim.x + blockIdx.x] = n[tid];
}

// ... the sums of those before each, in place (of few tiles the next kernel
// takes them itself, a launch less: 4.6 us) ...
__global__ void __launch_bounds__(1024) token_scan(uint32_t *counts, int64_t n) {
  __shared__ uint32_t parts[16];
  uint32_t carry = 0;
  for (int64_t at = 0; at < n; at += 4096) {
    const int64_t i = at + threadIdx.x * 4;
    uint32_t v[4], all;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = i + k < n ? counts[i + k] : 0;
    uint32_t run = carry + scan_1024(v[0] + v[1] + v[2] + v[3], parts, &all);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < n) counts[i + k] = run;
      run += v[k];
    }
    carry += all;
  }
}

// ... and every token to its place.
__global__ void __launch_bounds__(1024)
token_scatter(Tokens tokens, const uint32_t *keys, const uint32_t *places, int64_t count, uint32_t vocab, int shift,
              int bits, const uint32_t *counts, uint32_t *keys_out, uint32_t *places_out, uint32_t *joins) {
  __shared__ uint16_t before[16 << kMaxBits];
  __shared__ uint32_t first[1 << kMaxBits], parts[16];
  if (blockIdx.x == 0 && threadIdx.x < 2) joins[threadIdx.x] = 0;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kTile + wave * 64 * kEach + lane;
  uint32_t key[kEach], place[kEach], digit[kEach], rank[kEach], total;
  bool live[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int64_t i = mine + 64 * j;
    live[j] = i < count;
    key[j] = !live[j] ? 0 : keys ? keys[i] : tokens.key(i, vocab);
    place[j] = !live[j] ? 0 : keys ? places[i] : static_cast<uint32_t>(i);
    digit[j] = key[j] >> shift & ((1u << bits) - 1);
  }
  const int tiles = gridDim.x;
  if (tiles > kFewTiles) {
    if (tid < (1 << bits)) first[tid] = counts[static_cast<int64_t>(tid) * tiles + blockIdx.x];
  } else {
    uint32_t all, earlier = 0, sum = 0;
    if (tid < (1 << bits)) {
      for (int k = 0; k < tiles; ++k) {
        const uint32_t n = counts[tid * tiles + k];
        earlier += k < static_cast<int>(blockIdx.x) ? n : 0;
        sum += n;
      }
    }
    const uint32_t base = scan_1024(sum, parts, &all);
    if (tid < (1 << bits)) first[tid] = base + earlier;
  }
  tile_ranks<kEach>(digit, live, bits, before, rank, &total);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (!live[j]) continue;
    const uint32_t to = first[digit[j]] + before[(wave << bits) + digit[j]] + rank[j];
    keys_out[to] = key[j];
    places_out[to] = place[j];
  }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
struct Sums {
  const uint32_t *keys, *places;   // sorted
  int64_t count;
  uint32_t vocab;
  int64_t width, grad_pitch, weight_pitch;
  float scale;
  int accumulate;
  int piece;                       // tokens per piece
  int64_t pieces;
  int lanes;                       // threads to a row
  int64_t blocks;                  // blocks of columns
  float *partials;                 // [pieces][2][partial_pitch]
  int64_t partial_pitch;           // the width, in whole 16 bytes
  int64_t work;                    // workgroups that add rows up; those behind them clear rows ...
  int clear_rows;                  // ... so many each
  uint32_t *joins;                 // pieces with a run that begins there and reaches out: how many short ones, how
                                   // many long ones, which (the long ones from the end)
};
constexpr int kClearRows = 256;    // rows of the table per such workgroup, at most
constexpr int kShortRun = 8;       // pieces of a run that one group of threads adds up

template <class TW, Spread M>
__device__ __forceinline__ void write_row(const Sums &p, typename TW::S *weight, uint32_t v, const Columns &c,
                                          float *acc) {
  typename TW::S *row = weight + static_cast<int64_t>(v) * p.weight_pitch;
  float out[kColumns];
#pragma unroll
  for (int k = 0; k < kColumns; ++k) out[k] = times(acc[k], p.scale);
  if (p.accumulate) {
    float old[kColumns];
    load_columns<TW, M>(row, c, old);
#pragma unroll
    for (int k = 0; k < kColumns; ++k) out[k] += old[k];
  }
  store_columns<TW, M, true>(row, c, out);
}

// Partial sums: of the run that reaches into a piece (which = 0) or out of it.
__device__ __forceinline__ float *partial_row(const Sums &p, int64_t piece, int which) {
  return p.partials + (piece * 2 + which) * p.partial_pitch;
}

template <class TG, class TW, Spread M, bool WAVE>
__global__ void __launch_bounds__(256)
embedding_sums(Sums p, const typename TG::S *grad, typename TW::S *weight) {
  const int64_t group = group_index();
  if (group >= p.work) {
    if (p.accumulate) return;           // (a grid in two dimensions may have some to spare)
    __shared__ int absent[kClearRows];
    const int64_t row0 = (group - p.work) * p.clear_rows;
    if (threadIdx.x < p.clear_rows) {
      const int64_t v = row0 + threadIdx.x;
      bool none = v < p.vocab;
      if (none) {
        const int64_t at = first_not_below(p.keys, p.count, static_cast<uint32_t>(v));
        none = at == p.count || p.keys[at] != v;
      }
      absent[threadIdx.x] = none;
    }
    __syncthreads();
    const float zero[kColumns] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int r = threadIdx.x / p.lanes; r < p.clear_rows; r += 256 / p.lanes) {
      if (!absent[r]) continue;
      typename TW::S *row = weight + (row0 + r) * p.weight_pitch;
      for (int64_t b = 0; b < p.blocks; ++b)
        store_columns<TW, M, true>(row, Columns(M, b, threadIdx.x % p.lanes, p.lanes, p.width), zero);
    }
    return;
  }
  const int groups = 256 / p.lanes, lane = threadIdx.x % p.lanes;
  const int64_t unit = group * groups + threadIdx.x / p.lanes;
  const int64_t piece = unit / p.blocks;
  if (piece >= p.pieces) return;
  const Columns c(M, unit % p.blocks, lane, p.lanes, p.width);
  const int64_t begin = piece * p.piece, end = min(begin + p.piece, p.count);
  const int n = static_cast<int>(end - begin);
  // A wave that has one piece holds its tokens, one per lane, and takes them
  // from there; narrow rows' groups share waves and read them one by one.
  const int at = static_cast<int>(min<int64_t>(threadIdx.x & 63, n - 1));
  const uint32_t my_key = p.keys[begin + at], my_place = p.places[begin + at];
  const uint32_t before = begin > 0 ? p.keys[begin - 1] : p.vocab, behind = end < p.count ? p.keys[end] : p.vocab;
  auto key_of = [&](int i) -> uint32_t {
    return WAVE ? static_cast<uint32_t>(__builtin_amdgcn_readlane(my_key, i)) : p.keys[begin + min(i, n - 1)];
  };
  auto place_of = [&](int i) -> uint32_t {
    return WAVE ? static_cast<uint32_t>(__builtin_amdgcn_readlane(my_place, i)) : p.places[begin + min(i, n - 1)];
  };
  uint32_t run = key_of(0);
  bool reaches_in = before == run;
  float acc[kColumns] = {0, 0, 0, 0, 0, 0, 0, 0};
  constexpr int kAhead = 8;
  for (int i = 0; i < n; i += kAhead) {
    uint32_t key[kAhead], place[kAhead];
    float v[kAhead][kColumns];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) key[a] = key_of(i + a), place[a] = place_of(i + a);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (i + a >= n) key[a] = p.vocab;
      if (key[a] < p.vocab) load_columns<TG, M>(grad + static_cast<int64_t>(place[a]) * p.grad_pitch, c, v[a]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (key[a] != run && run < p.vocab && i + a < n) {
        if (reaches_in) store_columns<EF32, M>(partial_row(p, piece, 0), c, acc);
        else write_row<TW, M>(p, weight, run, c, acc);
        reaches_in = false;
#pragma unroll
        for (int k = 0; k < kColumns; ++k) acc[k] = 0.0f;
      }
      if (i + a < n) run = key[a];
      if (key[a] < p.vocab) {
#pragma unroll
        for (int k = 0; k < kColumns; ++k) acc[k] += v[a][k];
      }
    }
  }
  if (run >= p.vocab) return;                          // padding
  const bool reaches_out = behind == run;
  if (reaches_out && !reaches_in && lane == 0 && unit % p.blocks == 0) {
    const int64_t far = begin + static_cast<int64_t>(kShortRun) * p.piece;
    const bool is_long = far < p.count && p.keys[far] == run;
    const int64_t i = atomicAdd(p.joins + (is_long ? 1 : 0), 1u);
    p.joins[is_long ? 1 + p.pieces - i : 2 + i] = static_cast<uint32_t>(piece);
  }
  if (reaches_in || reaches_out) store_columns<EF32, M>(partial_row(p, piece, reaches_in ? 0 : 1), c, acc);
  else write_row<TW, M>(p, weight, run, c, acc);
}

// The runs that begin in a piece and reach out of it, whose number is known on
// the GPU only: workgroups take them from the lists that embedding_sums left.
// The partial sums of a run are cut into as many consecutive parts as there
// are groups of threads on a row; each group adds one up, and then the first
// those in order.  Short runs have groups as wide as the row (up to 256
// threads), long ones of kJoinLanes, so that 16 share their parts.  (10007 x
// 1531 values with a run of 370 partial sums: 98 us with wide groups only; 32768
// x 4096 with 600 short runs: 65 us with narrow groups only.)
constexpr int kJoinLanes = 16;
constexpr int kJoinGroups = 2048;

template <class TW, Spread M>
__global__ void __launch_bounds__(256) embedding_join(Sums p, typename TW::S *weight, int long_lanes, int64_t long_blocks) {
  __shared__ float sums[256][kColumns + 1];
  const int64_t n_short = p.joins[0] * p.blocks, n_long = p.joins[1] * long_blocks;
  for (int64_t item = blockIdx.x; item < n_short + n_long; item += gridDim.x) {
    const bool is_long = item < n_long;               // the longest work first
    const int lanes = is_long ? long_lanes : p.lanes, groups = 256 / lanes;
    const int64_t blocks = is_long ? long_blocks : p.blocks, i = is_long ? item : item - n_long;
    const int64_t piece = p.joins[is_long ? 1 + p.pieces - i / blocks : 2 + i / blocks];
    const uint32_t run = p.keys[(piece + 1) * p.piece - 1];
    // the pieces that begin within the run
    int64_t parts = 1;
    for (int more = 256; more == 256;) {
      const int64_t at = (piece + parts + threadIdx.x) * p.piece;
      more = __syncthreads_count(at < p.count && p.keys[at] == run);
      parts += more;
    }
    const int lane = threadIdx.x % lanes, mine = threadIdx.x / lanes;
    const Columns c(M, i % blocks, lane, lanes, p.width);
    const int used = static_cast<int>(min<int64_t>(groups, parts));     // groups with a share
    const int64_t from = parts * min(mine, used) / used, to = parts * min(mine + 1, used) / used;
    float acc[kColumns] = {0, 0, 0, 0, 0, 0, 0, 0};
    constexpr int kAhead = 8;
    for (int64_t k0 = from; k0 < to; k0 += kAhead) {
      float v[kAhead][kColumns];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (k0 + a < to) load_columns<EF32, M>(partial_row(p, piece + k0 + a, k0 + a == 0), c, v[a]);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (k0 + a >= to) continue;
#pragma unroll
        for (int k = 0; k < kColumns; ++k) acc[k] += v[a][k];
      }
    }
#pragma unroll
    for (int k = 0; k < kColumns; ++k) sums[threadIdx.x][k] = acc[k];
    __syncthreads();
    if (mine == 0) {
      for (int g = 1; g < used; ++g) {
#pragma unroll
        for (int k = 0; k < kColumns; ++k) acc[k] += sums[g * lanes + lane][k];
      }
      write_row<TW, M>(p, weight, run, c, acc);
    }
    __syncthreads();
  }
}

// Few tokens of a small vocabulary: a workgroup per row of the table and
// kJoinLanes * 8 columns.  It looks through all tokens itself, each wave
// through a quarter of them in order, and its groups of threads add up
// consecutive parts of the row's gradients, and then theirs in order.  One
// launch and no sort (us in this way and the others', bf16 into fp32 of 128 columns:
//     4096 tokens into   256         512         1024        2048        4096 rows
//     uniform            7.1  20.6   7.2  23.2   8.0  25.2   13   25     22   24
//     by falling rank    16   20     16   22     15   23     15   23     22   24
//     half of them one   47   23     47   24     48   26     49   25     52   25
//     64 tokens          5.2  13.7   5.4  11.9   5.9  12.1   8.4  12.1   13   12.5
// The tokens' frequencies are not known here: the bounds leave out sizes that
// would gain if no token were frequent, and do not shut out a token that fills
// the batch, whose row one workgroup adds up: 4096 of one into 256 rows 88 and 22.)
constexpr int kRowTokens = 4096;                       // at most: their places fit 16 KiB of LDS
constexpr int64_t kRowReads = int64_t(1) << 21;        // tokens read by all workgroups, at most
constexpr int64_t kRowGroups = 4096;                   // workgroups, at most

template <class TG, class TW, Spread M>
__global__ void __launch_bounds__(256)
embedding_row_sums(Tokens tokens, int count, Sums p, const typename TG::S *grad, typename TW::S *weight) {
  constexpr int kQuarter = kRowTokens / 4;
  __shared__ uint16_t found[4][kQuarter], list[kRowTokens];
  __shared__ int found_n[4];
  __shared__ float sums[256][kColumns + 1];
  const uint32_t v = static_cast<uint32_t>(blockIdx.x / p.blocks);
  {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int quarter = (count + 3) / 4, first = wave * quarter, end = min(first + quarter, count);
    const uint64_t lower = (uint64_t(1) << lane) - 1;
    int n = 0;
    constexpr int kRounds = kQuarter / 64;
    bool mine[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int i = first + 64 * k + lane;
      mine[k] = i < end && tokens.key(i, p.vocab) == v;
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const uint64_t with = __ballot(mine[k]);
      if (mine[k]) found[wave][n + __popcll(with & lower)] = static_cast<uint16_t>(first + 64 * k + lane);
      n += __popcll(with);
    }
    if (lane == 0) found_n[wave] = n;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w) before += found_n[w];
    for (int k = lane; k < n; k += 64) list[before + k] = found[wave][k];
    __syncthreads();
  }
  const int n = found_n[0] + found_n[1] + found_n[2] + found_n[3];
  if (n == 0 && p.accumulate) return;
  const int groups = 256 / p.lanes, lane = threadIdx.x % p.lanes, mine = threadIdx.x / p.lanes;
  const Columns c(M, blockIdx.x % p.blocks, lane, p.lanes, p.width);
  const int from = n * mine / groups, to = n * (mine + 1) / groups;
  float acc[kColumns] = {0, 0, 0, 0, 0, 0, 0, 0};
  constexpr int kAhead = 8;
  for (int i = from; i < to; i += kAhead) {
    float x[kAhead][kColumns];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (i + a < to) load_columns<TG, M>(grad + static_cast<int64_t>(list[i + a]) * p.grad_pitch, c, x[a]);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (i + a >= to) continue;
#pragma unroll
      for (int k = 0; k < kColumns; ++k) acc[k] += x[a][k];
    }
  }
#pragma unroll
  for (int k = 0; k < kColumns; ++k) sums[threadIdx.x][k] = acc[k];
  __syncthreads();
  if (mine > 0) return;
  for (int g = 1; g < groups; ++g) {
#pragma unroll
    for (int k = 0; k < kColumns; ++k) acc[k] += sums[g * p.lanes + lane][k];
  }
  write_row<TW, M>(p, weight, v, c, acc);
}

// ---------------------------------------------------------------------------
// plan of a gradient call
// ---------------------------------------------------------------------------
struct Plan {
  int passes, bits;                  // digits of the sort
  bool many;                         // more than one workgroup's
  bool by_row;                       // a workgroup per row of the table
  int64_t tiles;
  int lanes, piece;
  int64_t blocks, pieces;
  size_t keys, places, keys2, places2, counts, joins, partials, bytes;   // offsets in the workspace
};

Plan plan_of(int64_t count, int64_t vocab, int64_t width) {
  Plan p{};
  int bits = 1;
  while (vocab >> bits) ++bits;      // of 0 .. vocab, padding included
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.tiles = (count + kTile - 1) / kTile;
  p.many = count > kOnce * 1024;
  p.lanes = lanes_for(width, kJoinLanes);
  p.by_row = count <= kRowTokens &&
             vocab * blocks_of(width, p.lanes) <= std::min(kRowGroups, kRowReads / std::max<int64_t>(count, 1));
  if (!p.by_row) p.lanes = lanes_for(width);
  p.blocks = blocks_of(width, p.lanes);
  // pieces of 8 to 64 tokens (a lane each): about 1024 workgroups where there are so many
  // (32768 x 4096 tokens: 199 us, with 2048 207)
  p.piece = static_cast<int>(std::clamp<int64_t>(count * p.blocks * p.lanes / 256 / 1024, 8, 64));
  p.pieces = (count + p.piece - 1) / p.piece;
  if (p.by_row) {
    p.bytes = 0;
    return p;
  }
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.keys = take(4 * count);
  p.places = take(4 * count);
  p.keys2 = p.many ? take(4 * count) : 0;
  p.places2 = p.many ? take(4 * count) : 0;
  p.counts = p.many ? take(4 * (p.tiles << p.bits)) : 0;
  p.joins = take(4 * (2 + p.pieces));
  p.partials = take(8 * p.pieces * ((width + 3) / 4 * 4));
  p.bytes = at;
  return p;
}

}  // namespace

hipError_t launch_embedding(const void *tokens, int token_bits, int64_t count, const TokenRows &weight, int64_t vocab,
                            int64_t width, float scale, const TokenRows &out, hipStream_t s) {
  const int lanes = lanes_for(width);
  const int64_t blocks = blocks_of(width, lanes);
  const int64_t grid = (count * blocks + 256 / lanes - 1) / (256 / lanes);
  return with_type(weight.dtype, [&](auto tw) {
    return with_type(out.dtype, [&](auto to) {
      return with_spread(spread_of(weight, out), [&](auto m) {
        using TW = decltype(tw);
        using TO = decltype(to);
        embedding_rows<TW, TO, m.value><<<grid_of(grid), dim3(256), 0, s>>>(
            Tokens{tokens, token_bits}, count, static_cast<const typename TW::S *>(weight.data), vocab, width,
            weight.pitch, scale, static_cast<typename TO::S *>(out.data), out.pitch, lanes, blocks);
        return hipGetLastError();
      });
    });
  });
}

size_t embedding_grad_bytes(int64_t count, int64_t vocab, int64_t width) { return plan_of(count, vocab, width).bytes; }

hipError_t launch_embedding_grad(const void *tokens, int token_bits, int64_t count, const TokenRows &grad,
                                 int64_t vocab, int64_t width, float scale, const TokenRows &grad_weight,
                                 bool accumulate, void *workspace, hipStream_t s) {
  const Plan plan = plan_of(count, vocab, width);
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  auto words = [&](size_t at) { return reinterpret_cast<uint32_t *>(ws + at); };
  const Tokens t{tokens, token_bits};
  const uint32_t v = static_cast<uint32_t>(vocab);
  uint32_t *keys = words(plan.keys), *places = words(plan.places), *joins = words(plan.joins);
  if (plan.by_row) {
    // no sort
  } else if (!plan.many) {
    const int n = static_cast<int>(count);
    auto sort = [&](auto each) {
      token_sort_once<decltype(each)::value>
          <<<dim3(1), dim3(1024), 0, s>>>(t, n, v, plan.passes, plan.bits, keys, places, joins);
    };
    // (its time goes with the tokens per thread: 1000 into 30000 x 300 26.3 us, 29.1
    // with four of them)
    if (n <= 1024) sort(std::integral_constant<int, 1>{});
    else if (n <= 2048) sort(std::integral_constant<int, 2>{});
    else if (n <= 4096) sort(std::integral_constant<int, 4>{});
    else sort(std::integral_constant<int, kOnce>{});
  } else {
    uint32_t *keys2 = words(plan.keys2), *places2 = words(plan.places2), *counts = words(plan.counts);
    for (int pass = 0; pass < plan.passes; ++pass) {
      const uint32_t *from = pass ? keys2 : nullptr;
      const int shift = pass * plan.bits;
      token_count<<<dim3(plan.tiles), dim3(1024), 0, s>>>(t, from, count, v, shift, plan.bits, counts);
      if (plan.tiles > kFewTiles) token_scan<<<dim3(1), dim3(1024), 0, s>>>(counts, plan.tiles << plan.bits);
      token_scatter<<<dim3(plan.tiles), dim3(1024), 0, s>>>(t, from, places2, count, v, shift, plan.bits, counts, keys,
                                                           places, joins);
      if (pass + 1 < plan.passes) std::swap(keys, keys2), std::swap(places, places2);
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int groups = 256 / plan.lanes;
  const int64_t work = (plan.pieces * plan.blocks + groups - 1) / groups;
  // rows that a workgroup clears: about 32768 elements (56523 x 81: 22 us in all, 48 with eight rows)
  const int clear_rows = static_cast<int>(std::clamp<int64_t>(32768 / width, 8, kClearRows));
  Sums p{keys, places, count, v, width, grad.pitch, grad_weight.pitch, scale, accumulate ? 1 : 0, plan.piece,
         plan.pieces, plan.lanes, plan.blocks, reinterpret_cast<float *>(ws + plan.partials),
         (width + 3) / 4 * 4,
         work, clear_rows, joins};
  const int64_t clear = accumulate ? 0 : (vocab + clear_rows - 1) / clear_rows;
  const int join_lanes = lanes_for(width, kJoinLanes);
  const int64_t join_blocks = blocks_of(width, join_lanes);
  return with_type(grad.dtype, [&](auto tg) {
    return with_type(grad_weight.dtype, [&](auto tw) {
      return with_spread(spread_of(grad, grad_weight), [&](auto m) {
        using TG = decltype(tg);
        using TW = decltype(tw);
        typename TW::S *w = static_cast<typename TW::S *>(grad_weight.data);
        const typename TG::S *g = static_cast<const typename TG::S *>(grad.data);
        if (plan.by_row) {
          embedding_row_sums<TG, TW, m.value>
              <<<dim3(vocab * plan.blocks), dim3(256), 0, s>>>(t, static_cast<int>(count), p, g, w);
          return hipGetLastError();
        }
        const dim3 grid = grid_of(clear + work);
        if (plan.lanes >= 64) embedding_sums<TG, TW, m.value, true><<<grid, dim3(256), 0, s>>>(p, g, w);
        else embedding_sums<TG, TW, m.value, false><<<grid, dim3(256), 0, s>>>(p, g, w);
        if (plan.pieces > 1)
          embedding_join<TW, m.value><<<dim3(std::min<int64_t>(plan.pieces * join_blocks, kJoinGroups)), dim3(256), 0,
                                        s>>>(p, w, join_lanes, join_blocks);
        return hipGetLastError();
      });
    });
  });
}

}  // namespace gns
