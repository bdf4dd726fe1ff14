// Token embedding and its gradient, written for CDNA4 (gfx950).
//
// * embedding_rows   -- out[i] = scale weight[tokens[i]]: HBM-bound, 8
//                       elements per thread in 16-byte accesses.
// * token_sort_once, token_count, token_scan, token_scatter
//                    -- a stable sort of the tokens by radix, with the
//                       position of each: up to 4096 tokens in one workgroup,
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

#include "gns_elem.h"
#include "gns_kernels.h"

namespace gns {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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
// a thread has eight columns: eight consecutive ones where rows begin on 16
// bytes (WIDE), else every lanes-th, so that a group's accesses stay together.
constexpr int kColumns = 8;

struct Columns {
  int64_t first;      // the thread's first column
  int step;           // to its next one
  int n;              // how many it has
};

template <bool WIDE>
__device__ __forceinline__ Columns columns_of(int64_t block, int lane, int lanes, int64_t width) {
  const int64_t base = block * lanes * kColumns;
  Columns c;
  c.first = base + (WIDE ? lane * kColumns : lane);
  c.step = WIDE ? 1 : lanes;
  const int64_t left = width - c.first;
  c.n = left <= 0 ? 0 : static_cast<int>(min<int64_t>(kColumns, WIDE ? left : (left + lanes - 1) / lanes));
  return c;
}

// (a row's last piece may be short; the others are whole and take 16-byte accesses)
template <class T, bool WIDE>
__device__ __forceinline__ void load_columns(const typename T::S *row, const Columns &c, float *v) {
  using S = typename T::S;
  if (WIDE && c.n == kColumns) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(row + c.first);
    if constexpr (sizeof(S) == 4) {
      const u32x4 a = p[0], b = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
      const u32x4 a = p[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = T::ld(static_cast<S>(a[i] & 0xffff));
        v[2 * i + 1] = T::ld(static_cast<S>(a[i] >> 16));
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kColumns; ++i) v[i] = i < c.n ? T::ld(row[c.first + i * c.step]) : 0.0f;
}

template <class T, bool WIDE>
__device__ __forceinline__ void store_columns(typename T::S *row, const Columns &c, const float *v) {
  using S = typename T::S;
  if (WIDE && c.n == kColumns) {
    u32x4 *p = reinterpret_cast<u32x4 *>(row + c.first);
    if constexpr (sizeof(S) == 4) {
      u32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __float_as_uint(v[i]);
        b[i] = __float_as_uint(v[4 + i]);
      }
      p[0] = a;
      p[1] = b;
    } else {
      u32x4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = T::st2(v[2 * i], v[2 * i + 1]);
      p[0] = a;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kColumns; ++i)
    if (i < c.n) row[c.first + i * c.step] = T::st(v[i]);
}

// Threads to a row: enough for its columns, at most a workgroup.
int lanes_for(int64_t width) {
  int lanes = 1;
  while (lanes < 256 && lanes * kColumns < width) lanes *= 2;
  return lanes;
}

bool wide_rows(const TokenRows &r) {
  const int64_t elem = dtype_size(r.dtype);
  return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.pitch * elem % 16 == 0;
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
template <class TW, class TO, bool WIDE>
__global__ void __launch_bounds__(256)
embedding_rows(Tokens tokens, int64_t count, const typename TW::S *weight, int64_t vocab, int64_t width,
               int64_t weight_pitch, float scale, typename TO::S *out, int64_t out_pitch, int lanes, int64_t blocks) {
  const int groups = 256 / lanes, lane = threadIdx.x % lanes;
  const int64_t unit = group_index() * groups + threadIdx.x / lanes;
  const int64_t i = unit / blocks;
  if (i >= count) return;
  const int64_t t = tokens[i];
  const Columns c = columns_of<WIDE>(unit % blocks, lane, lanes, width);
  float v[kColumns] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (t >= 0 && t < vocab) {
    load_columns<TW, WIDE>(weight + t * weight_pitch, c, v);
#pragma unroll
    for (int k = 0; k < kColumns; ++k) v[k] = times(v[k], scale);
  }
  store_columns<TO, WIDE>(out + i * out_pitch, c, v);
}

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
constexpr int kTile = 4096;            // tokens per workgroup of 1024 threads
constexpr int kEach = kTile / 1024;
constexpr int kMaxBits = 10;           // of a digit: one thread per value

// Rank of each of a tile's tokens among those of its digit.  Wave w holds
// tokens 256 w .. 256 w + 255, 64 at a time in order, so ranks keep the order.
// before[w * bins + d] becomes the number of digit d in earlier waves, *total
// (thread d) that of the whole tile.
__device__ __forceinline__ void tile_ranks(const uint32_t *digit, const bool *live, int bits, uint16_t *before,
                                           uint32_t *rank, uint32_t *total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = 1 << bits;
  for (int k = tid; k < 16 * bins / 2; k += 1024) reinterpret_cast<uint32_t *>(before)[k] = 0;
  __syncthreads();
  volatile uint16_t *mine = before + wave * bins;
  const uint64_t lower = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    uint64_t same = __ballot(live[j]);
    for (int b = 0; b < bits; ++b) {
      const bool one = digit[j] >> b & 1;
      const uint64_t with = __ballot(one);
      same &= one ? with : ~with;
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

// Up to kTile tokens: all digits in one workgroup.
__global__ void __launch_bounds__(1024)
token_sort_once(Tokens tokens, int count, uint32_t vocab, int passes, int bits, uint32_t *keys, uint32_t *places) {
  __shared__ uint16_t before[16 << kMaxBits];
  __shared__ uint32_t first[1 << kMaxBits], parts[16];
  __shared__ uint32_t key_at[kTile], place_at[kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int mine = wave * 64 * kEach + lane;
  uint32_t key[kEach], place[kEach];
  bool live[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = mine + 64 * j;
    live[j] = i < count;
    key[j] = live[j] ? tokens.key(i, vocab) : 0;
    place[j] = i;
  }
  for (int pass = 0; pass < passes; ++pass) {
    uint32_t digit[kEach], rank[kEach], total, all;
#pragma unroll
    for (int j = 0; j < kEach; ++j) digit[j] = key[j] >> (pass * bits) & ((1u << bits) - 1);
    tile_ranks(digit, live, bits, before, rank, &total);
    const uint32_t at = scan_1024(tid < (1 << bits) ? total : 0, parts, &all);
    if (tid < (1 << bits)) first[tid] = at;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (!live[j]) continue;
      const uint32_t to = first[digit[j]] + before[(wave << bits) + digit[j]] + rank[j];
      key_at[to] = key[j];
      place_at[to] = place[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (!live[j]) continue;
      key[j] = key_at[mine + 64 * j];
      place[j] = place_at[mine + 64 * j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
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

// ... the sums of those before each, in place ...
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
              int bits, const uint32_t *counts, uint32_t *keys_out, uint32_t *places_out) {
  __shared__ uint16_t before[16 << kMaxBits];
  __shared__ uint32_t first[1 << kMaxBits];
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
  if (tid < (1 << bits)) first[tid] = counts[static_cast<int64_t>(tid) * gridDim.x + blockIdx.x];
  tile_ranks(digit, live, bits, before, rank, &total);
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
  float *partials;                 // [pieces][2][width]: of the run that reaches in, of the one that reaches out
  int64_t clear_groups;            // workgroups that clear rows
};
constexpr int kClearRows = 16;     // rows of the table per such workgroup

__device__ __forceinline__ int64_t first_not_below(const uint32_t *keys, int64_t n, uint32_t v) {
  int64_t low = 0, high = n;
  while (low < high) {
    const int64_t mid = (low + high) / 2;
    if (keys[mid] < v) low = mid + 1;
    else high = mid;
  }
  return low;
}

template <class TW, bool WIDE>
__device__ __forceinline__ void write_row(const Sums &p, typename TW::S *weight, uint32_t v, const Columns &c,
                                          float *acc) {
  typename TW::S *row = weight + static_cast<int64_t>(v) * p.weight_pitch;
  float out[kColumns];
#pragma unroll
  for (int k = 0; k < kColumns; ++k) out[k] = times(acc[k], p.scale);
  if (p.accumulate) {
    float old[kColumns];
    load_columns<TW, WIDE>(row, c, old);
#pragma unroll
    for (int k = 0; k < kColumns; ++k) out[k] += old[k];
  }
  store_columns<TW, WIDE>(row, c, out);
}

__device__ __forceinline__ void write_partial(const Sums &p, int64_t piece, int which, const Columns &c,
                                              const float *acc) {
  float *row = p.partials + (piece * 2 + which) * p.width;
#pragma unroll
  for (int k = 0; k < kColumns; ++k)
    if (k < c.n) row[c.first + k * c.step] = acc[k];
}

template <class TG, class TW, bool WIDE>
__global__ void __launch_bounds__(256)
embedding_sums(Sums p, const typename TG::S *grad, typename TW::S *weight) {
  const int64_t group = group_index();
  if (group < p.clear_groups) {
    __shared__ int absent[kClearRows];
    const int64_t row0 = group * kClearRows;
    if (threadIdx.x < kClearRows) {
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
    for (int r = 0; r < kClearRows; ++r) {
      if (!absent[r]) continue;
      typename TW::S *row = weight + (row0 + r) * p.weight_pitch;
      for (int64_t b = 0; b * 256 * kColumns < p.width; ++b)
        store_columns<TW, WIDE>(row, columns_of<WIDE>(b, threadIdx.x, 256, p.width), zero);
    }
    return;
  }
  const int groups = 256 / p.lanes, lane = threadIdx.x % p.lanes;
  const int64_t unit = (group - p.clear_groups) * groups + threadIdx.x / p.lanes;
  const int64_t piece = unit / p.blocks;
  if (piece >= p.pieces) return;
  const Columns c = columns_of<WIDE>(unit % p.blocks, lane, p.lanes, p.width);
  const int64_t begin = piece * p.piece, end = min(begin + p.piece, p.count);
  uint32_t run = p.keys[begin];
  bool reaches_in = begin > 0 && p.keys[begin - 1] == run;
  float acc[kColumns] = {0, 0, 0, 0, 0, 0, 0, 0};
  constexpr int kAhead = 4;
  for (int64_t i = begin; i < end; i += kAhead) {
    uint32_t key[kAhead];
    float v[kAhead][kColumns];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const bool in = i + a < end;
      key[a] = in ? p.keys[i + a] : p.vocab;
      if (key[a] < p.vocab) load_columns<TG, WIDE>(grad + static_cast<int64_t>(p.places[i + a]) * p.grad_pitch, c, v[a]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (key[a] != run && run < p.vocab && i + a < end) {
        if (reaches_in) write_partial(p, piece, 0, c, acc);
        else write_row<TW, WIDE>(p, weight, run, c, acc);
        reaches_in = false;
#pragma unroll
        for (int k = 0; k < kColumns; ++k) acc[k] = 0.0f;
      }
      if (i + a < end) run = key[a];
      if (key[a] < p.vocab) {
#pragma unroll
        for (int k = 0; k < kColumns; ++k) acc[k] += v[a][k];
      }
    }
  }
  if (run >= p.vocab) return;                          // padding
  const bool reaches_out = end < p.count && p.keys[end] == run;
  if (reaches_in || reaches_out) write_partial(p, piece, reaches_in ? 0 : 1, c, acc);
  else write_row<TW, WIDE>(p, weight, run, c, acc);
}

// The runs that begin in a piece and reach out of it.
template <class TW, bool WIDE>
__global__ void __launch_bounds__(256) embedding_join(Sums p, typename TW::S *weight) {
  const int groups = 256 / p.lanes, lane = threadIdx.x % p.lanes;
  const int64_t unit = group_index() * groups + threadIdx.x / p.lanes;
  const int64_t piece = unit / p.blocks, begin = piece * p.piece, end = begin + p.piece;
  if (piece >= p.pieces || end >= p.count) return;
  const uint32_t run = p.keys[end - 1];
  if (run >= p.vocab || p.keys[end] != run) return;
  if (p.keys[begin] == run && begin > 0 && p.keys[begin - 1] == run) return;
  const int64_t last = (first_not_below(p.keys, p.count, run + 1) - 1) / p.piece;
  const Columns c = columns_of<WIDE>(unit % p.blocks, lane, p.lanes, p.width);
  float acc[kColumns];
  load_columns<EF32, false>(p.partials + (piece * 2 + 1) * p.width, c, acc);
  constexpr int kAhead = 4;
  for (int64_t i = piece + 1; i <= last; i += kAhead) {
    float v[kAhead][kColumns];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (i + a <= last) load_columns<EF32, false>(p.partials + (i + a) * 2 * p.width, c, v[a]);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (i + a > last) continue;
#pragma unroll
      for (int k = 0; k < kColumns; ++k) acc[k] += v[a][k];
    }
  }
  write_row<TW, WIDE>(p, weight, run, c, acc);
}

// ---------------------------------------------------------------------------
// plan of a gradient call
// ---------------------------------------------------------------------------
struct Plan {
  int passes, bits;                  // digits of the sort
  int64_t tiles;
  int lanes, piece;
  int64_t blocks, pieces;
  size_t keys, places, keys2, places2, counts, partials, bytes;   // offsets in the workspace
};

Plan plan_of(int64_t count, int64_t vocab, int64_t width) {
  Plan p;
  int bits = 1;
  while (vocab >> bits) ++bits;      // of 0 .. vocab, padding included
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.tiles = (count + kTile - 1) / kTile;
  p.lanes = lanes_for(width);
  p.blocks = (width + static_cast<int64_t>(p.lanes) * kColumns - 1) / (p.lanes * kColumns);
  // pieces of 8 to 64 tokens: about a thousand workgroups where there are so many
  p.piece = static_cast<int>(std::clamp<int64_t>(count * p.blocks * p.lanes / 256 / 1024, 8, 64));
  p.pieces = (count + p.piece - 1) / p.piece;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.keys = take(4 * count);
  p.places = take(4 * count);
  p.keys2 = p.tiles > 1 ? take(4 * count) : 0;
  p.places2 = p.tiles > 1 ? take(4 * count) : 0;
  p.counts = p.tiles > 1 ? take(4 * (p.tiles << p.bits)) : 0;
  p.partials = take(8 * p.pieces * width);
  p.bytes = at;
  return p;
}

}  // namespace

hipError_t launch_embedding(const void *tokens, int token_bits, int64_t count, const TokenRows &weight, int64_t vocab,
                            int64_t width, float scale, const TokenRows &out, hipStream_t s) {
  const int lanes = lanes_for(width);
  const int64_t blocks = (width + static_cast<int64_t>(lanes) * kColumns - 1) / (lanes * kColumns);
  const int64_t grid = (count * blocks + 256 / lanes - 1) / (256 / lanes);
  const bool wide = wide_rows(weight) && wide_rows(out);
  return with_type(weight.dtype, [&](auto tw) {
    return with_type(out.dtype, [&](auto to) {
      using TW = decltype(tw);
      using TO = decltype(to);
      auto run = [&](auto kernel) {
        kernel<<<grid_of(grid), dim3(256), 0, s>>>(Tokens{tokens, token_bits}, count,
                                               static_cast<const typename TW::S *>(weight.data), vocab, width,
                                               weight.pitch, scale, static_cast<typename TO::S *>(out.data), out.pitch,
                                               lanes, blocks);
        return hipGetLastError();
      };
      return wide ? run(embedding_rows<TW, TO, true>) : run(embedding_rows<TW, TO, false>);
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
  uint32_t *keys = words(plan.keys), *places = words(plan.places);
  if (plan.tiles == 1) {
    token_sort_once<<<dim3(1), dim3(1024), 0, s>>>(t, static_cast<int>(count), v, plan.passes, plan.bits, keys, places);
  } else if (plan.tiles > 1) {
    uint32_t *keys2 = words(plan.keys2), *places2 = words(plan.places2), *counts = words(plan.counts);
    for (int pass = 0; pass < plan.passes; ++pass) {
      const uint32_t *from = pass ? keys2 : nullptr;
      const int shift = pass * plan.bits;
      token_count<<<dim3(plan.tiles), dim3(1024), 0, s>>>(t, from, count, v, shift, plan.bits, counts);
      token_scan<<<dim3(1), dim3(1024), 0, s>>>(counts, plan.tiles << plan.bits);
      token_scatter<<<dim3(plan.tiles), dim3(1024), 0, s>>>(t, from, places2, count, v, shift, plan.bits, counts, keys,
                                                           places);
      if (pass + 1 < plan.passes) std::swap(keys, keys2), std::swap(places, places2);
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  Sums p{keys, places, count, v, width, grad.pitch, grad_weight.pitch, scale, accumulate ? 1 : 0, plan.piece,
         plan.pieces, plan.lanes, plan.blocks, reinterpret_cast<float *>(ws + plan.partials),
         accumulate ? 0 : (vocab + kClearRows - 1) / kClearRows};
  const int groups = 256 / plan.lanes;
  const int64_t work = (plan.pieces * plan.blocks + groups - 1) / groups;
  const bool wide = wide_rows(grad) && wide_rows(grad_weight);
  return with_type(grad.dtype, [&](auto tg) {
    return with_type(grad_weight.dtype, [&](auto tw) {
      using TG = decltype(tg);
      using TW = decltype(tw);
      auto run = [&](auto sums, auto join) {
        const typename TG::S *g = static_cast<const typename TG::S *>(grad.data);
        typename TW::S *w = static_cast<typename TW::S *>(grad_weight.data);
        if (p.clear_groups + work > 0) sums<<<grid_of(p.clear_groups + work), dim3(256), 0, s>>>(p, g, w);
        if (plan.pieces > 1) join<<<grid_of(work), dim3(256), 0, s>>>(p, w);
        return hipGetLastError();
      };
      return wide ? run(embedding_sums<TG, TW, true>, embedding_join<TW, true>)
                  : run(embedding_sums<TG, TW, false>, embedding_join<TW, false>);
    });
  });
}

}  // namespace gns
