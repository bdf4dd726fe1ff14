// Host side of the operators over lists of tensors (include/gns.h): building
// a list's table, argument checks and the launches.  Nothing allocates device
// memory, nothing synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/gns.h"
#include "gns_kernels.h"
#include "gns_timing.h"

namespace {

using gns::kListArrays;
using gns::kListUnit;
using gns::LaunchScope;
using gns::ListChunk;
using gns::ListEntry;
using gns::ListView;

static_assert(sizeof(gns::AdamwBias) <= GNS_ADAMW_WORKSPACE_BYTES, "room for the bias factors");
static_assert(kListArrays == GNS_LIST_MAX_ARRAYS, "header and library agree on the arrays");

constexpr int64_t kMaxCount = int64_t(1) << 20;
constexpr int64_t kMaxElements = int64_t(1) << 42;   // per list
constexpr size_t kArrivedBytes = 256;   // of the workspace: the count of finished chunks
constexpr int64_t kMaxSpan = int64_t(1) << 58;       // elements between an entry's first and last: byte
                                                     // offsets fit an int64
// What a norm leaves in the last-level cache for the pass after it (see
// chunk_part): all of its 256 MiB.  With 128, 192, 256 and 400 MB, and with
// everything read so, norm and AdamW of 67M fp32 gradients take 363, 353, 345,
// 343 and 343 us, and a norm of 1.07 GB alone 161, 162, 164, 166 and 180.
constexpr double kLastLevelCache = 256.0 * (1 << 20);

// One workgroup of 256 threads per chunk: a grid holds 2^24 of them.  Pieces
// of whole chunks are at most 2^42 / 2^23 (dense) or, with one element to a
// row, 2^42 / 2^20; the rest is at most one short chunk per entry.
constexpr int64_t kMaxChunks = (int64_t(1) << 24) - 1;

// Units per chunk: about 16384 chunks for a large list, at least 1024 units
// (8192 elements), at most 2^20 (so that offsets within a dense chunk fit 32
// bits).
int64_t chunk_units_for(int64_t units) {
  int64_t c = 1024;
  while (c * 16384 < units && c < (int64_t(1) << 20)) c *= 2;
  return c;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Shape {
  int64_t elements = 0, per_row = 0, units = 0;
  bool dense = true;   // every array contiguous: one row
};

gns_status entry_shape(const gns_tensor *tensors, int arrays, int64_t count, int64_t i, Shape *sh) {
  const gns_tensor &t = tensors[i];
  if (t.rows < 0 || t.cols < 0) return GNS_E_SHAPE;
  if (t.rows > 0 && t.cols > kMaxElements / t.rows) return GNS_E_SHAPE;
  sh->elements = t.rows * t.cols;
  for (int a = 0; a < arrays; ++a) {
    const gns_tensor &x = tensors[a * count + i];
    if (x.rows != t.rows || x.cols != t.cols) return GNS_E_SHAPE;
    if (x.dtype != GNS_F32 && x.dtype != GNS_BF16 && x.dtype != GNS_F16) return GNS_E_DTYPE;
    if (sh->elements == 0) continue;
    if (x.pitch < 0 || (x.rows > 1 && x.pitch > kMaxSpan / x.rows)) return GNS_E_SHAPE;
    if (!x.data) return GNS_E_NULL;
    if (reinterpret_cast<uintptr_t>(x.data) % gns::dtype_size(x.dtype)) return GNS_E_PARAM;
    if (x.rows > 1 && x.pitch != x.cols) sh->dense = false;
  }
  if (sh->elements == 0) {
    sh->per_row = 1;
    sh->units = 0;
  } else {
    sh->per_row = ceil_div(sh->dense ? sh->elements : t.cols, kListUnit);
    sh->units = sh->dense ? sh->per_row : t.rows * sh->per_row;
  }
  return GNS_OK;
}

struct Totals {
  int64_t elements = 0, chunk_units = 0, chunks = 0;
  size_t bytes = 0;
};

gns_status list_totals(const gns_tensor *tensors, int arrays, int64_t count, Totals *tt) {
  if ((arrays != 1 && arrays != 2 && arrays != 4 && arrays != 5) || count < 0 || count > kMaxCount)
    return GNS_E_SHAPE;
  if (count > 0 && !tensors) return GNS_E_NULL;
  int64_t units = 0;
  for (int64_t i = 0; i < count; ++i) {
    Shape sh;
    const gns_status st = entry_shape(tensors, arrays, count, i, &sh);
    if (st != GNS_OK) return st;
    tt->elements += sh.elements;
    units += sh.units;
    if (tt->elements > kMaxElements) return GNS_E_SHAPE;
  }
  tt->chunk_units = chunk_units_for(units);
  for (int64_t i = 0; i < count; ++i) {
    Shape sh;
    entry_shape(tensors, arrays, count, i, &sh);
    tt->chunks += ceil_div(sh.units, tt->chunk_units);
  }
  if (tt->chunks > kMaxChunks) return GNS_E_SHAPE;
  tt->bytes = sizeof(ListEntry) * count + sizeof(ListChunk) * tt->chunks;
  return GNS_OK;
}

// The memory of one array of one entry: rows of `width` bytes, `pitch` apart.
struct Region {
  uintptr_t begin, end;
  uint64_t width, pitch;   // pitch 0: one row
  int array;
};

// Whether two regions whose spans meet may share bytes.  Rows of the same
// pitch, as column slices of one matrix have, are compared within one period;
// anything else that interleaves counts as shared.
bool may_share(const Region &x, const Region &y) {
  const uint64_t pitch = x.pitch ? x.pitch : y.pitch;
  if (pitch == 0 || (x.pitch && y.pitch && x.pitch != y.pitch)) return true;
  const uint64_t d = (y.begin - x.begin) % pitch;   // y begins no earlier than x
  return !(x.width <= d && d + y.width <= pitch);
}

unsigned find_overlaps(const gns_tensor *tensors, int arrays, int64_t count) {
  unsigned bits = 0;
  std::vector<Region> all;
  all.reserve(static_cast<size_t>(arrays) * count);
  for (int a = 0; a < arrays; ++a) {
    for (int64_t i = 0; i < count; ++i) {
      const gns_tensor &t = tensors[a * count + i];
      if (t.rows == 0 || t.cols == 0) continue;
      const uint64_t sz = gns::dtype_size(t.dtype);
      Region r{reinterpret_cast<uintptr_t>(t.data), 0, t.cols * sz, 0, a};
      if (t.rows > 1 && t.pitch == t.cols) {
        r.width *= t.rows;
      } else if (t.rows > 1) {
        r.pitch = t.pitch * sz;
        if (t.pitch < t.cols) bits |= 1u << (kListArrays * a + a);   // rows share memory
      }
      r.end = r.begin + (t.rows > 1 && t.pitch != t.cols ? (t.rows - 1) * r.pitch : 0) + r.width;
      all.push_back(r);
    }
  }
  std::sort(all.begin(), all.end(), [](const Region &x, const Region &y) { return x.begin < y.begin; });
  for (size_t i = 0; i < all.size(); ++i) {
    for (size_t j = i + 1; j < all.size() && all[j].begin < all[i].end; ++j) {
      const int a = std::min(all[i].array, all[j].array), b = std::max(all[i].array, all[j].array);
      const unsigned bit = 1u << (kListArrays * a + b);
      if (!(bits & bit) && may_share(all[i], all[j])) bits |= bit;
    }
  }
  return bits;
}

// How many of the list's last chunks hold kLastLevelCache bytes of array 0.
int64_t chunks_at_end(const gns_tensor *grads, int64_t count, const ListEntry *entries, int64_t chunk_units) {
  double room = kLastLevelCache;
  int64_t n = 0;
  for (int64_t i = count; i-- > 0;) {
    const double each = static_cast<double>(chunk_units) * kListUnit * gns::dtype_size(grads[i].dtype);
    const int64_t fit = std::min<int64_t>(entries[i].chunks, static_cast<int64_t>(room / each));
    n += fit;
    if (fit < entries[i].chunks) break;
    room -= std::min(room, static_cast<double>(grads[i].rows) * grads[i].cols * gns::dtype_size(grads[i].dtype));
  }
  return n;
}

ListView view_of(const gns_tensor_list *l, const void *table) {
  ListView v;
  v.entries = static_cast<const ListEntry *>(table);
  v.chunks = reinterpret_cast<const ListChunk *>(v.entries + l->count);
  v.count = l->count;
  v.n_chunks = l->chunks;
  v.chunk_units = l->chunk_units;
  v.keep_from = l->keep_from;
  return v;
}

bool valid_list(const gns_tensor_list *l) {
  return (l->arrays == 1 || l->arrays == 2 || l->arrays == 4 || l->arrays == 5) && l->count >= 0 &&
         l->count <= kMaxCount && l->chunks >= 0 && l->chunks <= kMaxChunks && l->chunk_units >= 1 &&
         l->keep_from >= 0 && l->keep_from <= l->chunks &&
         l->table_bytes == sizeof(ListEntry) * l->count + sizeof(ListChunk) * l->chunks;
}

bool overlap(const gns_tensor_list *l, int a, int b) {
  return l->overlaps >> (kListArrays * std::min(a, b) + std::max(a, b)) & 1;
}

gns_status norm_and_clip(const gns_tensor_list *list, const void *table, gns_norm kind, double max_norm,
                         double eps, const float *inv_scale, float *result, float *tensor_norms,
                         void *workspace, size_t workspace_bytes, bool clip, hipStream_t s) {
  if (!list) return GNS_E_NULL;
  if (!valid_list(list)) return GNS_E_SHAPE;
  if ((kind != GNS_NORM_L2 && kind != GNS_NORM_MAX) || !(max_norm >= 0.0) || !(eps >= 0.0) || std::isinf(eps))
    return GNS_E_PARAM;
  if (!result || (list->count > 0 && !table)) return GNS_E_NULL;
  if (!workspace || workspace_bytes < gns_tensor_list_workspace_bytes(list) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GNS_E_WORKSPACE;
  const int dst = list->arrays == 2 ? 1 : 0;
  for (int a = 0; clip && a < list->arrays; ++a)
    if (overlap(list, a, dst)) return GNS_E_ALIAS;
  const ListView v = view_of(list, table);
  uint32_t *arrived = static_cast<uint32_t *>(workspace);
  uint64_t *partials = reinterpret_cast<uint64_t *>(static_cast<unsigned char *>(workspace) + kArrivedBytes);
  const double n = static_cast<double>(list->elements);
  const bool max = kind == GNS_NORM_MAX;
  const gns::NormArgs args{inv_scale, max_norm, eps, result};
  LaunchScope ls(s, clip ? "grad_clip" : "grad_norm", clip ? "list_partials+list_scale" : "list_partials",
                 (clip ? 3.0 : 2.0) * n, list->bytes[0] * (clip ? 2.0 : 1.0) + (clip ? list->bytes[dst] : 0.0));
  const hipError_t e = clip ? gns::launch_list_clip(v, dst, max, partials, arrived, args, tensor_norms, s)
                            : gns::launch_list_norm(v, max, partials, arrived, args, tensor_norms, s);
  ls.done();
  if (e != hipSuccess) return GNS_E_HIP;
  return GNS_OK;
}

// One update, the step-th or (with count) the one after *count.
gns_status adamw(const gns_tensor_list *list, const void *table, int64_t step, int64_t *count, double lr,
                 double beta1, double beta2, double eps, double weight_decay, const float *grad_scale,
                 gns::AdamwBias *bias, hipStream_t s) {
  if (!list) return GNS_E_NULL;
  if (!valid_list(list) || list->arrays < 4) return GNS_E_SHAPE;
  for (int a = 1; a <= 3; ++a)
    if (list->dtypes[a] & ~(1u << GNS_F32)) return GNS_E_DTYPE;
  if ((!count && step < 1) || !std::isfinite(lr) || !std::isfinite(weight_decay) || !(beta1 >= 0.0 && beta1 < 1.0) ||
      !(beta2 >= 0.0 && beta2 < 1.0) || !std::isfinite(eps) ||
      !(static_cast<float>(eps) > 0.0f))   // as the kernel has it: 0 / 0 where moments are zero
    return GNS_E_PARAM;
  if (list->count > 0 && !table) return GNS_E_NULL;
  for (int a = 1; a < list->arrays; ++a)
    for (int b = 0; b < list->arrays; ++b)
      if (overlap(list, a, b)) return GNS_E_ALIAS;
  gns::AdamwScalars h{};
  h.lr = lr;
  h.weight_decay = weight_decay;
  h.beta1 = static_cast<float>(beta1);
  h.one_minus_beta1 = static_cast<float>(1.0 - beta1);
  h.beta2 = static_cast<float>(beta2);
  h.one_minus_beta2 = static_cast<float>(1.0 - beta2);
  h.eps = static_cast<float>(eps);
  if (!count) {
    const double t = static_cast<double>(step);
    h.bias.bias1 = 1.0 - std::pow(beta1, t);
    h.bias.inv_sqrt_bias2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, t)));
  }
  double bytes = list->bytes[0] + list->bytes[4];
  for (int a = 1; a <= 3; ++a) bytes += 2.0 * list->bytes[a];
  LaunchScope ls(s, "adamw", count ? "adamw_count+list_adamw" : "list_adamw", 15.0 * list->elements, bytes);
  hipError_t e = count ? gns::launch_adamw_count(count, beta1, beta2, grad_scale, bias, s) : hipSuccess;
  if (e == hipSuccess)
    e = gns::launch_list_adamw(view_of(list, table), list->arrays == 5, h, count ? bias : nullptr, grad_scale, s);
  ls.done();
  return e == hipSuccess ? GNS_OK : GNS_E_HIP;
}

}  // namespace

extern "C" {

size_t gns_tensor_list_bytes(const gns_tensor *tensors, int arrays, int64_t count) {
  Totals tt;
  return list_totals(tensors, arrays, count, &tt) == GNS_OK ? std::max<size_t>(tt.bytes, 16) : 0;
}

gns_status gns_tensor_list_build(const gns_tensor *tensors, int arrays, int64_t count, const float *lr_scale,
                                 const float *wd_scale, void *table, size_t table_bytes, gns_tensor_list *list) {
  Totals tt;
  gns_status st = list_totals(tensors, arrays, count, &tt);
  if (st != GNS_OK) return st;
  if (!table || !list) return GNS_E_NULL;
  for (int64_t i = 0; i < count; ++i)
    if ((lr_scale && !std::isfinite(lr_scale[i])) || (wd_scale && !std::isfinite(wd_scale[i]))) return GNS_E_PARAM;
  if (table_bytes < tt.bytes || (reinterpret_cast<uintptr_t>(table) & 15)) return GNS_E_WORKSPACE;
  gns_tensor_list l{};
  l.arrays = arrays;
  l.count = count;
  l.elements = tt.elements;
  l.chunks = tt.chunks;
  l.chunk_units = tt.chunk_units;
  l.table_bytes = tt.bytes;
  try {
    l.overlaps = find_overlaps(tensors, arrays, count);
  } catch (const std::bad_alloc &) {
    return GNS_E_HIP;
  }
  ListEntry *entries = static_cast<ListEntry *>(table);
  ListChunk *chunks = reinterpret_cast<ListChunk *>(entries + count);
  uint32_t at = 0;
  for (int64_t i = 0; i < count; ++i) {
    Shape sh;
    entry_shape(tensors, arrays, count, i, &sh);
    ListEntry e{};
    for (int a = 0; a < arrays; ++a) {
      const gns_tensor &t = tensors[a * count + i];
      e.data[a] = t.data;
      e.pitch[a] = sh.dense ? 0 : t.pitch;
      e.dtype[a] = static_cast<uint8_t>(t.dtype);
      l.dtypes[a] |= 1u << t.dtype;
      l.bytes[a] += static_cast<double>(sh.elements) * gns::dtype_size(t.dtype);
    }
    e.cols = sh.dense ? sh.elements : tensors[i].cols;
    e.per_row = sh.per_row;
    e.units = sh.units;
    e.first_chunk = at;
    e.chunks = static_cast<uint32_t>(ceil_div(sh.units, tt.chunk_units));
    e.lr_scale = lr_scale ? lr_scale[i] : 1.0f;
    e.wd_scale = wd_scale ? wd_scale[i] : 1.0f;
    std::memcpy(entries + i, &e, sizeof(e));
    for (uint32_t c = 0; c < e.chunks; ++c) chunks[at + c] = ListChunk{static_cast<uint32_t>(i), c};
    at += e.chunks;
  }
  l.keep_from = l.chunks - chunks_at_end(tensors, count, entries, tt.chunk_units);
  *list = l;
  return GNS_OK;
}

size_t gns_tensor_list_workspace_bytes(const gns_tensor_list *list) {
  return list && valid_list(list) ? kArrivedBytes + sizeof(uint64_t) * list->chunks : 0;
}

gns_status gns_grad_norm(const gns_tensor_list *list, const void *table, gns_norm kind, double max_norm,
                         double eps, const float *inv_scale, float *result, float *tensor_norms,
                         void *workspace, size_t workspace_bytes, void *stream) {
  return norm_and_clip(list, table, kind, max_norm, eps, inv_scale, result, tensor_norms, workspace,
                       workspace_bytes, false, static_cast<hipStream_t>(stream));
}

gns_status gns_grad_clip(const gns_tensor_list *list, const void *table, gns_norm kind, double max_norm,
                         double eps, const float *inv_scale, float *result, float *tensor_norms,
                         void *workspace, size_t workspace_bytes, void *stream) {
  return norm_and_clip(list, table, kind, max_norm, eps, inv_scale, result, tensor_norms, workspace,
                       workspace_bytes, true, static_cast<hipStream_t>(stream));
}

gns_status gns_adamw_step(const gns_tensor_list *list, const void *table, int64_t step, double lr,
                          double beta1, double beta2, double eps, double weight_decay,
                          const float *grad_scale, void *stream) {
  return adamw(list, table, step, nullptr, lr, beta1, beta2, eps, weight_decay, grad_scale, nullptr,
               static_cast<hipStream_t>(stream));
}

gns_status gns_adamw_step_counted(const gns_tensor_list *list, const void *table, int64_t *count, double lr,
                                  double beta1, double beta2, double eps, double weight_decay,
                                  const float *grad_scale, void *workspace, size_t workspace_bytes,
                                  void *stream) {
  if (!count) return GNS_E_NULL;
  if (reinterpret_cast<uintptr_t>(count) % sizeof(*count)) return GNS_E_PARAM;
  if (!workspace || workspace_bytes < GNS_ADAMW_WORKSPACE_BYTES || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return GNS_E_WORKSPACE;
  return adamw(list, table, 0, count, lr, beta1, beta2, eps, weight_decay, grad_scale,
               static_cast<gns::AdamwBias *>(workspace), static_cast<hipStream_t>(stream));
}

}  // extern "C"
