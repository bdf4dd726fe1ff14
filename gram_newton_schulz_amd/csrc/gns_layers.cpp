// Host side of the token embedding and of the MXFP4 layers (include/gns.h):
// argument checks and the launches.  Nothing allocates device memory, nothing
// synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/gns.h"
#include "gns_kernels.h"
#include "gns_timing.h"

namespace {

using gns::LaunchScope;
using gns::MxMatrix;

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxVocab = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxWidth = int64_t(1) << 24;
// The product addresses a panel of 256 rows of codes with 32 bits.
constexpr int64_t kMaxAxis = int64_t(1) << 23;
constexpr int64_t kMaxElements = int64_t(1) << 42;
constexpr int64_t kMaxSpan = int64_t(1) << 56;       // elements: byte offsets fit an int64

bool valid_dtype(gns_dtype d) { return d == GNS_F32 || d == GNS_BF16 || d == GNS_F16; }
bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Memory of an argument: rows of `width` bytes, `pitch` apart (0: one row).
struct Region {
  uintptr_t begin = 0, end = 0;
  uint64_t width = 0, pitch = 0;
};

Region bytes_at(const void *p, uint64_t n) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return p && n ? Region{b, b + n, n, 0} : Region{};
}

Region rows_at(const void *p, int64_t batch, int64_t rows, int64_t cols, int64_t pitch, int64_t batch_stride,
               int elem) {
  if (!p || batch == 0 || rows == 0 || cols == 0) return Region{};
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  const uint64_t last = (batch - 1) * batch_stride + (rows - 1) * pitch + cols;
  const bool periodic = pitch > cols && (batch == 1 || batch_stride % pitch == 0);
  return Region{b, b + last * elem, static_cast<uint64_t>(cols) * elem,
                periodic ? static_cast<uint64_t>(pitch) * elem : 0};
}

// Whether two arguments may share bytes.  Column slices of one matrix (rows of
// the same pitch) are compared within one period; other spans that meet count
// as shared.
bool meet(const Region &a, const Region &b) {
  if (a.begin >= b.end || b.begin >= a.end) return false;
  if (a.pitch == 0 || a.pitch != b.pitch) return true;
  const Region &x = a.begin <= b.begin ? a : b, &y = a.begin <= b.begin ? b : a;
  const uint64_t d = (y.begin - x.begin) % x.pitch;
  return !(x.width <= d && d + y.width <= x.pitch);
}

// ---------------------------------------------------------------------------
// embedding
// ---------------------------------------------------------------------------
struct EmbeddingSizes {
  const void *tokens;
  int token_bits;
  int64_t count, vocab, width;
  int token_bytes() const { return token_bits / 8; }
};

bool embedding_size(int64_t count, int64_t vocab, int64_t width) {
  return count >= 0 && count <= kMaxTokens && vocab >= 0 && vocab <= kMaxVocab && width >= 0 && width <= kMaxWidth &&
         (width == 0 || std::max(count, vocab) <= kMaxElements / width);
}

gns_status check_embedding(const EmbeddingSizes &z, const void *table, gns_dtype table_dtype, int64_t table_pitch,
                           const void *rows, gns_dtype rows_dtype, int64_t rows_pitch, double scale,
                           bool table_written) {
  if (!embedding_size(z.count, z.vocab, z.width) || table_pitch < 0 || rows_pitch < 0 || table_pitch > kMaxSpan / kMaxVocab ||
      rows_pitch > kMaxSpan / kMaxTokens)
    return GNS_E_SHAPE;
  if ((table_written ? z.vocab : z.count) > 1 && (table_written ? table_pitch : rows_pitch) < z.width)
    return GNS_E_SHAPE;
  if (!valid_dtype(table_dtype) || !valid_dtype(rows_dtype)) return GNS_E_DTYPE;
  if ((z.token_bits != 32 && z.token_bits != 64) || !std::isfinite(scale) ||
      !std::isfinite(static_cast<float>(scale)))
    return GNS_E_PARAM;
  if (z.width > 0) {
    if (z.count > 0 && (!z.tokens || !rows)) return GNS_E_NULL;
    if (z.vocab > 0 && !table) return GNS_E_NULL;
  }
  if (!aligned(z.tokens, z.token_bytes()) || !aligned(table, gns::dtype_size(table_dtype)) ||
      !aligned(rows, gns::dtype_size(rows_dtype)))
    return GNS_E_PARAM;
  return GNS_OK;
}

// ---------------------------------------------------------------------------
// MXFP4
// ---------------------------------------------------------------------------
bool mx_size(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 0 || rows < 0 || cols < 0 || rows > kMaxAxis || cols > kMaxAxis || batch > kMaxElements) return false;
  const int64_t each = (rows + 31) / 32 * 32 * ((cols + 127) / 128 * 128);
  return each == 0 || batch <= kMaxElements / each;
}

MxMatrix mx_of(const gns_mxfp4 *q) {
  return q ? MxMatrix{static_cast<uint8_t *>(q->codes), static_cast<uint8_t *>(q->scales), q->batch, q->rows, q->cols}
           : MxMatrix{};
}

gns_status check_mx(const MxMatrix &q) {
  if (!mx_size(q.batch, q.rows, q.cols)) return GNS_E_SHAPE;
  if (q.batch == 0 || q.rows == 0 || q.cols == 0) return GNS_OK;
  if (!q.codes || !q.scales) return GNS_E_NULL;
  return aligned(q.codes, 16) && aligned(q.scales, 16) ? GNS_OK : GNS_E_PARAM;
}

// 128 x 128 tiles of a matrix, as an upper bound on workgroups
bool grid_fits(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t each = ((rows + 127) / 128) * ((cols + 127) / 128);
  return each == 0 || batch <= ((int64_t(1) << 24) - 1) / each;
}

bool strides_ok(int64_t batch, int64_t rows, int64_t pitch, int64_t batch_stride) {
  return pitch >= 0 && batch_stride >= 0 && pitch <= kMaxSpan / std::max<int64_t>(rows, 1) &&
         batch_stride <= kMaxSpan / std::max<int64_t>(batch, 1);
}

gns_status check_out(const gns::MxOutput &o, gns_dtype dtype, int64_t batch, int64_t m, int64_t n, int accumulate) {
  if (!valid_dtype(dtype)) return GNS_E_DTYPE;
  if (!strides_ok(batch, m, o.pitch, o.batch_stride) || (m > 1 && o.pitch < n)) return GNS_E_SHAPE;
  if (batch > 1 && m > 0) {
    // matrices one behind the other, or their rows beside one another
    const bool behind = o.batch_stride >= (m - 1) * o.pitch + n;
    const bool beside = o.batch_stride >= n && o.pitch >= (batch - 1) * o.batch_stride + n;
    if (!behind && !beside) return GNS_E_SHAPE;
  }
  if (accumulate != 0 && accumulate != 1) return GNS_E_PARAM;
  if (batch == 0 || m == 0 || n == 0) return GNS_OK;
  if (!o.out) return GNS_E_NULL;
  return aligned(o.out, gns::dtype_size(dtype)) ? GNS_OK : GNS_E_PARAM;
}

bool workspace_ok(const void *ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && aligned(ws, 256));
}

double mx_bytes(const MxMatrix &q) { return static_cast<double>(q.code_bytes()) + q.scale_bytes(); }

size_t round_256(size_t n) { return (n + 255) & ~size_t(255); }

gns_status product(const MxMatrix &a, const MxMatrix &b, const gns::MxOutput &o, void *workspace, hipStream_t s) {
  const double m = a.rows, n = b.rows, each = gns::dtype_size(o.dtype);
  LaunchScope ls(s, "mxfp4_matmul", "mx_gemm", 2.0 * a.batch * m * n * a.cols,
                 mx_bytes(a) + mx_bytes(b) + a.batch * m * n * each * (o.accumulate ? 2 : 1));
  const hipError_t e = gns::launch_mx_matmul(a, b, o, workspace, s);
  ls.done();
  return e == hipSuccess ? GNS_OK : GNS_E_HIP;
}

}  // namespace

extern "C" {

gns_status gns_embedding(const void *tokens, int token_bits, int64_t count, const void *weight,
                         gns_dtype weight_dtype, int64_t vocab, int64_t width, int64_t weight_pitch, double scale,
                         void *out, gns_dtype out_dtype, int64_t out_pitch, void *stream) {
  const EmbeddingSizes z{tokens, token_bits, count, vocab, width};
  const gns_status st = check_embedding(z, weight, weight_dtype, weight_pitch, out, out_dtype, out_pitch, scale, false);
  if (st != GNS_OK) return st;
  if (count == 0 || width == 0) return GNS_OK;
  const Region written = rows_at(out, 1, count, width, out_pitch, 0, gns::dtype_size(out_dtype));
  if (meet(written, rows_at(weight, 1, vocab, width, weight_pitch, 0, gns::dtype_size(weight_dtype))) ||
      meet(written, bytes_at(tokens, count * z.token_bytes())))
    return GNS_E_ALIAS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double n = static_cast<double>(count) * width;
  LaunchScope ls(s, "embedding", "embedding_rows", n,
                 n * (gns::dtype_size(weight_dtype) + gns::dtype_size(out_dtype)) + count * z.token_bytes());
  const hipError_t e = gns::launch_embedding(
      tokens, token_bits, count, gns::TokenRows{const_cast<void *>(weight), weight_dtype, weight_pitch}, vocab, width,
      static_cast<float>(scale), gns::TokenRows{out, out_dtype, out_pitch}, s);
  ls.done();
  return e == hipSuccess ? GNS_OK : GNS_E_HIP;
}

size_t gns_embedding_grad_workspace_bytes(int64_t count, int64_t vocab, int64_t width) {
  if (!embedding_size(count, vocab, width)) return 0;
  return round_256(gns::embedding_grad_bytes(count, vocab, width));
}

gns_status gns_embedding_grad(const void *tokens, int token_bits, int64_t count, const void *grad,
                              gns_dtype grad_dtype, int64_t grad_pitch, int64_t vocab, int64_t width, double scale,
                              void *grad_weight, gns_dtype grad_weight_dtype, int64_t grad_weight_pitch,
                              int accumulate, void *workspace, size_t workspace_bytes, void *stream) {
  const EmbeddingSizes z{tokens, token_bits, count, vocab, width};
  const gns_status st = check_embedding(z, grad_weight, grad_weight_dtype, grad_weight_pitch, grad, grad_dtype,
                                        grad_pitch, scale, true);
  if (st != GNS_OK) return st;
  if (accumulate != 0 && accumulate != 1) return GNS_E_PARAM;
  const size_t need = gns_embedding_grad_workspace_bytes(count, vocab, width);
  if (!workspace_ok(workspace, workspace_bytes, need)) return GNS_E_WORKSPACE;
  if (vocab == 0 || width == 0 || (count == 0 && accumulate)) return GNS_OK;
  const int ge = gns::dtype_size(grad_dtype), we = gns::dtype_size(grad_weight_dtype);
  const Region written = rows_at(grad_weight, 1, vocab, width, grad_weight_pitch, 0, we);
  const Region scratch = bytes_at(workspace, need);
  const Region read[] = {rows_at(grad, 1, count, width, grad_pitch, 0, ge), bytes_at(tokens, count * z.token_bytes())};
  if (meet(written, scratch)) return GNS_E_ALIAS;
  for (const Region &r : read)
    if (meet(written, r) || meet(scratch, r)) return GNS_E_ALIAS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double n = static_cast<double>(count) * width;
  LaunchScope ls(s, "embedding_grad", "embedding_sums", n,
                 n * ge + static_cast<double>(accumulate ? 2 * std::min(count, vocab) : vocab) * width * we);
  const hipError_t e = gns::launch_embedding_grad(
      tokens, token_bits, count, gns::TokenRows{const_cast<void *>(grad), grad_dtype, grad_pitch}, vocab, width,
      static_cast<float>(scale), gns::TokenRows{grad_weight, grad_weight_dtype, grad_weight_pitch}, accumulate != 0,
      workspace, s);
  ls.done();
  return e == hipSuccess ? GNS_OK : GNS_E_HIP;
}

size_t gns_mxfp4_code_bytes(int64_t batch, int64_t rows, int64_t cols) {
  return mx_size(batch, rows, cols) ? MxMatrix{nullptr, nullptr, batch, rows, cols}.code_bytes() : 0;
}

size_t gns_mxfp4_scale_bytes(int64_t batch, int64_t rows, int64_t cols) {
  return mx_size(batch, rows, cols) ? MxMatrix{nullptr, nullptr, batch, rows, cols}.scale_bytes() : 0;
}

gns_status gns_mxfp4_quantize(const void *x, gns_dtype dtype, int64_t pitch, int64_t batch_stride,
                              const uint8_t *noise, const gns_mxfp4 *by_rows, const gns_mxfp4 *by_columns,
                              void *stream) {
  if (!by_rows && !by_columns) return GNS_E_NULL;
  const MxMatrix r = mx_of(by_rows), c = mx_of(by_columns);
  gns_status st = GNS_OK;
  if (by_rows && (st = check_mx(r)) != GNS_OK) return st;
  if (by_columns && (st = check_mx(c)) != GNS_OK) return st;
  if (by_rows && by_columns && (r.batch != c.batch || r.rows != c.cols || r.cols != c.rows)) return GNS_E_SHAPE;
  const int64_t batch = by_rows ? r.batch : c.batch, rows = by_rows ? r.rows : c.cols,
                cols = by_rows ? r.cols : c.rows;
  if (!grid_fits(batch, rows, cols) || !strides_ok(batch, rows, pitch, batch_stride)) return GNS_E_SHAPE;
  if (!valid_dtype(dtype)) return GNS_E_DTYPE;
  if (batch == 0 || rows == 0 || cols == 0) return GNS_OK;
  if (!x) return GNS_E_NULL;
  const int elem = gns::dtype_size(dtype);
  if (!aligned(x, elem)) return GNS_E_PARAM;
  const Region in = rows_at(x, batch, rows, cols, pitch, batch_stride, elem);
  const Region bytes = bytes_at(noise, batch * rows * cols);
  const Region out[] = {bytes_at(r.codes, by_rows ? r.code_bytes() : 0), bytes_at(r.scales, by_rows ? r.scale_bytes() : 0),
                        bytes_at(c.codes, by_columns ? c.code_bytes() : 0),
                        bytes_at(c.scales, by_columns ? c.scale_bytes() : 0)};
  for (int i = 0; i < 4; ++i) {
    if (meet(out[i], in) || meet(out[i], bytes)) return GNS_E_ALIAS;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return GNS_E_ALIAS;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double n = static_cast<double>(batch) * rows * cols;
  LaunchScope ls(s, "mxfp4_quantize", "mx_quantize", 4.0 * n,
                 n * (elem + (noise ? 1 : 0)) + (by_rows ? mx_bytes(r) : 0.0) + (by_columns ? mx_bytes(c) : 0.0));
  const hipError_t e =
      gns::launch_mx_quantize(gns::MxInput{x, dtype, pitch, batch_stride, noise}, batch, rows, cols, r, c, s);
  ls.done();
  return e == hipSuccess ? GNS_OK : GNS_E_HIP;
}

gns_status gns_mxfp4_dequantize(const gns_mxfp4 *q, void *out, gns_dtype dtype, void *stream) {
  if (!q) return GNS_E_NULL;
  const MxMatrix m = mx_of(q);
  const gns_status st = check_mx(m);
  if (st != GNS_OK) return st;
  if (!valid_dtype(dtype)) return GNS_E_DTYPE;
  if (!grid_fits(m.batch, m.rows, m.cols)) return GNS_E_SHAPE;
  if (m.batch == 0 || m.rows == 0 || m.cols == 0) return GNS_OK;
  if (!out) return GNS_E_NULL;
  if (!aligned(out, gns::dtype_size(dtype))) return GNS_E_PARAM;
  const uint64_t n = static_cast<uint64_t>(m.batch) * m.rows * m.cols;
  const Region written = bytes_at(out, n * gns::dtype_size(dtype));
  if (meet(written, bytes_at(m.codes, m.code_bytes())) || meet(written, bytes_at(m.scales, m.scale_bytes())))
    return GNS_E_ALIAS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  LaunchScope ls(s, "mxfp4_dequantize", "mx_dequantize", static_cast<double>(n),
                 mx_bytes(m) + static_cast<double>(n) * gns::dtype_size(dtype));
  const hipError_t e = gns::launch_mx_dequantize(m, out, dtype, s);
  ls.done();
  return e == hipSuccess ? GNS_OK : GNS_E_HIP;
}

size_t gns_mxfp4_matmul_workspace_bytes(int64_t batch, int64_t m, int64_t n, int64_t k) {
  if (!mx_size(batch, m, k) || !mx_size(batch, n, k) || !grid_fits(batch, m, n)) return 0;
  return round_256(gns::mx_matmul_bytes(batch, m, n, k));
}

gns_status gns_mxfp4_matmul(const gns_mxfp4 *a, const gns_mxfp4 *b, void *out, gns_dtype out_dtype, int64_t out_pitch,
                            int64_t out_batch_stride, int accumulate, void *workspace, size_t workspace_bytes,
                            void *stream) {
  if (!a || !b) return GNS_E_NULL;
  const MxMatrix ma = mx_of(a), mb = mx_of(b);
  gns_status st = check_mx(ma);
  if (st == GNS_OK) st = check_mx(mb);
  if (st != GNS_OK) return st;
  if (ma.batch != mb.batch || ma.cols != mb.cols || !grid_fits(ma.batch, ma.rows, mb.rows)) return GNS_E_SHAPE;
  const gns::MxOutput o{out, out_dtype, out_pitch, out_batch_stride, accumulate == 1};
  st = check_out(o, out_dtype, ma.batch, ma.rows, mb.rows, accumulate);
  if (st != GNS_OK) return st;
  const size_t need = gns_mxfp4_matmul_workspace_bytes(ma.batch, ma.rows, mb.rows, ma.cols);
  if (!workspace_ok(workspace, workspace_bytes, need)) return GNS_E_WORKSPACE;
  if (ma.batch == 0 || ma.rows == 0 || mb.rows == 0 || (ma.cols == 0 && accumulate)) return GNS_OK;
  const Region written = rows_at(out, ma.batch, ma.rows, mb.rows, out_pitch, out_batch_stride, gns::dtype_size(out_dtype));
  const Region scratch = bytes_at(workspace, need);
  if (meet(written, scratch)) return GNS_E_ALIAS;
  for (const MxMatrix &q : {ma, mb})
    for (const Region &r : {bytes_at(q.codes, q.code_bytes()), bytes_at(q.scales, q.scale_bytes())})
      if (meet(written, r) || meet(scratch, r)) return GNS_E_ALIAS;
  return product(ma, mb, o, workspace, static_cast<hipStream_t>(stream));
}

size_t gns_mxfp4_linear_workspace_bytes(int64_t batch, int64_t m, int64_t n, int64_t k) {
  if (!mx_size(batch, m, k) || !mx_size(batch, n, k) || !grid_fits(batch, m, n)) return 0;
  if (gns::mx_linear_quantizes(batch, m, n, k)) return 0;
  return round_256(gns_mxfp4_code_bytes(batch, m, k)) + round_256(gns_mxfp4_scale_bytes(batch, m, k)) +
         gns_mxfp4_matmul_workspace_bytes(batch, m, n, k);
}

gns_status gns_mxfp4_linear(const void *x, gns_dtype dtype, int64_t pitch, int64_t batch_stride, int64_t m,
                            const gns_mxfp4 *w, void *out, gns_dtype out_dtype, int64_t out_pitch,
                            int64_t out_batch_stride, int accumulate, void *workspace, size_t workspace_bytes,
                            void *stream) {
  if (!w) return GNS_E_NULL;
  const MxMatrix mw = mx_of(w);
  gns_status st = check_mx(mw);
  if (st != GNS_OK) return st;
  const int64_t batch = mw.batch, n = mw.rows, k = mw.cols;
  if (!mx_size(batch, m, k) || !grid_fits(batch, m, n) || !grid_fits(batch, m, k) ||
      !strides_ok(batch, m, pitch, batch_stride))
    return GNS_E_SHAPE;
  if (!valid_dtype(dtype)) return GNS_E_DTYPE;
  const gns::MxOutput o{out, out_dtype, out_pitch, out_batch_stride, accumulate == 1};
  st = check_out(o, out_dtype, batch, m, n, accumulate);
  if (st != GNS_OK) return st;
  const size_t need = gns_mxfp4_linear_workspace_bytes(batch, m, n, k);
  if (!workspace_ok(workspace, workspace_bytes, need)) return GNS_E_WORKSPACE;
  if (batch == 0 || m == 0 || n == 0 || (k == 0 && accumulate)) return GNS_OK;
  if (k > 0 && !x) return GNS_E_NULL;
  const int elem = gns::dtype_size(dtype);
  if (!aligned(x, elem)) return GNS_E_PARAM;
  const Region written = rows_at(out, batch, m, n, out_pitch, out_batch_stride, gns::dtype_size(out_dtype));
  const Region scratch = bytes_at(workspace, need);
  if (meet(written, scratch)) return GNS_E_ALIAS;
  for (const Region &r : {rows_at(x, batch, m, k, pitch, batch_stride, elem), bytes_at(mw.codes, mw.code_bytes()),
                          bytes_at(mw.scales, mw.scale_bytes())})
    if (meet(written, r) || meet(scratch, r)) return GNS_E_ALIAS;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const gns::MxInput in{x, dtype, pitch, batch_stride, nullptr};
  if (gns::mx_linear_quantizes(batch, m, n, k)) {
    const double each = static_cast<double>(batch) * m;
    LaunchScope ls(s, "mxfp4_matmul", "mx_thin", 2.0 * each * n * k,
                   each * k * elem + mx_bytes(mw) + each * n * gns::dtype_size(out_dtype) * (accumulate ? 2 : 1));
    const hipError_t e = gns::launch_mx_linear(in, m, mw, o, s);
    ls.done();
    return e == hipSuccess ? GNS_OK : GNS_E_HIP;
  }
  uint8_t *at = static_cast<uint8_t *>(workspace);
  MxMatrix q{at, nullptr, batch, m, k};
  q.scales = at + round_256(q.code_bytes());
  if (k > 0) {
    const double each = static_cast<double>(batch) * m * k;
    LaunchScope ls(s, "mxfp4_quantize", "mx_quantize", 4.0 * each, each * elem + mx_bytes(q));
    const hipError_t e =
        gns::launch_mx_quantize(in, batch, m, k, q, MxMatrix{}, s);
    ls.done();
    if (e != hipSuccess) return GNS_E_HIP;
  }
  return product(q, mw, o, q.scales + round_256(q.scale_bytes()), s);
}

}  // extern "C"
