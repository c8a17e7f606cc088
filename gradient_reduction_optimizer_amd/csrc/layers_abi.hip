// C-ABI entry points of the layers: lookups, the sort of positions by row, the
// lookup's gradient, experts' products.  They keep nothing between calls; every
// check happens on the host before the first launch.
#include <hip/hip_runtime.h>

#include <limits>

#include "host.h"
#include "layers.h"

using namespace gro;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;  // of one matrix, with its strides

uint64_t up256(uint64_t n) { return (n + 255) / 256 * 256; }

int64_t elem_bytes(const gro_matrix& m) { return m.type == GRO_FP32 ? 4 : 2; }

int check_matrix(const gro_matrix* m, const char* what) {
  if (m == nullptr) return set_error(GRO_E_INVALID, "%s is NULL", what);
  if (m->type != GRO_BF16 && m->type != GRO_FP32) return set_error(GRO_E_INVALID, "%s: unknown type %d", what, m->type);
  if (m->reserved != 0) return set_error(GRO_E_INVALID, "%s: nonzero reserved field", what);
  if (m->rows < 0 || m->cols < 0 || m->rows > kMaxIds || m->cols > kMaxIds || m->stride < 0 || m->stride > kMaxElems)
    return set_error(GRO_E_INVALID, "%s: %lld x %lld elements, stride %lld", what, (long long)m->rows,
                     (long long)m->cols, (long long)m->stride);
  if (m->rows > 1 && m->stride < m->cols)
    return set_error(GRO_E_INVALID, "%s: rows of %lld elements %lld apart overlap", what, (long long)m->cols,
                     (long long)m->stride);
  if (m->rows > 0 && m->rows * double(m->stride) > double(kMaxElems))
    return set_error(GRO_E_INVALID, "%s: too large", what);
  if (m->rows == 0 || m->cols == 0) return GRO_OK;
  if (m->data == nullptr || !aligned_to(m->data, uintptr_t(elem_bytes(*m))))
    return set_error(GRO_E_INVALID, "%s: data is NULL or not aligned to its elements", what);
  return GRO_OK;
}

Matrix device_matrix(const gro_matrix& m) {
  return Matrix{m.data, m.rows, m.cols, m.stride, m.type == GRO_FP32 ? 1 : 0};
}

// Bytes from a first to a last element, and where they lie: `count` blocks of `bytes`
// each, `step` bytes apart.
struct Area {
  uintptr_t at;
  uint64_t count, bytes, step;
  uint64_t span() const { return count == 0 || bytes == 0 ? 0 : (count - 1) * step + bytes; }
};

Area area_of(const gro_matrix& m) {
  const uint64_t b = uint64_t(elem_bytes(m));
  return Area{reinterpret_cast<uintptr_t>(m.data), uint64_t(m.rows), uint64_t(m.cols) * b, uint64_t(m.stride) * b};
}

Area area_of(const void* p, uint64_t bytes) { return Area{reinterpret_cast<uintptr_t>(p), 1, bytes, bytes}; }

// Whether two areas have a byte in common.  Columns of one matrix beside each other
// (blocks equally far apart) have none.
bool overlap(const Area& a, const Area& b) {
  const uint64_t x = a.span(), y = b.span();
  if (x == 0 || y == 0 || a.at + x <= b.at || b.at + y <= a.at) return false;
  if (a.count > 1 && b.count > 1 && a.step == b.step) {
    const uint64_t apart = a.at <= b.at ? (b.at - a.at) % a.step : a.step - 1 - (a.at - b.at - 1) % a.step;
    return apart < a.bytes || a.step - apart < b.bytes;
  }
  return true;
}

int check_apart(const Area& written, const char* what, const Area& other, const char* with) {
  if (overlap(written, other)) return set_error(GRO_E_INVALID, "%s and %s overlap", what, with);
  return GRO_OK;
}

int check_array(const void* p, uint64_t count, uintptr_t bytes, const char* what) {
  if (count > 0 && (p == nullptr || !aligned_to(p, bytes)))
    return set_error(GRO_E_INVALID, "%s is NULL or not aligned to its elements", what);
  return GRO_OK;
}

int check_ids(const void* ids, int32_t type, int64_t n, int64_t first, int64_t n_rows) {
  if (type != GRO_INT32 && type != GRO_INT64) return set_error(GRO_E_INVALID, "unknown type of ids %d", type);
  if (n < 0 || n > kMaxIds) return set_error(GRO_E_INVALID, "%lld ids", (long long)n);
  if (n_rows < 0 || n_rows > kMaxTableRows)
    return set_error(GRO_E_INVALID, "%lld rows (at most %lld)", (long long)n_rows, (long long)kMaxTableRows);
  if (first < 0 || first > std::numeric_limits<int64_t>::max() - n_rows)
    return set_error(GRO_E_INVALID, "first_row %lld", (long long)first);
  return check_array(ids, uint64_t(n), type == GRO_INT64 ? 8 : 4, "d_ids");
}

uint64_t id_bytes(int32_t type, int64_t n) { return uint64_t(n) * (type == GRO_INT64 ? 8 : 4); }

int check_workspace(const void* ws, uint64_t bytes, uint64_t need) {
  if (need == 0) return GRO_OK;
  if (ws == nullptr || !aligned_to(ws, 256)) return set_error(GRO_E_INVALID, "workspace must be 256-byte aligned");
  if (bytes < need)
    return set_error(GRO_E_INVALID, "workspace has %llu bytes, the call needs %llu", (unsigned long long)bytes,
                     (unsigned long long)need);
  return GRO_OK;
}

// Where the arrays of a sort's workspace lie; none is needed up to kSortTile ids.
struct SortWorkspace {
  uint64_t pairs = 0, counts = 0, bases = 0, total = 0;
  int64_t chunk = 0;
  int32_t n_chunks = 0, n_buckets = 0;
};
SortWorkspace sort_workspace(int64_t n, int64_t n_rows) {
  SortWorkspace w;
  if (n <= kSortTile) return w;
  const int bits = bucket_bits(n, n_rows);
  w.n_buckets = int32_t(std::max<int64_t>(1, (n_rows + (int64_t(1) << bits) - 1) >> bits));
  w.chunk = sort_chunk(n);
  w.n_chunks = int32_t((n + w.chunk - 1) / w.chunk);
  w.counts = bits > 0 ? up256(uint64_t(n) * 8) : 0;
  // chunks as short as the shorter lists' that a caller may sort in the same workspace
  const uint64_t chunks = uint64_t(std::min<int64_t>((n + kSortChunk - 1) / kSortChunk, kMaxSortChunks));
  w.bases = w.counts + up256(chunks * uint64_t(w.n_buckets) * 4);
  w.total = w.bases + up256(uint64_t(w.n_buckets + 1) * 4);
  return w;
}

uint64_t grad_workspace(int64_t n, int64_t cols) {
  // as many runs as any list of up to n ids has
  const int64_t runs = n < kRunsFrom ? 0 : std::min<int64_t>(n / kShortRun, kMaxRuns);
  return up256(uint64_t(runs) * uint64_t((cols + 7) / 8 * 8) * 4);
}

int check_sizes(int64_t n, int64_t other, const uint64_t* bytes, const char* what) {
  if (bytes == nullptr) return set_error(GRO_E_INVALID, "bytes is NULL");
  if (n < 0 || n > kMaxIds) return set_error(GRO_E_INVALID, "%lld ids", (long long)n);
  if (other < 0 || other > kMaxIds) return set_error(GRO_E_INVALID, "%lld %s", (long long)other, what);
  return GRO_OK;
}

// ------------------------------------------------------------ experts' products
int check_weights(const gro_experts* w, const char* what) {
  if (w == nullptr) return set_error(GRO_E_INVALID, "%s is NULL", what);
  const gro_matrix one = {w->data, w->outer, w->inner, w->stride, w->type, w->reserved};
  if (w->n_experts < 0 || w->n_experts > GRO_MAX_EXPERTS)
    return set_error(GRO_E_INVALID, "%s: %d experts (at most %d)", what, w->n_experts, GRO_MAX_EXPERTS);
  gro_matrix m = one;
  if (w->n_experts == 0) m.rows = 0;
  const int rc = check_matrix(&m, what);
  if (rc != GRO_OK) return rc;
  const int64_t span = w->outer == 0 || w->inner == 0 ? 0 : (w->outer - 1) * w->stride + w->inner;
  if (w->expert_stride < 0 || (w->n_experts > 1 && w->expert_stride < span))
    return set_error(GRO_E_INVALID, "%s: matrices of %lld elements %lld apart overlap", what, (long long)span,
                     (long long)w->expert_stride);
  if (w->n_experts * double(w->expert_stride) > double(kMaxElems)) return set_error(GRO_E_INVALID, "%s: too large", what);
  return GRO_OK;
}

Area area_of(const gro_experts& w) {
  const uint64_t b = w.type == GRO_FP32 ? 4 : 2;
  const uint64_t span = w.outer == 0 || w.inner == 0 ? 0 : uint64_t((w.outer - 1) * w.stride + w.inner) * b;
  const uint64_t n = uint64_t(w.n_experts);
  return Area{reinterpret_cast<uintptr_t>(w.data), n, span, uint64_t(w.expert_stride) * b};
}

int check_bf16(int32_t type, const char* what) {
  if (type != GRO_BF16) return set_error(GRO_E_INVALID, "%s: the products take BF16", what);
  return GRO_OK;
}

// FP32 sums of a product in parts.
uint64_t parts_workspace(int parts, int64_t elems) { return parts > 1 ? up256(uint64_t(parts) * uint64_t(elems) * 4) : 0; }

// Forward (mode kForward: from inner to outer) and input gradient (the other way).
int run_product(const gro_matrix* in, const gro_experts* w, const int32_t* starts, const gro_matrix* out, void* d_workspace,
                uint64_t bytes, ExpertsMode mode, const char* in_name, const char* out_name, void* stream) {
  clear_error();
  int rc = check_matrix(in, in_name);
  if (rc == GRO_OK) rc = check_weights(w, "weights");
  if (rc == GRO_OK) rc = check_matrix(out, out_name);
  if (rc == GRO_OK) rc = check_bf16(in->type, in_name);
  if (rc == GRO_OK) rc = check_bf16(w->type, "weights");
  if (rc == GRO_OK) rc = check_array(starts, 1, 4, "d_starts");
  if (rc != GRO_OK) return rc;
  const int64_t from = mode == kForward ? w->inner : w->outer, to = mode == kForward ? w->outer : w->inner;
  if (in->rows != out->rows || in->cols != from || out->cols != to)
    return set_error(GRO_E_INVALID, "%s is %lld x %lld and %s %lld x %lld with weights of %lld x %lld", in_name,
                     (long long)in->rows, (long long)in->cols, out_name, (long long)out->rows, (long long)out->cols,
                     (long long)w->outer, (long long)w->inner);
  const int parts = experts_parts(mode, w->n_experts, in->rows, w->inner, w->outer);
  const uint64_t need = parts_workspace(parts, in->rows * to);
  rc = check_workspace(d_workspace, bytes, need);
  const Area ws = area_of(d_workspace, need);
  if (rc == GRO_OK) rc = check_apart(area_of(*out), out_name, area_of(*in), in_name);
  if (rc == GRO_OK) rc = check_apart(area_of(*out), out_name, area_of(*w), "the weights");
  const Area runs = area_of(starts, uint64_t(w->n_experts + 1) * 4);
  if (rc == GRO_OK) rc = check_apart(area_of(*out), out_name, runs, "d_starts");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", area_of(*out), out_name);
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", area_of(*in), in_name);
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", area_of(*w), "the weights");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", runs, "d_starts");
  if (rc != GRO_OK) return rc;
  ExpertsLaunch a = {};
  a.a = static_cast<const uint16_t*>(in->data);
  a.b = static_cast<const uint16_t*>(w->data);
  a.c = out->data;
  a.a_stride = in->stride;
  a.b_stride = w->stride;
  a.c_stride = out->stride;
  a.b_expert = w->expert_stride;
  a.starts = starts;
  a.n_experts = w->n_experts;
  a.rows = in->rows;
  a.inner = w->inner;
  a.outer = w->outer;
  a.c_fp32 = out->type == GRO_FP32;
  a.n_parts = parts;
  a.partials = static_cast<float*>(d_workspace);
  a.c_part = in->rows * to;
  if (experts_tiles(a, mode) > kMaxExpertsTiles) return set_error(GRO_E_INVALID, "product of too many tiles");
  const hipError_t e = launch_experts(a, mode, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GRO_OK : hip_fail(e, "experts' product launch");
}

}  // namespace

extern "C" int gro_row_sort_workspace(int64_t n, int64_t n_rows, uint64_t* bytes) {
  clear_error();
  const int rc = check_sizes(n, n_rows, bytes, "rows");
  if (rc != GRO_OK) return rc;
  if (n_rows > kMaxTableRows)
    return set_error(GRO_E_INVALID, "%lld rows (at most %lld)", (long long)n_rows, (long long)kMaxTableRows);
  *bytes = sort_workspace(n, n_rows).total;
  return GRO_OK;
}

extern "C" int gro_row_sort(const void* d_ids, int32_t id_type, int64_t n, int64_t first_row, int64_t n_rows,
                            int32_t* d_order, int32_t* d_starts, void* d_workspace, uint64_t bytes, void* stream) {
  clear_error();
  int rc = check_ids(d_ids, id_type, n, first_row, n_rows);
  if (rc == GRO_OK) rc = check_array(d_order, uint64_t(n), 4, "d_order");
  if (rc == GRO_OK) rc = check_array(d_starts, 1, 4, "d_starts");
  if (rc != GRO_OK) return rc;
  const SortWorkspace w = sort_workspace(n, n_rows);
  rc = check_workspace(d_workspace, bytes, w.total);
  if (rc != GRO_OK) return rc;
  const Area ids = area_of(d_ids, id_bytes(id_type, n)), order = area_of(d_order, uint64_t(n) * 4),
             starts = area_of(d_starts, uint64_t(n_rows + 1) * 4), ws = area_of(d_workspace, w.total);
  rc = check_apart(order, "d_order", ids, "d_ids");
  if (rc == GRO_OK) rc = check_apart(starts, "d_starts", ids, "d_ids");
  if (rc == GRO_OK) rc = check_apart(order, "d_order", starts, "d_starts");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", ids, "d_ids");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", order, "d_order");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", starts, "d_starts");
  if (rc != GRO_OK) return rc;
  char* at = static_cast<char*>(d_workspace);
  RowSortLaunch a = {};
  a.ids = d_ids;
  a.wide_ids = id_type == GRO_INT64;
  a.n = n;
  a.first = first_row;
  a.n_rows = n_rows;
  a.order = d_order;
  a.starts = d_starts;
  if (w.total > 0) {
    a.pairs = reinterpret_cast<uint32_t*>(at + w.pairs);
    a.counts = reinterpret_cast<uint32_t*>(at + w.counts);
    a.bases = reinterpret_cast<uint32_t*>(at + w.bases);
    a.n_chunks = w.n_chunks;
    a.n_buckets = w.n_buckets;
    a.chunk = w.chunk;
  }
  const hipError_t e = launch_row_sort(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GRO_OK : hip_fail(e, "row sort launch");
}

extern "C" int gro_lookup(const gro_matrix* table, int64_t first_row, const void* d_ids, int32_t id_type, double scale,
                          const gro_matrix* out, void* stream) {
  clear_error();
  int rc = check_matrix(table, "table");
  if (rc == GRO_OK) rc = check_matrix(out, "out");
  if (rc == GRO_OK) rc = check_ids(d_ids, id_type, out->rows, first_row, table->rows);
  if (rc != GRO_OK) return rc;
  if (table->cols != out->cols)
    return set_error(GRO_E_INVALID, "rows of %lld elements from a table of %lld", (long long)out->cols,
                     (long long)table->cols);
  rc = check_apart(area_of(*out), "out", area_of(*table), "the table");
  if (rc == GRO_OK) rc = check_apart(area_of(*out), "out", area_of(d_ids, id_bytes(id_type, out->rows)), "d_ids");
  if (rc != GRO_OK) return rc;
  LookupLaunch a = {};
  a.table = device_matrix(*table);
  a.first = first_row;
  a.ids = d_ids;
  a.wide_ids = id_type == GRO_INT64;
  a.scale = float(scale);
  a.out = device_matrix(*out);
  const hipError_t e = launch_lookup(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GRO_OK : hip_fail(e, "lookup launch");
}

extern "C" int gro_lookup_grad_workspace(int64_t n, int64_t cols, uint64_t* bytes) {
  clear_error();
  const int rc = check_sizes(n, cols, bytes, "columns");
  if (rc != GRO_OK) return rc;
  *bytes = grad_workspace(n, cols);
  return GRO_OK;
}

extern "C" int gro_lookup_grad(const gro_matrix* dy, const int32_t* d_order, const int32_t* d_starts, double scale,
                               int32_t accumulate, const gro_matrix* out, void* d_workspace, uint64_t bytes,
                               void* stream) {
  clear_error();
  int rc = check_matrix(dy, "dy");
  if (rc == GRO_OK) rc = check_matrix(out, "out");
  if (rc == GRO_OK) rc = check_array(d_order, uint64_t(dy->rows), 4, "d_order");
  if (rc == GRO_OK) rc = check_array(d_starts, 1, 4, "d_starts");
  if (rc != GRO_OK) return rc;
  if (dy->cols != out->cols)
    return set_error(GRO_E_INVALID, "rows of %lld elements for a table of %lld", (long long)dy->cols,
                     (long long)out->cols);
  if (out->rows > kMaxTableRows)
    return set_error(GRO_E_INVALID, "%lld rows (at most %lld)", (long long)out->rows, (long long)kMaxTableRows);
  if (out->cols > kMaxGradCols)
    return set_error(GRO_E_INVALID, "%lld columns (at most %lld)", (long long)out->cols, (long long)kMaxGradCols);
  if (accumulate != 0 && accumulate != 1) return set_error(GRO_E_INVALID, "accumulate is 0 or 1");
  const uint64_t need = grad_workspace(dy->rows, dy->cols);
  rc = check_workspace(d_workspace, bytes, need);
  if (rc != GRO_OK) return rc;
  const Area o = area_of(*out), ws = area_of(d_workspace, need), order = area_of(d_order, uint64_t(dy->rows) * 4),
             starts = area_of(d_starts, uint64_t(out->rows + 1) * 4);
  rc = check_apart(o, "out", area_of(*dy), "dy");
  if (rc == GRO_OK) rc = check_apart(o, "out", order, "d_order");
  if (rc == GRO_OK) rc = check_apart(o, "out", starts, "d_starts");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", o, "out");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", area_of(*dy), "dy");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", order, "d_order");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", starts, "d_starts");
  if (rc != GRO_OK) return rc;
  LookupGradLaunch a = {};
  a.dy = device_matrix(*dy);
  a.order = d_order;
  a.starts = d_starts;
  a.scale = float(scale);
  a.accumulate = accumulate;
  a.out = device_matrix(*out);
  a.partials = static_cast<float*>(d_workspace);
  a.run = run_tokens(dy->rows);
  a.n_runs = whole_runs(dy->rows);
  const hipError_t e = launch_lookup_grad(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GRO_OK : hip_fail(e, "lookup gradient launch");
}

extern "C" int gro_experts_workspace(int32_t n_experts, int64_t rows, int64_t inner, int64_t outer, uint64_t* bytes) {
  clear_error();
  const int rc = check_sizes(rows, inner, bytes, "columns");
  if (rc != GRO_OK) return rc;
  if (n_experts < 0 || n_experts > GRO_MAX_EXPERTS || outer < 0 || outer > kMaxIds ||
      double(n_experts) * double(inner) * double(outer) > double(kMaxElems) ||
      double(rows) * double(std::max(inner, outer)) > double(kMaxElems))
    return set_error(GRO_E_INVALID, "%d experts of %lld x %lld, %lld rows", n_experts, (long long)outer, (long long)inner,
                     (long long)rows);
  const auto need = [&](ExpertsMode mode, int64_t elems) {
    return parts_workspace(experts_parts(mode, n_experts, rows, inner, outer), elems);
  };
  *bytes = std::max(std::max(need(kForward, rows * outer), need(kInputGrad, rows * inner)),
                    need(kWeightGrad, n_experts * outer * inner));
  return GRO_OK;
}

extern "C" int gro_experts_forward(const gro_matrix* x, const gro_experts* weights, const int32_t* d_starts,
                                   const gro_matrix* y, void* d_workspace, uint64_t bytes, void* stream) {
  return run_product(x, weights, d_starts, y, d_workspace, bytes, kForward, "x", "y", stream);
}

extern "C" int gro_experts_input_grad(const gro_matrix* dy, const gro_experts* weights, const int32_t* d_starts,
                                      const gro_matrix* dx, void* d_workspace, uint64_t bytes, void* stream) {
  return run_product(dy, weights, d_starts, dx, d_workspace, bytes, kInputGrad, "dy", "dx", stream);
}

extern "C" int gro_experts_weight_grad(const gro_matrix* dy, const gro_matrix* x, const int32_t* d_starts,
                                       int32_t accumulate, const gro_experts* dw, void* d_workspace, uint64_t bytes,
                                       void* stream) {
  clear_error();
  int rc = check_matrix(dy, "dy");
  if (rc == GRO_OK) rc = check_matrix(x, "x");
  if (rc == GRO_OK) rc = check_weights(dw, "dw");
  if (rc == GRO_OK) rc = check_bf16(dy->type, "dy");
  if (rc == GRO_OK) rc = check_bf16(x->type, "x");
  if (rc == GRO_OK) rc = check_array(d_starts, 1, 4, "d_starts");
  if (rc != GRO_OK) return rc;
  if (dy->rows != x->rows || dy->cols != dw->outer || x->cols != dw->inner)
    return set_error(GRO_E_INVALID, "dy is %lld x %lld and x %lld x %lld with weights of %lld x %lld",
                     (long long)dy->rows, (long long)dy->cols, (long long)x->rows, (long long)x->cols,
                     (long long)dw->outer, (long long)dw->inner);
  if (accumulate != 0 && accumulate != 1) return set_error(GRO_E_INVALID, "accumulate is 0 or 1");
  const int parts = experts_parts(kWeightGrad, dw->n_experts, dy->rows, dw->inner, dw->outer);
  const int64_t elems = dw->n_experts * dw->outer * dw->inner;
  const uint64_t need = parts_workspace(parts, elems);
  rc = check_workspace(d_workspace, bytes, need);
  if (rc != GRO_OK) return rc;
  const Area o = area_of(*dw), ws = area_of(d_workspace, need),
             starts = area_of(d_starts, uint64_t(dw->n_experts + 1) * 4);
  rc = check_apart(o, "dw", area_of(*dy), "dy");
  if (rc == GRO_OK) rc = check_apart(o, "dw", area_of(*x), "x");
  if (rc == GRO_OK) rc = check_apart(o, "dw", starts, "d_starts");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", o, "dw");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", area_of(*dy), "dy");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", area_of(*x), "x");
  if (rc == GRO_OK) rc = check_apart(ws, "the workspace", starts, "d_starts");
  if (rc != GRO_OK) return rc;
  ExpertsLaunch a = {};
  a.a = static_cast<const uint16_t*>(dy->data);
  a.b = static_cast<const uint16_t*>(x->data);
  a.c = dw->data;
  a.a_stride = dy->stride;
  a.b_stride = x->stride;
  a.c_stride = dw->stride;
  a.c_expert = dw->expert_stride;
  a.starts = d_starts;
  a.n_experts = dw->n_experts;
  a.rows = dy->rows;
  a.inner = dw->inner;
  a.outer = dw->outer;
  a.c_fp32 = dw->type == GRO_FP32;
  a.accumulate = accumulate;
  a.partials = static_cast<float*>(d_workspace);
  a.n_parts = parts;
  a.c_part = elems;
  if (experts_tiles(a, kWeightGrad) > kMaxExpertsTiles) return set_error(GRO_E_INVALID, "product of too many tiles");
  const hipError_t e = launch_experts(a, kWeightGrad, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GRO_OK : hip_fail(e, "experts' weight gradient launch");
}
