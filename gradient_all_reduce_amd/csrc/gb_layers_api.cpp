// gb_layers_api.cpp — the C ABI of the token-sum layers (include/gbreduce.h):
// argument validation and launch.  Nothing is enqueued unless every argument
// is valid; no call allocates device memory.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "gb_internal.h"
#include "gb_layers.h"
#include "gb_overlap.h"

namespace {

gb_status fail(gb_status s, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return gb::fail_status(s, msg);
}

gb_status from_hip(hipError_t e, const char* what) {
  if (e == hipSuccess) return GB_OK;
  return fail(GB_ERR_HIP, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool half_or_f32(int dtype) { return dtype == GB_DTYPE_F32 || dtype == GB_DTYPE_F16 || dtype == GB_DTYPE_BF16; }
size_t elem_size(int dtype) {
  if (dtype == GB_DTYPE_I64) return 8;
  return dtype == GB_DTYPE_F32 || dtype == GB_DTYPE_I32 ? 4 : 2;
}

gb_status check_type(int dtype, const char* fn, const char* name) {
  if (half_or_f32(dtype)) return GB_OK;
  return fail(GB_ERR_UNSUPPORTED, "%s: %s = %d is not float32, float16 or bfloat16", fn, name, dtype);
}

// A buffer of n values, which may be absent if `needed` is false.
gb_status check_pointer(const void* p, size_t align, bool needed, const char* fn, const char* name) {
  if (p == nullptr) return needed ? fail(GB_ERR_INVALID_ARG, "%s: %s is NULL", fn, name) : GB_OK;
  if (!aligned(p, align)) return fail(GB_ERR_MISALIGNED, "%s: %s = %p is not %zu-byte aligned", fn, name, p, align);
  return GB_OK;
}

// The stride of a rows x cols array: its extent stays within GB_MAX_N values,
// and rows that are written lie apart (those of an input may repeat).
gb_status check_stride(size_t stride, size_t rows, size_t cols, bool written, const char* fn, const char* name) {
  if (written && rows > 1 && stride < cols) {
    return fail(GB_ERR_INVALID_ARG, "%s: %s = %zu is less than the %zu values of a row", fn, name, stride, cols);
  }
  if (rows > 1 && stride > GB_MAX_N / rows) {
    return fail(GB_ERR_INVALID_ARG, "%s: %zu rows %zu apart (%s) exceed GB_MAX_N = %zu values", fn, rows, stride, name,
                GB_MAX_N);
  }
  return GB_OK;
}
gb_status check_shape(size_t rows, size_t cols, const char* fn, const char* rows_name, const char* cols_name) {
  if (cols > 0 && rows > GB_MAX_N / cols) {
    return fail(GB_ERR_INVALID_ARG, "%s: %s = %zu times %s = %zu exceeds GB_MAX_N = %zu", fn, rows_name, rows,
                cols_name, cols, GB_MAX_N);
  }
  return GB_OK;
}
// Bytes from the first value of the array to its last.
size_t extent(size_t rows, size_t stride, size_t cols, size_t size) {
  return rows == 0 || cols == 0 ? 0 : ((rows - 1) * stride + cols) * size;
}

gb_status check_cols(size_t cols, const char* fn) {
  if (cols >= 1 && cols <= GB_NORM_MAX_COLS) return GB_OK;
  return fail(GB_ERR_INVALID_ARG, "%s: cols = %zu is outside 1..%d", fn, cols, GB_NORM_MAX_COLS);
}

gb_status check_workspace(const void* workspace, size_t bytes, size_t needed, const char* fn) {
  if (needed == 0) return GB_OK;
  if (workspace == nullptr || bytes < needed) {
    return fail(GB_ERR_WORKSPACE, "%s: workspace %p of %zu bytes, %zu needed", fn, workspace, bytes, needed);
  }
  if (!aligned(workspace, GB_ALIGN)) {
    return fail(GB_ERR_MISALIGNED, "%s: workspace = %p is not %d-byte aligned", fn, workspace, GB_ALIGN);
  }
  return GB_OK;
}

// An input array that may also be the output: the same address and stride.
void add_alias(gb::Spans* ins, const void* p, size_t stride, size_t bytes, size_t rows, const gb::Rows& out,
               const char* name) {
  if (p == out.p && (stride == out.stride || rows <= 1)) return;
  ins->add(p, bytes, name);
}

#define GB_TRY(call)                      \
  do {                                    \
    const gb_status try_status = (call);  \
    if (try_status != GB_OK) return try_status; \
  } while (0)

gb_status norm_forward(const char* fn, gb::NormArgs a, double eps, hipStream_t stream) {
  GB_TRY(check_cols(a.cols, fn));
  GB_TRY(check_shape(a.rows, a.cols, fn, "rows", "cols"));
  GB_TRY(check_type(a.dtype, fn, "dtype"));
  if (a.w != nullptr || a.b != nullptr) GB_TRY(check_type(a.param_dtype, fn, "param_dtype"));
  if (!(eps > 0.0) || !((float)eps > 0.0f) || !std::isfinite((float)eps)) {
    return fail(GB_ERR_INVALID_ARG, "%s: eps = %g is not finite and above 0 in binary32", fn, eps);
  }
  if (a.rows == 0) return GB_OK;
  const size_t e = elem_size(a.dtype), pe = elem_size(a.param_dtype);
  GB_TRY(check_pointer(a.y.p, e, true, fn, "y"));
  GB_TRY(check_pointer(a.x.p, e, true, fn, "x"));
  GB_TRY(check_stride(a.y.stride, a.rows, a.cols, true, fn, "y_stride"));
  GB_TRY(check_stride(a.x.stride, a.rows, a.cols, false, fn, "x_stride"));
  GB_TRY(check_pointer(a.w, pe, false, fn, "weight"));
  GB_TRY(check_pointer(a.b, pe, false, fn, "bias"));
  GB_TRY(check_pointer(a.mean, 4, false, fn, "mean"));
  GB_TRY(check_pointer(a.rstd, 4, false, fn, "rstd"));
  gb::Spans outs, ins;
  outs.add(a.y.p, extent(a.rows, a.y.stride, a.cols, e), "y");
  outs.add(a.mean, 4 * a.rows, "mean");
  outs.add(a.rstd, 4 * a.rows, "rstd");
  add_alias(&ins, a.x.p, a.x.stride, extent(a.rows, a.x.stride, a.cols, e), a.rows, a.y, "x");
  ins.add(a.w, pe * a.cols, "weight");
  ins.add(a.b, pe * a.cols, "bias");
  GB_TRY(gb::check_disjoint(fn, outs, ins));
  a.eps = (float)eps;
  return from_hip(gb::launch_layer_norm(a, stream), fn);
}

gb_status norm_backward(const char* fn, gb::NormGradArgs a, int accumulate, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  GB_TRY(check_cols(a.cols, fn));
  GB_TRY(check_shape(a.rows, a.cols, fn, "rows", "cols"));
  GB_TRY(check_type(a.dtype, fn, "dtype"));
  if (a.w != nullptr) GB_TRY(check_type(a.param_dtype, fn, "param_dtype"));
  const bool sums = a.dw != nullptr || a.db != nullptr;
  if (sums) GB_TRY(check_type(a.grad_dtype, fn, "grad_dtype"));
  if (accumulate != 0 && accumulate != 1) {
    return fail(GB_ERR_INVALID_ARG, "%s: accumulate = %d is not 0 or 1", fn, accumulate);
  }
  const size_t e = elem_size(a.dtype), pe = elem_size(a.param_dtype), ge = elem_size(a.grad_dtype);
  GB_TRY(check_pointer(a.dw, ge, false, fn, "dweight"));
  GB_TRY(check_pointer(a.db, ge, false, fn, "dbias"));
  gb::Spans outs, ins;
  outs.add(a.dw, ge * a.cols, "dweight");
  outs.add(a.db, ge * a.cols, "dbias");
  if (a.rows > 0) {
    if (a.dx.p == nullptr && !sums) return fail(GB_ERR_INVALID_ARG, "%s: dx, dweight and dbias are all NULL", fn);
    GB_TRY(check_pointer(a.dx.p, e, false, fn, "dx"));
    GB_TRY(check_pointer(a.dy.p, e, true, fn, "dy"));
    GB_TRY(check_pointer(a.x.p, e, true, fn, "x"));
    if (a.dx.p != nullptr) GB_TRY(check_stride(a.dx.stride, a.rows, a.cols, true, fn, "dx_stride"));
    GB_TRY(check_stride(a.dy.stride, a.rows, a.cols, false, fn, "dy_stride"));
    GB_TRY(check_stride(a.x.stride, a.rows, a.cols, false, fn, "x_stride"));
    GB_TRY(check_pointer(a.mean, 4, true, fn, "mean"));
    GB_TRY(check_pointer(a.rstd, 4, true, fn, "rstd"));
    GB_TRY(check_pointer(a.w, pe, false, fn, "weight"));
    const size_t needed = sums ? gb_layer_norm_workspace_bytes(a.rows, a.cols) : 0;
    GB_TRY(check_workspace(workspace, workspace_bytes, needed, fn));
    if (a.dx.p != nullptr) outs.add(a.dx.p, extent(a.rows, a.dx.stride, a.cols, e), "dx");
    if (sums) outs.add(workspace, needed, "workspace");
    add_alias(&ins, a.dy.p, a.dy.stride, extent(a.rows, a.dy.stride, a.cols, e), a.rows, a.dx, "dy");
    add_alias(&ins, a.x.p, a.x.stride, extent(a.rows, a.x.stride, a.cols, e), a.rows, a.dx, "x");
    ins.add(a.mean, 4 * a.rows, "mean");
    ins.add(a.rstd, 4 * a.rows, "rstd");
    ins.add(a.w, pe * a.cols, "weight");
  } else if (!sums || accumulate) {
    return GB_OK;
  }
  GB_TRY(gb::check_disjoint(fn, outs, ins));
  a.accumulate = accumulate != 0;
  a.partials = static_cast<float*>(workspace);
  a.partial_stride = gb::norm_partial_stride(a.cols);
  return from_hip(gb::launch_layer_norm_grad(a, stream), fn);
}

gb_status check_ids(const void* ids, int id_dtype, size_t tokens, size_t vocab, size_t dim, int64_t first,
                    const char* fn) {
  if (tokens > GB_EMBEDDING_MAX_TOKENS || vocab > GB_EMBEDDING_MAX_VOCAB || dim > GB_EMBEDDING_MAX_DIM) {
    return fail(GB_ERR_INVALID_ARG, "%s: tokens = %zu, vocab = %zu or dim = %zu is beyond %zu, %zu and %zu", fn,
                tokens, vocab, dim, (size_t)GB_EMBEDDING_MAX_TOKENS, (size_t)GB_EMBEDDING_MAX_VOCAB,
                (size_t)GB_EMBEDDING_MAX_DIM);
  }
  GB_TRY(check_shape(tokens, dim, fn, "tokens", "dim"));
  GB_TRY(check_shape(vocab, dim, fn, "vocab", "dim"));
  if (first > INT64_MAX - (int64_t)vocab) {  // an id's distance from first, without a sign, then names one row
    return fail(GB_ERR_INVALID_ARG, "%s: first = %lld and vocab = %zu pass the largest id", fn, (long long)first,
                vocab);
  }
  if (id_dtype != GB_DTYPE_I32 && id_dtype != GB_DTYPE_I64) {
    return fail(GB_ERR_UNSUPPORTED, "%s: id_dtype = %d is not int32 or int64", fn, id_dtype);
  }
  return check_pointer(ids, elem_size(id_dtype), tokens > 0 && dim > 0, fn, "ids");
}
gb_status check_factor(double scale, const char* fn) {
  if (std::isfinite(scale) && std::isfinite((float)scale)) return GB_OK;
  return fail(GB_ERR_INVALID_ARG, "%s: scale = %g is not finite in binary32", fn, scale);
}

gb_status embedding_forward(const char* fn, gb::LookArgs a, double scale, hipStream_t stream) {
  GB_TRY(check_type(a.out_dtype, fn, "out_dtype"));
  GB_TRY(check_type(a.table_dtype, fn, "table_dtype"));
  GB_TRY(check_ids(a.ids, a.id_dtype, a.tokens, a.vocab, a.dim, a.first, fn));
  GB_TRY(check_factor(scale, fn));
  if (a.tokens == 0 || a.dim == 0) return GB_OK;
  const size_t oe = elem_size(a.out_dtype), te = elem_size(a.table_dtype);
  GB_TRY(check_pointer(a.out.p, oe, true, fn, "out"));
  GB_TRY(check_pointer(a.table.p, te, a.vocab > 0, fn, "table"));
  GB_TRY(check_stride(a.out.stride, a.tokens, a.dim, true, fn, "out_stride"));
  GB_TRY(check_stride(a.table.stride, a.vocab, a.dim, false, fn, "table_stride"));
  gb::Spans outs, ins;
  outs.add(a.out.p, extent(a.tokens, a.out.stride, a.dim, oe), "out");
  ins.add(a.table.p, extent(a.vocab, a.table.stride, a.dim, te), "table");
  ins.add(a.ids, elem_size(a.id_dtype) * a.tokens, "ids");
  GB_TRY(gb::check_disjoint(fn, outs, ins));
  a.scale = (float)scale;
  return from_hip(gb::launch_embedding(a, stream), fn);
}

gb_status embedding_backward(const char* fn, gb::LookGradArgs a, double scale, int accumulate, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  GB_TRY(check_type(a.grad_dtype, fn, "grad_dtype"));
  GB_TRY(check_type(a.dtype, fn, "dtype"));
  GB_TRY(check_ids(a.ids, a.id_dtype, a.tokens, a.vocab, a.dim, a.first, fn));
  GB_TRY(check_factor(scale, fn));
  if (accumulate != 0 && accumulate != 1) {
    return fail(GB_ERR_INVALID_ARG, "%s: accumulate = %d is not 0 or 1", fn, accumulate);
  }
  if (a.vocab == 0 || a.dim == 0 || (a.tokens == 0 && accumulate)) return GB_OK;
  const size_t ge = elem_size(a.grad_dtype), e = elem_size(a.dtype);
  GB_TRY(check_pointer(a.dtable.p, ge, true, fn, "dtable"));
  GB_TRY(check_pointer(a.dout.p, e, a.tokens > 0, fn, "dout"));
  GB_TRY(check_stride(a.dtable.stride, a.vocab, a.dim, true, fn, "dtable_stride"));
  GB_TRY(check_stride(a.dout.stride, a.tokens, a.dim, false, fn, "dout_stride"));
  const size_t needed = a.tokens > 0 ? gb_embedding_workspace_bytes(a.tokens, a.vocab, a.dim) : 0;
  GB_TRY(check_workspace(workspace, workspace_bytes, needed, fn));
  gb::Spans outs, ins;
  outs.add(a.dtable.p, extent(a.vocab, a.dtable.stride, a.dim, ge), "dtable");
  outs.add(workspace, needed, "workspace");
  ins.add(a.dout.p, extent(a.tokens, a.dout.stride, a.dim, e), "dout");
  ins.add(a.ids, elem_size(a.id_dtype) * a.tokens, "ids");
  GB_TRY(gb::check_disjoint(fn, outs, ins));
  a.scale = (float)scale;
  a.accumulate = accumulate != 0;
  a.workspace = static_cast<char*>(workspace);
  return from_hip(gb::launch_embedding_grad(a, stream), fn);
}

gb::Rows rows_of(const void* p, size_t stride) { return gb::Rows{const_cast<void*>(p), stride}; }
// A size as a kernel argument of 32 bits; one that does not fit is refused by its check whatever it becomes.
uint32_t narrow(size_t v) { return v > UINT32_MAX ? UINT32_MAX : (uint32_t)v; }

}  // namespace

extern "C" {

gb_status gb_layer_norm_forward(int dtype, void* y, size_t y_stride, const void* x, size_t x_stride, size_t rows,
                                size_t cols, int param_dtype, const void* weight, const void* bias, double eps,
                                float* mean, float* rstd, void* stream) {
  return gb::traced_call("gb_layer_norm_forward", stream, -1, rows, -1, [&](const char* fn) -> gb_status {
    return norm_forward(fn, gb::NormArgs{rows_of(y, y_stride), rows_of(x, x_stride), rows, narrow(cols), dtype,
                                         param_dtype, weight, bias, 0.0f, mean, rstd},
                        eps, static_cast<hipStream_t>(stream));
  });
}

size_t gb_layer_norm_workspace_bytes(size_t rows, size_t cols) {
  if (cols < 1 || cols > GB_NORM_MAX_COLS || rows > GB_MAX_N / cols) return 0;
  size_t groups = 0;
  for (int dtype : {GB_DTYPE_F32, GB_DTYPE_F16, GB_DTYPE_BF16}) {
    const size_t g = gb::norm_grad_groups(rows, cols, dtype);
    groups = g > groups ? g : groups;
  }
  return groups * 2 * gb::norm_partial_stride(cols) * sizeof(float);
}

gb_status gb_layer_norm_backward(int dtype, void* dx, size_t dx_stride, const void* dy, size_t dy_stride,
                                 const void* x, size_t x_stride, size_t rows, size_t cols, const float* mean,
                                 const float* rstd, int param_dtype, const void* weight, int grad_dtype,
                                 void* dweight, void* dbias, int accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return gb::traced_call("gb_layer_norm_backward", stream, -1, rows, -1, [&](const char* fn) -> gb_status {
    gb::NormGradArgs a = {};
    a.dx = rows_of(dx, dx_stride);
    a.dy = rows_of(dy, dy_stride);
    a.x = rows_of(x, x_stride);
    a.rows = rows;
    a.cols = narrow(cols);
    a.dtype = dtype;
    a.param_dtype = param_dtype;
    a.grad_dtype = grad_dtype;
    a.mean = mean;
    a.rstd = rstd;
    a.w = weight;
    a.dw = dweight;
    a.db = dbias;
    return norm_backward(fn, a, accumulate, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
  });
}

gb_status gb_embedding_forward(int out_dtype, void* out, size_t out_stride, int table_dtype, const void* table,
                               size_t table_stride, size_t vocab, size_t dim, int id_dtype, const void* ids,
                               size_t tokens, int64_t first, double scale, void* stream) {
  return gb::traced_call("gb_embedding_forward", stream, -1, tokens, -1, [&](const char* fn) -> gb_status {
    return embedding_forward(fn, gb::LookArgs{rows_of(out, out_stride), rows_of(table, table_stride), ids, tokens,
                                              vocab, dim, first, 0.0f, out_dtype, table_dtype, id_dtype},
                             scale, static_cast<hipStream_t>(stream));
  });
}

size_t gb_embedding_workspace_bytes(size_t tokens, size_t vocab, size_t dim) {
  if (tokens > GB_EMBEDDING_MAX_TOKENS || vocab > GB_EMBEDDING_MAX_VOCAB || dim > GB_EMBEDDING_MAX_DIM) return 0;
  if (tokens == 0 || vocab == 0 || dim == 0 || tokens > GB_MAX_N / dim || vocab > GB_MAX_N / dim) return 0;
  return gb::look_grad_layout(tokens, vocab, dim).total;
}

gb_status gb_embedding_backward(int grad_dtype, void* dtable, size_t dtable_stride, size_t vocab, size_t dim,
                                int dtype, const void* dout, size_t dout_stride, int id_dtype, const void* ids,
                                size_t tokens, int64_t first, int64_t padding, double scale, int accumulate,
                                void* workspace, size_t workspace_bytes, void* stream) {
  return gb::traced_call("gb_embedding_backward", stream, -1, tokens, -1, [&](const char* fn) -> gb_status {
    gb::LookGradArgs a = {};
    a.dtable = rows_of(dtable, dtable_stride);
    a.dout = rows_of(dout, dout_stride);
    a.ids = ids;
    a.tokens = tokens;
    a.vocab = vocab;
    a.dim = dim;
    a.first = first;
    a.padding = padding;
    a.dtype = dtype;
    a.grad_dtype = grad_dtype;
    a.id_dtype = id_dtype;
    return embedding_backward(fn, a, scale, accumulate, workspace, workspace_bytes,
                              static_cast<hipStream_t>(stream));
  });
}

}  // extern "C"
