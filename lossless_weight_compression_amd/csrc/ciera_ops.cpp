// Host side of the expert products and the 4-bit operators: argument checks and
// launches.  See include/ciera.h.
#include <hip/hip_runtime.h>

#include "ciera.h"
#include "ciera_host.h"
#include "ciera_ops_internal.h"

using namespace ciera;

namespace {

typedef unsigned __int128 u128;

constexpr uint64_t kMaxSide = (uint64_t)1 << 30;  // sides and their rounding up to a tile are 32-bit counts
constexpr uint32_t kMaxGroups = 65536;          // of a product: every workgroup adds up their tiles
constexpr uint64_t kMaxExtent = (uint64_t)1 << 60;

uint32_t elem_bytes(uint32_t dt) { return dt == CIERA_FP32 ? 4u : 2u; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
  uintptr_t at;
  uint64_t bytes;
};
bool overlap(Range a, Range b) {
  if (!a.bytes || !b.bytes) return false;
  return (u128)a.at < (u128)b.at + b.bytes && (u128)b.at < (u128)a.at + a.bytes;
}

bool empty(const ciera_matrix_t* m) { return m->groups == 0 || m->rows == 0 || m->cols == 0; }

// Type, sizes and strides of a matrix; its address range.  The pointer is
// looked at by check_data.
ciera_status_t check_matrix(const ciera_matrix_t* m, bool output, Range* r) {
  if (!m) return CIERA_ERR_INVALID_ARG;
  if (m->dtype != CIERA_BF16 && m->dtype != CIERA_FP32 && m->dtype != CIERA_FP16) return CIERA_ERR_INVALID_ARG;
  if (m->rows >= kMaxSide || m->cols >= kMaxSide || m->groups >= kMaxSide) return CIERA_ERR_UNSUPPORTED;
  *r = Range{reinterpret_cast<uintptr_t>(m->data), 0};
  if (empty(m)) return CIERA_OK;
  const u128 one = (u128)(m->rows - 1) * m->row_stride + m->cols;
  const u128 all = (u128)(m->groups - 1) * m->group_stride + one;
  if (all >= kMaxExtent) return CIERA_ERR_UNSUPPORTED;
  if (output && ((m->rows > 1 && m->row_stride < m->cols) || (m->groups > 1 && m->group_stride < one)))
    return CIERA_ERR_INVALID_ARG;
  r->bytes = (uint64_t)all * elem_bytes(m->dtype);
  return CIERA_OK;
}
bool bad_data(const ciera_matrix_t* m) {
  return !empty(m) && (!m->data || !aligned(m->data, elem_bytes(m->dtype)));
}

uint64_t padded(uint64_t cols) { return (cols + kMxColsPad - 1) / kMxColsPad * kMxColsPad; }

ciera_status_t check_mx(const ciera_mx_t* q, Range* codes, Range* scales) {
  if (!q) return CIERA_ERR_INVALID_ARG;
  if (q->reserved) return CIERA_ERR_INVALID_ARG;
  if (q->rows >= kMaxSide || q->cols >= kMaxSide || q->groups >= kMaxSide) return CIERA_ERR_UNSUPPORTED;
  const u128 values = (u128)q->groups * q->rows * padded(q->cols);
  if (values >= kMaxExtent) return CIERA_ERR_UNSUPPORTED;
  *codes = Range{reinterpret_cast<uintptr_t>(q->codes), (uint64_t)values / 2};
  *scales = Range{reinterpret_cast<uintptr_t>(q->scales), (uint64_t)values / kMxBlock};
  return CIERA_OK;
}
bool bad_data(const ciera_mx_t* q, Range codes) {
  return codes.bytes && (!q->codes || !aligned(q->codes, 16) || !q->scales || !aligned(q->scales, 4));
}

// Whether every row of every group starts at a multiple of 16 bytes.
bool flat(const ciera_matrix_t* m) {
  const uint64_t per = 16 / elem_bytes(m->dtype);
  return aligned(m->data, 16) && (m->rows <= 1 || m->row_stride % per == 0) &&
         (m->groups <= 1 || m->group_stride % per == 0);
}

hipStream_t hip_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

ciera_status_t launched(const char* what, hipError_t e) {
  if (e == hipSuccess) return CIERA_OK;
  if (e == hipErrorInvalidConfiguration) return CIERA_ERR_UNSUPPORTED;  // more workgroups than a grid holds
  return device_error(what, e);
}

// out: the output's range, which the kernels write while they read the offsets.
bool bad_offsets(const int32_t* offsets, uint32_t groups, Range out) {
  if (!offsets) return groups != 1;
  return !aligned(offsets, 4) || overlap(out, Range{reinterpret_cast<uintptr_t>(offsets), ((uint64_t)groups + 1) * 4});
}

}  // namespace

extern "C" {

ciera_status_t ciera_mx_sizes(uint32_t groups, uint64_t rows, uint64_t cols, uint64_t* code_bytes,
                              uint64_t* scale_bytes) {
  if (!code_bytes || !scale_bytes) return CIERA_ERR_INVALID_ARG;
  const ciera_mx_t q = {nullptr, nullptr, groups, 0, rows, cols};
  Range c, s;
  if (ciera_status_t e = check_mx(&q, &c, &s)) return e;
  *code_bytes = c.bytes;
  *scale_bytes = s.bytes;
  return CIERA_OK;
}

ciera_status_t ciera_mx_quantize(const ciera_matrix_t* x, uint32_t axis, const ciera_mx_t* q, void* stream) {
  Range rx, rc, rs;
  if (ciera_status_t e = check_matrix(x, false, &rx)) return e;
  if (ciera_status_t e = check_mx(q, &rc, &rs)) return e;
  if (axis > 1 || q->groups != x->groups || q->rows != (axis ? x->rows : x->cols) ||
      q->cols != (axis ? x->cols : x->rows))
    return CIERA_ERR_INVALID_ARG;
  if (empty(x)) return CIERA_OK;
  if (bad_data(x) || bad_data(q, rc)) return CIERA_ERR_INVALID_ARG;
  if (overlap(rx, rc) || overlap(rx, rs) || overlap(rc, rs)) return CIERA_ERR_INVALID_ARG;
  const MxQuantArgs a = {x->data, q->codes, q->scales, x->row_stride, x->group_stride,
                         (int32_t)x->groups, (int32_t)x->rows, (int32_t)x->cols};
  return launched("4-bit quantisation launch", launch_mx_quantize(x->dtype, axis, a, hip_stream(stream)));
}

ciera_status_t ciera_mx_dequantize(const ciera_mx_t* q, const ciera_matrix_t* out, void* stream) {
  Range ro, rc, rs;
  if (ciera_status_t e = check_mx(q, &rc, &rs)) return e;
  if (ciera_status_t e = check_matrix(out, true, &ro)) return e;
  if (q->groups != out->groups || q->rows != out->rows || q->cols != out->cols) return CIERA_ERR_INVALID_ARG;
  if (empty(out)) return CIERA_OK;
  if (bad_data(out) || bad_data(q, rc)) return CIERA_ERR_INVALID_ARG;
  if (overlap(ro, rc) || overlap(ro, rs)) return CIERA_ERR_INVALID_ARG;
  const MxDequantArgs a = {q->codes, q->scales, out->data, out->row_stride, out->group_stride,
                           (int32_t)out->groups, (int32_t)out->rows, (int32_t)out->cols};
  return launched("4-bit dequantisation launch", launch_mx_dequantize(out->dtype, a, hip_stream(stream)));
}

ciera_status_t ciera_mx_mm(const ciera_mx_t* a, const ciera_mx_t* b, const int32_t* offsets,
                           const ciera_matrix_t* out, void* stream) {
  Range ac, as, bc, bs, ro;
  if (ciera_status_t e = check_mx(a, &ac, &as)) return e;
  if (ciera_status_t e = check_mx(b, &bc, &bs)) return e;
  if (ciera_status_t e = check_matrix(out, true, &ro)) return e;
  if (a->groups != 1 || out->groups != 1 || a->cols != b->cols || out->rows != a->rows || out->cols != b->rows)
    return CIERA_ERR_INVALID_ARG;
  if (b->groups > kMaxGroups) return CIERA_ERR_UNSUPPORTED;
  if (b->groups == 0 || empty(out)) return CIERA_OK;
  if (bad_offsets(offsets, b->groups, ro)) return CIERA_ERR_INVALID_ARG;
  if (bad_data(out) || bad_data(a, ac) || bad_data(b, bc)) return CIERA_ERR_INVALID_ARG;
  if (overlap(ro, ac) || overlap(ro, as) || overlap(ro, bc) || overlap(ro, bs)) return CIERA_ERR_INVALID_ARG;
  const MxMmArgs g = {a->codes, a->scales, b->codes, b->scales, out->data, offsets, out->row_stride,
                      (int32_t)a->rows, (int32_t)padded(a->cols), (int32_t)b->rows, (int32_t)b->groups};
  return launched("4-bit product launch", launch_mx_mm(out->dtype, g, hip_stream(stream)));
}

ciera_status_t ciera_group_mm(const ciera_matrix_t* x, const ciera_matrix_t* w, uint32_t transpose_w,
                              const int32_t* offsets, const ciera_matrix_t* out, void* stream) {
  Range rx, rw, ro;
  if (ciera_status_t e = check_matrix(x, false, &rx)) return e;
  if (ciera_status_t e = check_matrix(w, false, &rw)) return e;
  if (ciera_status_t e = check_matrix(out, true, &ro)) return e;
  if (transpose_w > 1 || x->dtype == CIERA_FP32 || w->dtype != x->dtype ||
      (out->dtype != x->dtype && out->dtype != CIERA_FP32))
    return CIERA_ERR_INVALID_ARG;
  const uint64_t wk = transpose_w ? w->cols : w->rows, wn = transpose_w ? w->rows : w->cols;
  if (x->groups != 1 || out->groups != 1 || wk != x->cols || out->rows != x->rows || out->cols != wn)
    return CIERA_ERR_INVALID_ARG;
  if (w->groups > kMaxGroups) return CIERA_ERR_UNSUPPORTED;
  if (w->groups == 0 || empty(out)) return CIERA_OK;
  if (bad_offsets(offsets, w->groups, ro)) return CIERA_ERR_INVALID_ARG;
  if (bad_data(x) || bad_data(w) || bad_data(out)) return CIERA_ERR_INVALID_ARG;
  if (overlap(ro, rx) || overlap(ro, rw)) return CIERA_ERR_INVALID_ARG;
  const GroupMmArgs g = {x->data, w->data, out->data, offsets, x->row_stride, w->row_stride, out->row_stride,
                         w->group_stride, (int32_t)x->rows, (int32_t)x->cols, (int32_t)wn, (int32_t)w->groups};
  return launched("grouped product launch", launch_group_mm(x->dtype, out->dtype == CIERA_FP32, transpose_w == 1,
                                                            flat(x) && flat(w), g, hip_stream(stream)));
}

ciera_status_t ciera_group_wgrad(const ciera_matrix_t* x, const ciera_matrix_t* dy, const int32_t* offsets,
                                 const ciera_matrix_t* out, void* stream) {
  Range rx, rd, ro;
  if (ciera_status_t e = check_matrix(x, false, &rx)) return e;
  if (ciera_status_t e = check_matrix(dy, false, &rd)) return e;
  if (ciera_status_t e = check_matrix(out, true, &ro)) return e;
  if (x->dtype == CIERA_FP32 || dy->dtype != x->dtype || (out->dtype != x->dtype && out->dtype != CIERA_FP32))
    return CIERA_ERR_INVALID_ARG;
  if (x->groups != 1 || dy->groups != 1 || dy->rows != x->rows || out->rows != x->cols || out->cols != dy->cols)
    return CIERA_ERR_INVALID_ARG;
  if (out->groups > kMaxGroups) return CIERA_ERR_UNSUPPORTED;
  if (empty(out)) return CIERA_OK;
  if (bad_offsets(offsets, out->groups, ro)) return CIERA_ERR_INVALID_ARG;
  if (bad_data(x) || bad_data(dy) || bad_data(out)) return CIERA_ERR_INVALID_ARG;
  if (overlap(ro, rx) || overlap(ro, rd)) return CIERA_ERR_INVALID_ARG;
  const GroupWgradArgs g = {x->data, dy->data, out->data, offsets, x->row_stride, dy->row_stride, out->row_stride,
                            out->group_stride, (int32_t)x->rows, (int32_t)x->cols, (int32_t)dy->cols,
                            (int32_t)out->groups};
  return launched("grouped weight gradient launch", launch_group_wgrad(x->dtype, out->dtype == CIERA_FP32,
                                                                       flat(x) && flat(dy), g, hip_stream(stream)));
}

}  // extern "C"
