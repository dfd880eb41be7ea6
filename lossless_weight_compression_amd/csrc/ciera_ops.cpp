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

struct GqRanges {
  Range codes, scales, zeros;
};
ciera_status_t check_gq(const ciera_gq_t* q, GqRanges* r) {
  if (!q) return CIERA_ERR_INVALID_ARG;
  if (q->reserved || (q->block != 32 && q->block != 64 && q->block != 128) ||
      (q->scale_dtype != CIERA_BF16 && q->scale_dtype != CIERA_FP16))
    return CIERA_ERR_INVALID_ARG;
  if (q->rows >= kMaxSide || q->cols >= kMaxSide || q->groups >= kMaxSide) return CIERA_ERR_UNSUPPORTED;
  const u128 values = (u128)q->groups * q->rows * padded(q->cols);
  if (values >= kMaxExtent) return CIERA_ERR_UNSUPPORTED;
  const uint64_t blocks = (uint64_t)values / q->block;
  r->codes = Range{reinterpret_cast<uintptr_t>(q->codes), (uint64_t)values / 2};
  r->scales = Range{reinterpret_cast<uintptr_t>(q->scales), blocks * 2};
  r->zeros = Range{reinterpret_cast<uintptr_t>(q->zeros), q->zeros ? blocks : 0};
  return CIERA_OK;
}
bool bad_data(const ciera_gq_t* q, const GqRanges& r) {
  return r.codes.bytes && (!q->codes || !aligned(q->codes, 16) || !q->scales || !aligned(q->scales, 4) ||
                           !aligned(q->zeros, 4));
}
bool overlap(Range a, const GqRanges& r) { return overlap(a, r.codes) || overlap(a, r.scales) || overlap(a, r.zeros); }
uint32_t half_scales(const ciera_gq_t* q) { return q->scale_dtype == CIERA_FP16 ? ~0u : 0u; }
GqStack gq_stack(const ciera_gq_t* q) {
  return GqStack{q->codes, static_cast<const uint16_t*>(q->scales), q->zeros};
}

// Whether two matrices of one group share no element: their address ranges lie apart, or
// they are columns of one buffer.
bool apart(const ciera_matrix_t* a, Range ra, const ciera_matrix_t* b, Range rb) {
  if (!overlap(ra, rb)) return true;
  const uint64_t e = elem_bytes(a->dtype), row = a->row_stride * e;
  if (a->dtype != b->dtype || a->rows < 2 || b->rows < 2 || a->row_stride != b->row_stride) return false;
  // where a row of b begins within the row of a that it lies in or behind
  const uint64_t d = (ra.at <= rb.at ? rb.at - ra.at : row - (ra.at - rb.at) % row) % row;
  return d >= a->cols * e && d + b->cols * e <= row;
}
bool one_matrix(const ciera_matrix_t* m, uint64_t rows, uint64_t cols) {
  return m->groups == 1 && m->rows == rows && m->cols == cols;
}
bool same_shape(const ciera_matrix_t* a, const ciera_matrix_t* b) {
  return a->dtype == b->dtype && a->groups == b->groups && a->rows == b->rows && a->cols == b->cols;
}
bool bad_act(uint32_t act) { return act != CIERA_ACT_SILU && act != CIERA_ACT_GELU; }

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

ciera_status_t ciera_glu_mm(const ciera_matrix_t* x, const ciera_matrix_t* w_gate, const ciera_matrix_t* w_up,
                            uint32_t transpose_w, uint32_t act, const int32_t* offsets, const ciera_matrix_t* out,
                            const ciera_matrix_t* gate, const ciera_matrix_t* up, void* stream) {
  if ((gate == nullptr) != (up == nullptr)) return CIERA_ERR_INVALID_ARG;
  Range rx, rg, ru, ro[3];
  const ciera_matrix_t* o[3] = {out, gate, up};
  const int outs = gate ? 3 : 1;
  if (ciera_status_t e = check_matrix(x, false, &rx)) return e;
  if (ciera_status_t e = check_matrix(w_gate, false, &rg)) return e;
  if (ciera_status_t e = check_matrix(w_up, false, &ru)) return e;
  for (int i = 0; i < outs; i++)
    if (ciera_status_t e = check_matrix(o[i], true, &ro[i])) return e;
  if (transpose_w > 1 || bad_act(act) || x->dtype == CIERA_FP32 || w_gate->dtype != x->dtype ||
      !same_shape(w_gate, w_up) || (out->dtype != x->dtype && out->dtype != CIERA_FP32))
    return CIERA_ERR_INVALID_ARG;
  const uint64_t wk = transpose_w ? w_gate->cols : w_gate->rows, wn = transpose_w ? w_gate->rows : w_gate->cols;
  if (x->groups != 1 || wk != x->cols) return CIERA_ERR_INVALID_ARG;
  for (int i = 0; i < outs; i++)
    if (!one_matrix(o[i], x->rows, wn) || o[i]->dtype != out->dtype) return CIERA_ERR_INVALID_ARG;
  if (w_gate->groups > kMaxGroups) return CIERA_ERR_UNSUPPORTED;
  if (w_gate->groups == 0 || empty(out)) return CIERA_OK;
  if (bad_data(x) || bad_data(w_gate) || bad_data(w_up)) return CIERA_ERR_INVALID_ARG;
  for (int i = 0; i < outs; i++) {
    if (bad_data(o[i]) || bad_offsets(offsets, w_gate->groups, ro[i])) return CIERA_ERR_INVALID_ARG;
    if (overlap(ro[i], rx) || overlap(ro[i], rg) || overlap(ro[i], ru)) return CIERA_ERR_INVALID_ARG;
    for (int j = 0; j < i; j++)
      if (!apart(o[j], ro[j], o[i], ro[i])) return CIERA_ERR_INVALID_ARG;
  }
  const GluMmArgs g = {x->data, w_gate->data, w_up->data, out->data, gate ? gate->data : nullptr,
                       up ? up->data : nullptr, offsets, x->row_stride, w_gate->row_stride, w_up->row_stride,
                       w_gate->group_stride, w_up->group_stride, out->row_stride, gate ? gate->row_stride : 0,
                       up ? up->row_stride : 0, (int32_t)x->rows, (int32_t)x->cols, (int32_t)wn,
                       (int32_t)w_gate->groups, (int32_t)act};
  return launched("gated block launch", launch_glu_mm(x->dtype, out->dtype == CIERA_FP32, transpose_w == 1,
                                                      flat(x) && flat(w_gate) && flat(w_up), g, hip_stream(stream)));
}

ciera_status_t ciera_glu_grad(const ciera_matrix_t* dy, const ciera_matrix_t* w_down, uint32_t transpose_w,
                              uint32_t act, const int32_t* offsets, const ciera_matrix_t* gate,
                              const ciera_matrix_t* up, const ciera_matrix_t* dgate, const ciera_matrix_t* dup,
                              void* stream) {
  Range rx, rw, r[4];
  const ciera_matrix_t* m[4] = {gate, up, dgate, dup};
  if (ciera_status_t e = check_matrix(dy, false, &rx)) return e;
  if (ciera_status_t e = check_matrix(w_down, false, &rw)) return e;
  for (int i = 0; i < 4; i++)
    if (ciera_status_t e = check_matrix(m[i], i >= 2, &r[i])) return e;
  if (transpose_w > 1 || bad_act(act) || dy->dtype == CIERA_FP32 || w_down->dtype != dy->dtype ||
      (gate->dtype != dy->dtype && gate->dtype != CIERA_FP32))
    return CIERA_ERR_INVALID_ARG;
  const uint64_t wk = transpose_w ? w_down->cols : w_down->rows, wn = transpose_w ? w_down->rows : w_down->cols;
  if (dy->groups != 1 || wk != dy->cols) return CIERA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; i++)
    if (!one_matrix(m[i], dy->rows, wn) || m[i]->dtype != gate->dtype) return CIERA_ERR_INVALID_ARG;
  if (w_down->groups > kMaxGroups) return CIERA_ERR_UNSUPPORTED;
  if (w_down->groups == 0 || empty(dgate)) return CIERA_OK;
  if (bad_data(dy) || bad_data(w_down)) return CIERA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; i++)
    if (bad_data(m[i])) return CIERA_ERR_INVALID_ARG;
  for (int i = 2; i < 4; i++) {
    if (bad_offsets(offsets, w_down->groups, r[i]) || overlap(r[i], rx) || overlap(r[i], rw))
      return CIERA_ERR_INVALID_ARG;
    for (int j = 0; j < i; j++)
      if (!apart(m[j], r[j], m[i], r[i])) return CIERA_ERR_INVALID_ARG;
  }
  const GluGradArgs g = {dy->data, w_down->data, gate->data, up->data, dgate->data, dup->data, offsets,
                         dy->row_stride, w_down->row_stride, w_down->group_stride, gate->row_stride, up->row_stride,
                         dgate->row_stride, dup->row_stride, (int32_t)dy->rows, (int32_t)dy->cols, (int32_t)wn,
                         (int32_t)w_down->groups, (int32_t)act};
  return launched("gated block gradient launch", launch_glu_grad(dy->dtype, gate->dtype == CIERA_FP32, transpose_w == 1,
                                                                 flat(dy) && flat(w_down), g, hip_stream(stream)));
}

ciera_status_t ciera_glu_xgrad(const ciera_matrix_t* dgate, const ciera_matrix_t* dup, const ciera_matrix_t* w_gate,
                               const ciera_matrix_t* w_up, uint32_t transpose_w, const int32_t* offsets,
                               const ciera_matrix_t* out, void* stream) {
  Range ra, rb, rg, ru, ro;
  if (ciera_status_t e = check_matrix(dgate, false, &ra)) return e;
  if (ciera_status_t e = check_matrix(dup, false, &rb)) return e;
  if (ciera_status_t e = check_matrix(w_gate, false, &rg)) return e;
  if (ciera_status_t e = check_matrix(w_up, false, &ru)) return e;
  if (ciera_status_t e = check_matrix(out, true, &ro)) return e;
  if (transpose_w > 1 || dgate->dtype == CIERA_FP32 || w_gate->dtype != dgate->dtype || !same_shape(w_gate, w_up) ||
      !same_shape(dgate, dup) || (out->dtype != dgate->dtype && out->dtype != CIERA_FP32))
    return CIERA_ERR_INVALID_ARG;
  const uint64_t wk = transpose_w ? w_gate->cols : w_gate->rows, wn = transpose_w ? w_gate->rows : w_gate->cols;
  if (dgate->groups != 1 || wk != dgate->cols || !one_matrix(out, dgate->rows, wn)) return CIERA_ERR_INVALID_ARG;
  if (w_gate->groups > kMaxGroups) return CIERA_ERR_UNSUPPORTED;
  if (w_gate->groups == 0 || empty(out)) return CIERA_OK;
  if (bad_offsets(offsets, w_gate->groups, ro)) return CIERA_ERR_INVALID_ARG;
  if (bad_data(dgate) || bad_data(dup) || bad_data(w_gate) || bad_data(w_up) || bad_data(out))
    return CIERA_ERR_INVALID_ARG;
  if (overlap(ro, ra) || overlap(ro, rb) || overlap(ro, rg) || overlap(ro, ru)) return CIERA_ERR_INVALID_ARG;
  const GluXgradArgs g = {dgate->data, dup->data, w_gate->data, w_up->data, out->data, offsets, dgate->row_stride,
                          dup->row_stride, w_gate->row_stride, w_up->row_stride, w_gate->group_stride,
                          w_up->group_stride, out->row_stride, (int32_t)dgate->rows, (int32_t)dgate->cols, (int32_t)wn,
                          (int32_t)w_gate->groups};
  const bool all_flat = flat(dgate) && flat(dup) && flat(w_gate) && flat(w_up);
  return launched("gated block input gradient launch",
                  launch_glu_xgrad(dgate->dtype, out->dtype == CIERA_FP32, transpose_w == 1, all_flat, g,
                                   hip_stream(stream)));
}

ciera_status_t ciera_gq_sizes(uint32_t groups, uint64_t rows, uint64_t cols, uint32_t block, uint64_t* code_bytes,
                              uint64_t* scale_bytes, uint64_t* zero_bytes) {
  if (!code_bytes || !scale_bytes || !zero_bytes) return CIERA_ERR_INVALID_ARG;
  const ciera_gq_t q = {nullptr, nullptr, nullptr, groups, block, CIERA_BF16, 0, rows, cols};
  GqRanges r;
  if (ciera_status_t e = check_gq(&q, &r)) return e;
  *code_bytes = r.codes.bytes;
  *scale_bytes = r.scales.bytes;
  *zero_bytes = r.scales.bytes / 2;
  return CIERA_OK;
}

ciera_status_t ciera_gq_quantize(const ciera_matrix_t* x, uint32_t axis, const ciera_gq_t* q, void* stream) {
  Range rx;
  GqRanges rq;
  if (ciera_status_t e = check_matrix(x, false, &rx)) return e;
  if (ciera_status_t e = check_gq(q, &rq)) return e;
  if (axis > 1 || q->groups != x->groups || q->rows != (axis ? x->rows : x->cols) ||
      q->cols != (axis ? x->cols : x->rows))
    return CIERA_ERR_INVALID_ARG;
  if (empty(x)) return CIERA_OK;
  if (bad_data(x) || bad_data(q, rq)) return CIERA_ERR_INVALID_ARG;
  if (overlap(rx, rq) || overlap(rq.codes, rq.scales) || overlap(rq.codes, rq.zeros) || overlap(rq.scales, rq.zeros))
    return CIERA_ERR_INVALID_ARG;
  const GqQuantArgs a = {x->data, q->codes, static_cast<uint16_t*>(q->scales), q->zeros, x->row_stride,
                         x->group_stride, (int32_t)x->groups, (int32_t)x->rows, (int32_t)x->cols,
                         half_scales(q)};
  return launched("4-bit integer quantisation launch",
                  launch_gq_quantize(x->dtype, axis, q->block, a, hip_stream(stream)));
}

ciera_status_t ciera_gq_dequantize(const ciera_gq_t* q, const ciera_matrix_t* out, void* stream) {
  Range ro;
  GqRanges rq;
  if (ciera_status_t e = check_gq(q, &rq)) return e;
  if (ciera_status_t e = check_matrix(out, true, &ro)) return e;
  if (q->groups != out->groups || q->rows != out->rows || q->cols != out->cols) return CIERA_ERR_INVALID_ARG;
  if (empty(out)) return CIERA_OK;
  if (bad_data(out) || bad_data(q, rq)) return CIERA_ERR_INVALID_ARG;
  if (overlap(ro, rq)) return CIERA_ERR_INVALID_ARG;
  const GqDequantArgs a = {gq_stack(q), out->data, out->row_stride, out->group_stride, (int32_t)out->groups,
                           (int32_t)out->rows, (int32_t)out->cols, half_scales(q)};
  return launched("4-bit integer dequantisation launch",
                  launch_gq_dequantize(out->dtype, q->block, a, hip_stream(stream)));
}

static ciera_status_t gq_product(const ciera_matrix_t* x, const ciera_gq_t* w, const ciera_gq_t* w2, uint32_t act,
                                 const int32_t* offsets, const ciera_matrix_t* out, void* stream) {
  Range rx, ro;
  GqRanges rw, rw2;
  if (ciera_status_t e = check_matrix(x, false, &rx)) return e;
  if (ciera_status_t e = check_gq(w, &rw)) return e;
  if (ciera_status_t e = check_gq(w2, &rw2)) return e;
  if (ciera_status_t e = check_matrix(out, true, &ro)) return e;
  if (bad_act(act) || x->dtype == CIERA_FP32 || (out->dtype != x->dtype && out->dtype != CIERA_FP32) ||
      x->groups != 1 || x->cols != w->cols || !one_matrix(out, x->rows, w->rows))
    return CIERA_ERR_INVALID_ARG;
  if (w2->groups != w->groups || w2->block != w->block || w2->scale_dtype != w->scale_dtype || w2->rows != w->rows ||
      w2->cols != w->cols || (w2->zeros == nullptr) != (w->zeros == nullptr))
    return CIERA_ERR_INVALID_ARG;
  if (w->groups > kMaxGroups) return CIERA_ERR_UNSUPPORTED;
  if (w->groups == 0 || empty(out)) return CIERA_OK;
  if (bad_offsets(offsets, w->groups, ro)) return CIERA_ERR_INVALID_ARG;
  if (bad_data(x) || bad_data(out) || bad_data(w, rw) || bad_data(w2, rw2)) return CIERA_ERR_INVALID_ARG;
  if (overlap(ro, rx) || overlap(ro, rw) || overlap(ro, rw2)) return CIERA_ERR_INVALID_ARG;
  const GqMmArgs g = {x->data, {gq_stack(w), gq_stack(w2)}, out->data, offsets, x->row_stride, out->row_stride,
                      (int32_t)x->rows, (int32_t)x->cols, (int32_t)w->rows, (int32_t)w->groups, (int32_t)act,
                      half_scales(w), out->dtype == CIERA_FP32};
  return launched("4-bit integer product launch", launch_gq_mm(x->dtype, w != w2, w->block, flat(x), g, hip_stream(stream)));
}

ciera_status_t ciera_gq_mm(const ciera_matrix_t* x, const ciera_gq_t* w, const int32_t* offsets,
                           const ciera_matrix_t* out, void* stream) {
  return gq_product(x, w, w, CIERA_ACT_SILU, offsets, out, stream);
}

ciera_status_t ciera_gq_glu(const ciera_matrix_t* x, const ciera_gq_t* w_gate, const ciera_gq_t* w_up, uint32_t act,
                            const int32_t* offsets, const ciera_matrix_t* out, void* stream) {
  if (!w_gate || !w_up) return CIERA_ERR_INVALID_ARG;
  const ciera_gq_t second = *w_up;  // a second structure where the caller passes the same one twice
  return gq_product(x, w_gate, &second, act, offsets, out, stream);
}

}  // extern "C"
