// api_rows.cu -- the C ABI of the rows around an expert stage (include/moe_rows.h): argument checks and
// launches.
#include "host_checks.h"
#include "rows_internal.h"

namespace {

using namespace moe;

constexpr int64_t kMostValues = (int64_t)1 << 40;

moe_status check_slots(int64_t T, int32_t k) {
  if (T < 0 || k < 1 || k > rows::kMaxK) return fail(MOE_ERR_INVALID_ARG, "T must be >= 0 and k 1 to %d", rows::kMaxK);
  if (T > INT32_MAX / k) return fail(MOE_ERR_UNSUPPORTED, "T * k must be below 2^31");
  return MOE_OK;
}

moe_status check_experts(int32_t E) {
  if (E < 1 || E > rows::kMaxSortExperts) return fail(MOE_ERR_INVALID_ARG, "n_experts must be 1 to %d", rows::kMaxSortExperts);
  return MOE_OK;
}

// Rows of T tokens and of a buffer of R.
moe_status check_rows(int64_t T, int64_t R, int64_t d, int64_t ld) {
  if (R < 0 || d < 1) return fail(MOE_ERR_INVALID_ARG, "R must be >= 0 and d >= 1");
  if (ld < d) return fail(MOE_ERR_INVALID_ARG, "a row pitch is below the row's length");
  if (T > kMostValues / ld || R > kMostValues / d) return fail(MOE_ERR_UNSUPPORTED, "more than 2^40 values");
  return MOE_OK;
}

struct Span {
  const void* p;
  size_t bytes;
  const char* name;
};

// The written arrays overlap neither each other nor the read ones.
template <size_t W, size_t N>
moe_status check_apart(const Span (&written)[W], const Span (&read)[N]) {
  for (size_t i = 0; i < W; ++i) {
    if (!written[i].p) continue;
    for (size_t j = i + 1; j < W; ++j)
      if (written[j].p && overlap(written[i].p, written[i].bytes, written[j].p, written[j].bytes))
        return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", written[i].name, written[j].name);
    for (const Span& r : read)
      if (r.p && overlap(written[i].p, written[i].bytes, r.p, r.bytes))
        return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", written[i].name, r.name);
  }
  return MOE_OK;
}

size_t pitched(int64_t n, int64_t d, int64_t ld, int64_t size) { return n < 1 ? 0 : ((size_t)(n - 1) * ld + d) * size; }

moe_status sort_and_gather(const void* idx, int32_t idx_bytes, int64_t T, int32_t k, int32_t E, int32_t* counts, int32_t* slot_pos,
                           int32_t* row_slot, bool moves, const void* x, int32_t elem_bytes, int64_t d, int64_t ldx, int64_t R,
                           void* x_rows, const uint8_t* x_scales, uint8_t* row_scales, int64_t scale_bytes, const float* gates,
                           float* row_gates, bool sorts, void* workspace, size_t workspace_bytes, void* stream) {
  moe_status s = check_slots(T, k);
  if (s != MOE_OK) return s;
  const int64_t N = T * k;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (sorts) {
    if ((s = check_experts(E)) != MOE_OK) return s;
    if (idx_bytes != 4 && idx_bytes != 8) return fail(MOE_ERR_INVALID_ARG, "idx_bytes must be 4 or 8");
    const Ptr ptrs[] = {{idx, "idx", (size_t)idx_bytes, T == 0}, {counts, "counts", 4, false}, {row_slot, "row_slot", 4, true}};
    if ((s = check(ptrs)) != MOE_OK) return s;
  }
  if (moves) {
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return fail(MOE_ERR_INVALID_ARG, "elem_bytes must be 1, 2 or 4");
    if ((s = check_rows(T, R, d, ldx)) != MOE_OK) return s;
    const bool any = T > 0 && R > 0;  // an array without values may be null
    if (any && !x_scales != !row_scales) return fail(MOE_ERR_INVALID_ARG, "x_scales and row_scales go together");
    if (any && !gates != !row_gates) return fail(MOE_ERR_INVALID_ARG, "gates and row_gates go together");
    if (x_scales && (scale_bytes < 4 || scale_bytes % 4 != 0 || scale_bytes > kMostValues || R > kMostValues / scale_bytes || T > kMostValues / scale_bytes))
      return fail(MOE_ERR_INVALID_ARG, "scale_bytes must be a multiple of 4");
    const Ptr ptrs[] = {{x, "x", (size_t)elem_bytes, T == 0}, {x_rows, "x_rows", (size_t)elem_bytes, T == 0 || R == 0},
                        {x_scales, "x_scales", 4, true}, {row_scales, "row_scales", 4, true},
                        {gates, "gates", 4, true}, {row_gates, "row_gates", 4, true}};
    if ((s = check(ptrs)) != MOE_OK) return s;
  }
  const Ptr ptrs[] = {{slot_pos, "slot_pos", 4, T == 0}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  const size_t need = sorts ? moe_rows_workspace(T, k, E) : 0;
  if (need > 0) {
    if (!workspace || !aligned(workspace, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < need) return fail(MOE_ERR_INVALID_ARG, "workspace too small: %zu < %zu", workspace_bytes, need);
  }
  const size_t slots = (size_t)N * 4;
  const Span read_only[] = {{idx, sorts ? (size_t)N * idx_bytes : 0, "idx"},
                            {x, moves ? pitched(T, d, ldx, elem_bytes) : 0, "x"},
                            {x_scales, moves ? (size_t)T * scale_bytes : 0, "x_scales"},
                            {gates, slots, "gates"},
                            {sorts ? nullptr : slot_pos, slots, "slot_pos"}};
  const Span written[] = {{counts, sorts ? (size_t)E * 4 : 0, "counts"},
                          {sorts ? slot_pos : nullptr, slots, "slot_pos"},
                          {row_slot, sorts ? slots : 0, "row_slot"},
                          {x_rows, moves ? pitched(R, d, d, elem_bytes) : 0, "x_rows"},
                          {row_scales, moves && row_scales ? (size_t)R * scale_bytes : 0, "row_scales"},
                          {row_gates, moves ? (size_t)R * 4 : 0, "row_gates"},
                          {workspace, need, "the workspace"}};
  if ((s = check_apart(written, read_only)) != MOE_OK) return s;
  if (T == 0)
    return sorts ? cuda_status(cudaMemsetAsync(counts, 0, (size_t)E * 4, st), "clearing counts") : set_last_error(MOE_OK, "");

  rows::Args a{};
  a.idx = sorts ? idx : nullptr;
  a.idx64 = idx_bytes == 8;
  a.T = T;
  a.k = k;
  a.E = E;
  a.counts = counts;
  a.slot_pos = slot_pos;
  a.row_slot = row_slot;
  a.R = R;
  if (moves) {
    a.x = static_cast<const char*>(x);
    a.row_bytes = d * elem_bytes;
    a.ld_bytes = ldx * elem_bytes;
    a.x_rows = static_cast<char*>(x_rows);
    if (x_scales) {
      a.x_words = reinterpret_cast<const uint32_t*>(x_scales);
      a.row_words = reinterpret_cast<uint32_t*>(row_scales);
      a.words = scale_bytes / 4;
    }
    a.gates = gates;
    a.row_gates = row_gates;
  }
  return cuda_status(rows::launch_rows(a, need > 0 ? static_cast<int32_t*>(workspace) : nullptr, st), "launching the sorted rows");
}

}  // namespace

extern "C" {

size_t moe_rows_workspace(int64_t T, int32_t k, int32_t n_experts) {
  if (T < 0 || k < 1 || k > rows::kMaxK || T > INT32_MAX / k || n_experts < 1 || n_experts > rows::kMaxSortExperts) return 0;
  return rows::counts_first(T * k) ? ((size_t)rows::kCountBlocks * rows::count_pitch(n_experts) * sizeof(int32_t) + 255) / 256 * 256 : 0;
}

moe_status moe_rows_sort(const void* idx, int32_t idx_bytes, int64_t T, int32_t k, int32_t n_experts, int32_t* counts,
                         int32_t* slot_pos, int32_t* row_slot, void* workspace, size_t workspace_bytes, void* stream) {
  return sort_and_gather(idx, idx_bytes, T, k, n_experts, counts, slot_pos, row_slot, false, nullptr, 0, 0, 0, 0, nullptr, nullptr,
                         nullptr, 0, nullptr, nullptr, true, workspace, workspace_bytes, stream);
}

moe_status moe_rows_gather(const int32_t* slot_pos, int64_t T, int32_t k, const void* x, int32_t elem_bytes, int64_t d, int64_t ldx,
                           int64_t R, void* x_rows, const uint8_t* x_scales, uint8_t* row_scales, int64_t scale_bytes,
                           const float* gates, float* row_gates, void* stream) {
  return sort_and_gather(nullptr, 4, T, k, 1, nullptr, const_cast<int32_t*>(slot_pos), nullptr, true, x, elem_bytes, d, ldx, R, x_rows,
                         x_scales, row_scales, scale_bytes, gates, row_gates, false, nullptr, 0, stream);
}

moe_status moe_rows_dispatch(const void* idx, int32_t idx_bytes, int64_t T, int32_t k, int32_t n_experts, int32_t* counts,
                             int32_t* slot_pos, int32_t* row_slot, const void* x, int32_t elem_bytes, int64_t d, int64_t ldx, int64_t R,
                             void* x_rows, const uint8_t* x_scales, uint8_t* row_scales, int64_t scale_bytes, const float* gates,
                             float* row_gates, void* workspace, size_t workspace_bytes, void* stream) {
  return sort_and_gather(idx, idx_bytes, T, k, n_experts, counts, slot_pos, row_slot, true, x, elem_bytes, d, ldx, R, x_rows, x_scales,
                         row_scales, scale_bytes, gates, row_gates, true, workspace, workspace_bytes, stream);
}

moe_status moe_rows_combine(const void* y_rows, int32_t y_dtype, int64_t R, const int32_t* slot_pos, const float* gates, int64_t T,
                            int32_t k, int64_t d, const void* residual, void* out, int32_t out_dtype, void* stream) {
  if (!is_dtype(y_dtype) || !is_dtype(out_dtype)) return fail(MOE_ERR_INVALID_ARG, "bad dtype");
  moe_status s = check_slots(T, k);
  if (s != MOE_OK || (s = check_rows(T, R, d, d)) != MOE_OK) return s;
  if (T == 0) return set_last_error(MOE_OK, "");
  const size_t o = esize(out_dtype), slots = (size_t)(T * k) * 4, out_bytes = (size_t)(T * d) * o;
  const Ptr ptrs[] = {{y_rows, "y_rows", esize(y_dtype), R == 0}, {slot_pos, "slot_pos", 4, false}, {gates, "gates", 4, true},
                      {residual, "residual", o, true}, {out, "out", o, false}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  const Span written[] = {{out, out_bytes, "out"}};
  const Span read[] = {{y_rows, (size_t)(R * d) * esize(y_dtype), "y_rows"}, {slot_pos, slots, "slot_pos"}, {gates, slots, "gates"},
                       {residual == out ? nullptr : residual, out_bytes, "residual: it may only be residual itself"}};
  if ((s = check_apart(written, read)) != MOE_OK) return s;
  return cuda_status(rows::launch_combine(y_rows, y_dtype == MOE_BF16, R, slot_pos, gates, T, k, d, residual, out, out_dtype == MOE_BF16,
                                          static_cast<cudaStream_t>(stream)),
                     "launching the combine");
}

moe_status moe_rows_combine_backward(const void* dout, int32_t dout_dtype, const int32_t* slot_pos, const float* gates, int64_t T,
                                     int32_t k, int64_t d, int64_t R, const void* y_rows, void* dy_rows, int32_t y_dtype, float* dgates,
                                     void* stream) {
  if (!is_dtype(dout_dtype) || !is_dtype(y_dtype)) return fail(MOE_ERR_INVALID_ARG, "bad dtype");
  moe_status s = check_slots(T, k);
  if (s != MOE_OK || (s = check_rows(T, R, d, d)) != MOE_OK) return s;
  if (!dy_rows && !dgates && R > 0) return fail(MOE_ERR_INVALID_ARG, "no output is wanted");
  if (T == 0) return set_last_error(MOE_OK, "");
  const size_t a = esize(y_dtype), slots = (size_t)(T * k) * 4, row_bytes = (size_t)(R * d) * a;
  const Ptr ptrs[] = {{dout, "dout", esize(dout_dtype), false}, {slot_pos, "slot_pos", 4, false}, {gates, "gates", 4, true},
                      {y_rows, "y_rows", a, !dgates || R == 0}, {dy_rows, "dy_rows", a, true}, {dgates, "dgates", 4, true}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  const Span written[] = {{dy_rows, row_bytes, "dy_rows"}, {dgates, slots, "dgates"}};
  const Span read[] = {{dout, (size_t)(T * d) * esize(dout_dtype), "dout"}, {slot_pos, slots, "slot_pos"}, {gates, slots, "gates"},
                       {y_rows == dy_rows ? nullptr : y_rows, row_bytes, "y_rows: it may only be y_rows itself"}};
  if ((s = check_apart(written, read)) != MOE_OK) return s;
  return cuda_status(rows::launch_combine_backward(dout, dout_dtype == MOE_BF16, slot_pos, gates, T, k, d, R, y_rows, dy_rows,
                                                   y_dtype == MOE_BF16, dgates, static_cast<cudaStream_t>(stream)),
                     "launching the combine's backward");
}

}  // extern "C"
