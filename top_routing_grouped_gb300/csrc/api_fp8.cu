// api_fp8.cu -- the C ABI of the 8-bit operators (include/moe_fp8.h): argument checks,
// workspaces and launch sequences.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <new>

#include "fp8_internal.h"

struct moe_fp8_plan_s {
  bool experts;  // the expert stage (else one product)
  bool tc;       // tensor-core kernels (MOE_PATH_AUTO)
  bool few;      // ... those for few rows an expert
  int64_t rows;
  int k, n, E, n_seg, max_groups;  // expert stage: k = d, n = F
  int out_dtype;
  int64_t timeout_ns;
  // workspace: byte offsets
  size_t hdr, counts, offsets, mt_desc, pr_desc, h, h_scales, total;
  int device = -1;  // device the cached attribute belongs to
  int num_sms = 0;
};

namespace moe {
namespace fp8 {

// Which tensor-core kernels.  Those that make the weights the MMA's rows read each weight tile once for
// every 96 rows of a segment; the CTA pairs take 256 rows at the price of one.  Measured (experts;
// time of the pairs / time of the others, for 8 experts of 2048 x 8192, 32 of 2048 x 2048, 64 of
// 4096 x 2048): 16 rows a segment 1.07-1.11, 48 rows 1.04-1.08, 64 rows 1.03-1.06, 80 rows 1.01-1.04 (0.95
// for 4 of 2048 x 1024), 96 rows (half the segments need a second pass) 0.82-1.00, 128 rows 0.81-0.83.
// With few units of work (block of weight rows x group of rows) the pairs also leave SMs idle.  One
// segment: the others win as long as all units run at once (dense products K x n of 2048 x 2048, 4096 x
// 4096, 2048 x 8192, 512 x 4096, 8192 x 2048: 48 to 64 units 1.1-1.5, 96 to 128 units 1.02-1.27, 192 units
// 0.58-0.93; one row 1.3-2.7).  Several, of uneven counts: up to half of the SMs (4 of 512 x 512 and 2 of 2048 x
// 2048: 48 to 64 units 0.92-1.07, 100 0.99; 3 of 1024 x 2048: 80 units 0.99).
bool use_few(int64_t rows, int64_t n_seg, int64_t widest_out) {
  const int64_t units = ((rows + 95) / 96 + n_seg - 1) * ((widest_out + 127) / 128);
  return rows <= 72 * n_seg || units <= (n_seg == 1 ? 152 : 76);
}

}  // namespace fp8
}  // namespace moe

namespace {

using namespace moe;

moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status fail(moe_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_last_error(st, buf);
}

moe_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  return fail(MOE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Ptr {
  const void* p;
  const char* name;
  size_t align;
  bool may_be_null;
};
template <size_t N>
moe_status check(const Ptr (&ptrs)[N]) {
  for (const Ptr& q : ptrs) {
    if (!q.p && !q.may_be_null) return fail(MOE_ERR_INVALID_ARG, "%s is null", q.name);
    if (!aligned(q.p, q.align)) return fail(MOE_ERR_INVALID_ARG, "%s is not %zu-byte aligned", q.name, q.align);
  }
  return MOE_OK;
}

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

bool is_dtype(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
size_t esize(int32_t t) { return t == MOE_BF16 ? 2 : 4; }

moe_status check_sizes(int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 1) return fail(MOE_ERR_INVALID_ARG, "rows must be >= 0 and columns >= 1");
  if (ld < cols) return fail(MOE_ERR_INVALID_ARG, "a row pitch is below the row's length");
  if (rows > ((int64_t)1 << 40) / ld) return fail(MOE_ERR_UNSUPPORTED, "more than 2^40 values");
  return MOE_OK;
}

moe_status bind_device(moe_fp8_plan_t plan) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
  if (dev == plan->device) return MOE_OK;
  int sms = 0, major = 0, minor = 0;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return cuda_status(e, "cudaDeviceGetAttribute(SM count)");
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (plan->tc && !(major == 10 && minor == 3))
    return fail(MOE_ERR_UNSUPPORTED, "the tensor-core path needs an sm_103 device, found sm_%d%d", major, minor);
  plan->device = dev;
  plan->num_sms = sms;
  return MOE_OK;
}

moe_status make_plan(bool experts, int64_t rows, int32_t k, int32_t n, int32_t E, int32_t W, int32_t out_dtype,
                     int32_t path, int64_t timeout_ns, moe_fp8_plan_t* plan, size_t* workspace_bytes) {
  *plan = nullptr;
  if (rows < 1 || k < 1 || n < 1 || E < 1 || W < 1)
    return fail(MOE_ERR_INVALID_ARG, "rows, columns, experts and sources must be >= 1");
  if ((int64_t)E * W > kMaxExperts) return fail(MOE_ERR_INVALID_ARG, "n_sources * n_experts must be <= %d", kMaxExperts);
  if (path != MOE_PATH_AUTO && path != MOE_PATH_SIMT)
    return fail(MOE_ERR_INVALID_ARG, "the 8-bit products run on MOE_PATH_AUTO or MOE_PATH_SIMT");
  const bool tc = path == MOE_PATH_AUTO;
  if (tc && (k % 16 != 0 || n % 16 != 0))
    return fail(MOE_ERR_UNSUPPORTED, "the tensor-core path needs multiples of 16 columns (use MOE_PATH_SIMT)");
  const int64_t widest = k > n ? k : n;
  if (rows > INT32_MAX / 2 || rows > ((int64_t)1 << 40) / widest || (int64_t)E * widest > INT32_MAX / 8)
    return fail(MOE_ERR_UNSUPPORTED, "too many rows or weight rows");
  moe_fp8_plan_s* p = new (std::nothrow) moe_fp8_plan_s();
  if (!p) return fail(MOE_ERR_INTERNAL, "out of host memory");
  p->experts = experts;
  p->tc = tc;
  p->few = tc && fp8::use_few(rows, (int64_t)E * W, experts && k > n ? k : n);
  p->rows = rows;
  p->k = k;
  p->n = n;
  p->E = E;
  p->n_seg = E * W;
  p->out_dtype = out_dtype;
  p->timeout_ns = timeout_ns <= 0 ? 2000000000LL : timeout_ns < (int64_t)fp8::kMinTimeoutNs ? (int64_t)fp8::kMinTimeoutNs : timeout_ns;
  // groups of up to kGroupM m-tiles per segment, as moe_plan bounds them per expert
  p->max_groups = (int)(rows / ((int64_t)kTileM * kGroupM) + 2 * (int64_t)p->n_seg + 2);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  p->hdr = take(64 * sizeof(uint32_t));
  p->counts = take((size_t)p->n_seg * 4);
  p->offsets = take(((size_t)p->n_seg + 1) * 4);
  p->mt_desc = take((size_t)p->max_groups * kGroupM * 16);
  p->pr_desc = take((size_t)p->max_groups * (kGroupM / 2) * 16);
  if (experts) {
    p->h = take((size_t)rows * (size_t)n);
    p->h_scales = take((size_t)rows * (size_t)fp8::scale_cols(n));
  }
  p->total = off;
  *plan = p;
  *workspace_bytes = off;
  return set_last_error(MOE_OK, "");
}

// Tile tables of this call's segments (the tensor-core kernels find their tiles themselves).
moe_status begin(moe_fp8_plan_t plan, const int32_t* seg_counts, void* workspace, cudaStream_t st, Ws* ws) {
  moe_status s = bind_device(plan);
  if (s != MOE_OK) return s;
  char* b = static_cast<char*>(workspace);
  *ws = Ws{};
  ws->hdr = reinterpret_cast<uint32_t*>(b + plan->hdr);
  ws->counts = reinterpret_cast<int32_t*>(b + plan->counts);
  ws->offsets = reinterpret_cast<int32_t*>(b + plan->offsets);
  ws->mt_desc = reinterpret_cast<int4*>(b + plan->mt_desc);
  ws->pr_desc = reinterpret_cast<int4*>(b + plan->pr_desc);
  if (plan->tc) return MOE_OK;
  Shape shape{};
  shape.N = plan->rows;
  shape.max_groups = plan->max_groups;
  return cuda_status(fp8::launch_segments(shape, *ws, seg_counts, plan->n_seg, plan->E, st), "launching the segment scan");
}

moe_status product(moe_fp8_plan_t plan, int kind, const fp8::GemmArgs& g, const Ws& ws, const int32_t* seg_counts, bool first,
                   cudaStream_t st, const char* what) {
  cudaError_t e;
  if (!plan->tc)
    e = fp8::launch_gemm_simt(kind, g, ws, plan->num_sms, st);
  else
    e = (plan->few ? fp8::launch_gemm_few : fp8::launch_gemm_tc)(kind, g, ws, seg_counts, plan->n_seg, first, plan->device,
                                                                 plan->num_sms, plan->timeout_ns, st);
  return cuda_status(e, what);
}

moe_status check_workspace(moe_fp8_plan_t plan, const void* workspace, size_t bytes) {
  if (!workspace || !aligned(workspace, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (bytes < plan->total) return fail(MOE_ERR_INVALID_ARG, "workspace too small: %zu < %zu", bytes, plan->total);
  return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_fp8_scale_cols(int64_t cols) { return cols < 1 ? 0 : fp8::scale_cols(cols); }

moe_status moe_fp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx, int32_t block_rows,
                            int64_t expert_rows, void* q, uint8_t* scales, void* stream) {
  if (!is_dtype(x_dtype)) return fail(MOE_ERR_INVALID_ARG, "bad x_dtype");
  if (block_rows != 1 && block_rows != fp8::kBlock) return fail(MOE_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  moe_status s = check_sizes(rows, cols, ldx);
  if (s != MOE_OK) return s;
  if (block_rows == fp8::kBlock && (expert_rows < 1 || rows % expert_rows != 0))
    return fail(MOE_ERR_INVALID_ARG, "rows must be a multiple of expert_rows >= 1");
  if (rows == 0) return set_last_error(MOE_OK, "");
  const Ptr ptrs[] = {{x, "x", esize(x_dtype), false}, {q, "q", 16, false}, {scales, "scales", 16, false}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  const bool bf16 = x_dtype == MOE_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_status(block_rows == 1
                         ? fp8::launch_quantize_rows(x, bf16, rows, cols, ldx, q, scales, st)
                         : fp8::launch_quantize_blocks(x, bf16, rows, cols, ldx, expert_rows, q, scales, st),
                     "launching the quantisation");
}

moe_status moe_rmsnorm(const void* x, const void* residual, const float* weight, int32_t dtype, int64_t rows, int32_t d,
                       int64_t ldx, int64_t ldr, float eps, void* residual_out, void* out, void* q, uint8_t* scales,
                       float* rstd, void* stream) {
  if (!is_dtype(dtype)) return fail(MOE_ERR_INVALID_ARG, "bad dtype");
  if (!(eps >= 0.f) || !isfinite(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  moe_status s = check_sizes(rows, d, ldx);
  if (s != MOE_OK) return s;
  if (residual && ldr < d) return fail(MOE_ERR_INVALID_ARG, "a row pitch is below the row's length");
  if (d > fp8::kMaxNormCols) return fail(MOE_ERR_UNSUPPORTED, "d must be <= %d", fp8::kMaxNormCols);
  if (rows == 0) return set_last_error(MOE_OK, "");
  if (!q != !scales) return fail(MOE_ERR_INVALID_ARG, "q and scales go together");
  if (!residual_out && !out && !q && !rstd) return fail(MOE_ERR_INVALID_ARG, "no output is wanted");
  if ((residual_out == x && residual_out && ldx != d) || (residual && residual_out == residual && ldr != d))
    return fail(MOE_ERR_INVALID_ARG, "in place needs a pitch of d");
  const size_t a = esize(dtype);
  const Ptr ptrs[] = {{x, "x", a, false},     {residual, "residual", a, true}, {weight, "weight", 16, true},
                      {residual_out, "residual_out", a, true}, {out, "out", a, true},     {q, "q", 16, true},
                      {scales, "scales", 16, true},    {rstd, "rstd", 16, true}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  return cuda_status(fp8::launch_rmsnorm(x, residual, weight, dtype == MOE_BF16, rows, d, ldx, ldr, eps, residual_out, out,
                                         q, scales, rstd, static_cast<cudaStream_t>(stream)),
                     "launching the norm");
}

size_t moe_rmsnorm_backward_workspace(int64_t rows, int32_t d) {
  if (rows < 0 || d < 1) return 0;
  return ((size_t)fp8::rmsnorm_backward_parts(rows, d) * (size_t)d * sizeof(float) + 255) / 256 * 256;
}

moe_status moe_rmsnorm_backward(const void* dout, int32_t dout_dtype, const void* r, const float* weight,
                                const float* rstd, const void* dresidual, int32_t dtype, int64_t rows, int32_t d,
                                int64_t ldr, void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!is_dtype(dtype) || !is_dtype(dout_dtype)) return fail(MOE_ERR_INVALID_ARG, "bad dtype");
  moe_status s = check_sizes(rows, d, ldr);
  if (s != MOE_OK) return s;
  if (d > fp8::kMaxNormCols) return fail(MOE_ERR_UNSUPPORTED, "d must be <= %d", fp8::kMaxNormCols);
  const size_t a = esize(dtype);
  const bool any = rows > 0;
  const Ptr ptrs[] = {{dout, "dout", esize(dout_dtype), !any}, {r, "r", a, !any},          {weight, "weight", 16, true},
                      {rstd, "rstd", 16, !any},                {dresidual, "dresidual", a, true}, {dx, "dx", a, !any},
                      {dweight, "dweight", 16, true}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  if (any) {  // in place only where every row of dx lies on its own row of the input
    const size_t row = (size_t)d * a, bytes = (size_t)rows * row;
    const size_t dout_bytes = (size_t)rows * (size_t)d * esize(dout_dtype), r_bytes = (size_t)(rows - 1) * (size_t)ldr * a + row;
    if (overlap(dx, bytes, dout, dout_bytes) && !(dx == dout && dtype == dout_dtype))
      return fail(MOE_ERR_INVALID_ARG, "dx overlaps dout: it may only be dout itself, of its type");
    if (overlap(dx, bytes, r, r_bytes) && !(dx == r && ldr == d))
      return fail(MOE_ERR_INVALID_ARG, "dx overlaps r: it may only be r itself, with a pitch of d");
    if (dresidual && overlap(dx, bytes, dresidual, bytes) && dx != dresidual)
      return fail(MOE_ERR_INVALID_ARG, "dx overlaps dresidual: it may only be dresidual itself");
  }
  const size_t need = moe_rmsnorm_backward_workspace(rows, d);
  if (dweight && need > 0) {
    if (!workspace || !aligned(workspace, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < need) return fail(MOE_ERR_INVALID_ARG, "workspace too small: %zu < %zu", workspace_bytes, need);
  }
  return cuda_status(fp8::launch_rmsnorm_backward(dout, dout_dtype == MOE_BF16, r, weight, rstd, dresidual,
                                                  dtype == MOE_BF16, rows, d, ldr, dx, dweight,
                                                  static_cast<float*>(workspace), static_cast<cudaStream_t>(stream)),
                     "launching the norm's backward");
}

moe_status moe_fp8_matmul_plan(const moe_fp8_matmul_config* cfg, moe_fp8_plan_t* plan, size_t* workspace_bytes) {
  if (!cfg || !plan || !workspace_bytes) return fail(MOE_ERR_INVALID_ARG, "null argument");
  if (!is_dtype(cfg->out_dtype)) return fail(MOE_ERR_INVALID_ARG, "bad out_dtype");
  return make_plan(false, cfg->max_rows, cfg->k, cfg->n, cfg->n_experts, cfg->n_sources, cfg->out_dtype, cfg->path,
                   cfg->wait_timeout_ns, plan, workspace_bytes);
}

moe_status moe_fp8_expert_plan(const moe_expert_config* cfg, moe_fp8_plan_t* plan, size_t* workspace_bytes) {
  if (!cfg || !plan || !workspace_bytes) return fail(MOE_ERR_INVALID_ARG, "null argument");
  return make_plan(true, cfg->max_rows, cfg->d_model, cfg->d_expert, cfg->n_local_experts, cfg->n_sources, MOE_BF16,
                   cfg->path, cfg->wait_timeout_ns, plan, workspace_bytes);
}

void moe_fp8_plan_destroy(moe_fp8_plan_t plan) { delete plan; }

moe_status moe_fp8_matmul(moe_fp8_plan_t plan, const int32_t* seg_counts, const void* a, const uint8_t* a_scales,
                          const void* w, const uint8_t* w_scales, void* out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (!plan) return fail(MOE_ERR_INVALID_ARG, "null plan");
  if (plan->experts) return fail(MOE_ERR_INVALID_ARG, "moe_fp8_matmul needs a plan made by moe_fp8_matmul_plan");
  const Ptr ptrs[] = {{seg_counts, "seg_counts", 16, plan->n_seg == 1}, {a, "a", 16, false}, {a_scales, "a_scales", 16, false},
                      {w, "w", 16, false}, {w_scales, "w_scales", 16, false}, {out, "out", 16, false}};
  moe_status s = check(ptrs);
  if (s != MOE_OK || (s = check_workspace(plan, workspace, workspace_bytes)) != MOE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Ws ws;
  if ((s = begin(plan, seg_counts, workspace, st, &ws)) != MOE_OK) return s;
  fp8::GemmArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.sa = a_scales;
  g.b = static_cast<const uint8_t*>(w);
  g.sb = w_scales;
  g.out = out;
  g.rows = plan->rows;
  g.n = plan->n;
  g.K = plan->k;
  g.E = plan->E;
  return product(plan, plan->out_dtype == MOE_BF16 ? fp8::kOutBf16 : fp8::kOutF32, g, ws, seg_counts, true, st,
                 "launching the product");
}

moe_status moe_fp8_expert_forward(moe_fp8_plan_t plan, const int32_t* seg_counts, const void* x_rows,
                                  const uint8_t* x_scales, const float* gates, const void* w1, const uint8_t* w1_scales,
                                  const void* w3, const uint8_t* w3_scales, const void* w2, const uint8_t* w2_scales,
                                  void* y_rows, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan) return fail(MOE_ERR_INVALID_ARG, "null plan");
  if (!plan->experts) return fail(MOE_ERR_INVALID_ARG, "moe_fp8_expert_forward needs a plan made by moe_fp8_expert_plan");
  const Ptr ptrs[] = {{seg_counts, "seg_counts", 16, plan->n_seg == 1},
                      {x_rows, "x_rows", 16, false},
                      {x_scales, "x_scales", 16, false},
                      {gates, "gates", 16, false},
                      {w1, "w1", 16, false},
                      {w1_scales, "w1_scales", 16, false},
                      {w3, "w3", 16, false},
                      {w3_scales, "w3_scales", 16, false},
                      {w2, "w2", 16, false},
                      {w2_scales, "w2_scales", 16, false},
                      {y_rows, "y_rows", 16, false}};
  moe_status s = check(ptrs);
  if (s != MOE_OK || (s = check_workspace(plan, workspace, workspace_bytes)) != MOE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Ws ws;
  if ((s = begin(plan, seg_counts, workspace, st, &ws)) != MOE_OK) return s;
  uint8_t* b = static_cast<uint8_t*>(workspace);
  fp8::GemmArgs g{};
  g.a = static_cast<const uint8_t*>(x_rows);
  g.sa = x_scales;
  g.b = static_cast<const uint8_t*>(w1);
  g.sb = w1_scales;
  g.b3 = static_cast<const uint8_t*>(w3);
  g.sb3 = w3_scales;
  g.out = b + plan->h;
  g.out_scales = b + plan->h_scales;
  g.rows = plan->rows;
  g.n = plan->n;
  g.K = plan->k;
  g.E = plan->E;
  if ((s = product(plan, fp8::kSwiGLU, g, ws, seg_counts, true, st, "launching the SwiGLU product")) != MOE_OK) return s;
  g.a = b + plan->h;
  g.sa = b + plan->h_scales;
  g.b = static_cast<const uint8_t*>(w2);
  g.sb = w2_scales;
  g.b3 = nullptr;
  g.sb3 = nullptr;
  g.gate = gates;
  g.out = y_rows;
  g.out_scales = nullptr;
  g.n = plan->k;
  g.K = plan->n;
  return product(plan, fp8::kOutBf16, g, ws, seg_counts, false, st, "launching the down-projection");
}

moe_status moe_fp8_get_device_status(moe_fp8_plan_t plan, const void* workspace, void* stream) {
  if (!plan || !workspace) return fail(MOE_ERR_INVALID_ARG, "null argument");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_status(e, "synchronising the stream");
  uint32_t hdr[2] = {0, 0};
  e = cudaMemcpy(hdr, static_cast<const char*>(workspace) + plan->hdr, sizeof hdr, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_status(e, "reading the status word");
  if (hdr[0] == 0) return MOE_OK;
  if (hdr[0] == MOE_ERR_TIMEOUT || hdr[0] == MOE_ERR_INTERNAL)
    return fail((moe_status)hdr[0], "device reported %s at site 0x%x", moe_status_string((moe_status)hdr[0]), hdr[1]);
  return fail(MOE_ERR_INTERNAL, "device status word holds unknown value %u", hdr[0]);
}

moe_status moe_checkpoint_save_rows(const void* a, const void* b, int64_t rows, int32_t F, void* qa, uint8_t* sa,
                                    void* qb, uint8_t* sb, void* stream) {
  moe_status s = check_sizes(rows, F, F);
  if (s != MOE_OK) return s;
  if (rows == 0) return set_last_error(MOE_OK, "");
  const Ptr ptrs[] = {{a, "a", 16, false},   {b, "b", 16, false},   {qa, "qa", 16, false},
                      {sa, "sa", 16, false}, {qb, "qb", 16, false}, {sb, "sb", 16, false}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  return cuda_status(fp8::launch_checkpoint_save(a, b, rows, F, qa, sa, qb, sb, static_cast<cudaStream_t>(stream)),
                     "launching the checkpoint");
}

moe_status moe_checkpoint_restore_rows(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb, int64_t rows,
                                       int32_t F, void* a, void* b, void* h, void* stream) {
  moe_status s = check_sizes(rows, F, F);
  if (s != MOE_OK) return s;
  if (rows == 0) return set_last_error(MOE_OK, "");
  const Ptr ptrs[] = {{qa, "qa", 16, false}, {sa, "sa", 16, false}, {qb, "qb", 16, false}, {sb, "sb", 16, false},
                      {a, "a", 16, true},    {b, "b", 16, true},    {h, "h", 16, true}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  if (!a && !b && !h) return fail(MOE_ERR_INVALID_ARG, "no output is wanted");
  return cuda_status(fp8::launch_checkpoint_restore(qa, sa, qb, sb, rows, F, a, b, h, static_cast<cudaStream_t>(stream)),
                     "launching the restore");
}

moe_status moe_checkpoint_backward_rows(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb,
                                        const void* dh, int64_t rows, int32_t F, void* da, void* db, void* h,
                                        void* stream) {
  moe_status s = check_sizes(rows, F, F);
  if (s != MOE_OK) return s;
  if (rows == 0) return set_last_error(MOE_OK, "");
  const Ptr ptrs[] = {{qa, "qa", 16, false}, {sa, "sa", 16, false}, {qb, "qb", 16, false}, {sb, "sb", 16, false},
                      {dh, "dh", 16, false}, {da, "da", 16, false}, {db, "db", 16, false}, {h, "h", 16, true}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  return cuda_status(
      fp8::launch_checkpoint_backward(qa, sa, qb, sb, dh, rows, F, da, db, h, static_cast<cudaStream_t>(stream)),
      "launching the SwiGLU backward");
}

}  // extern "C"
