// rcc_adamw_host.cpp -- plans of the AdamW step over many tensors: checks, the
// tables in the caller's workspace, and the step's launches.
//
// A plan is checked once, where it is made; a step checks its numbers alone and
// launches.  The workspace holds, each on a boundary of 256 bytes: the status
// with the decision and a counter behind it, the norm's rows, the tensors, the
// items.
#include <new>
#include <unordered_map>

#include "host_internal.h"
#include "lm_internal.h"

struct rcc_adamw_s;

using namespace rcc::host;
using namespace rcc::lm;

namespace {

struct Plan {
  char* workspace = nullptr;
  size_t tensors_at = 0, items_at = 0;
  uint64_t items = 0;
  int sms = 0, device = 0;
  uint32_t seed = 0;
  bool eight = false, all_bf16 = true;
};

std::mutex g_plans_mu;
std::unordered_map<uintptr_t, Plan> g_plans;
uintptr_t g_next_plan = 0;

constexpr size_t kDecisionAt = 64, kArrivedAt = 128, kRowsAt = 256;
constexpr size_t kMaxNumel = size_t{1} << 40;
constexpr uint64_t kMaxItems = 0x7FFFFFFF;
static_assert(sizeof(rcc_adamw_status) <= kDecisionAt &&
                  kDecisionAt + sizeof(AdamWDecision) <= kArrivedAt,
              "status and decision share the first 256 bytes");

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Items of all tensors; 0 for tensors that no plan takes
uint64_t count_items(const rcc_adamw_tensor* t, int n) {
  if (!t || n < 1) return 0;
  uint64_t items = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].numel < 1 || t[i].numel > kMaxNumel) return 0;
    items += (t[i].numel + kAdamWItem - 1) / kAdamWItem;
    if (items > kMaxItems) return 0;
  }
  return items;
}

struct Layout {
  size_t tensors_at, items_at, bytes;
};
Layout layout_of(int n, uint64_t items, int rows) {
  Layout l;
  l.tensors_at = kRowsAt + round256((size_t)rows * sizeof(AdamWRow));
  l.items_at = l.tensors_at + round256((size_t)n * sizeof(AdamWTensor));
  l.bytes = l.items_at + round256((size_t)items * sizeof(AdamWItem));
  return l;
}

bool on(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

rcc_status check_tensor(const rcc_adamw_tensor& t, int i, bool eight) {
  const rcc_status bad = RCC_ERR_INVALID_ARGUMENT;
  if (t.grad_type != RCC_F32 && t.grad_type != RCC_BF16)
    return fail(bad, "tensor %d: grad_type %d is not an rcc_dtype", i, (int)t.grad_type);
  if (!t.grad || !t.param || !t.exp_avg || !t.exp_avg_sq)
    return fail(bad, "tensor %d lacks a gradient, parameter or state", i);
  if (!t.exp_avg_scale != !eight || !t.exp_avg_sq_scale != !eight)
    return fail(bad, "tensor %d: all states of a plan are fp32, or all have scales", i);
  const size_t grad = t.grad_type == RCC_BF16 ? 2 : 4, state = eight ? 1 : 4;
  if (!on(t.grad, grad) || !on(t.param, 4) || !on(t.exp_avg, state) || !on(t.exp_avg_sq, state) ||
      !on(t.exp_avg_scale, 4) || !on(t.exp_avg_sq_scale, 4) || !on(t.copy, 2))
    return fail(bad, "tensor %d: a buffer is not aligned to its elements", i);
  return RCC_OK;
}

// Vectors of eight elements: fp32 ones on boundaries of `fp32` bytes
bool vectors_of(const rcc_adamw_tensor& t, bool eight, size_t fp32) {
  const size_t state = eight ? 8 : fp32;
  return on(t.grad, t.grad_type == RCC_BF16 ? 16 : fp32) && on(t.param, fp32) &&
         on(t.exp_avg, state) && on(t.exp_avg_sq, state) && on(t.copy, 16);
}

rcc_status create(const rcc_adamw_tensor* tensors, int n, uint32_t seed, int64_t step,
                  double beta1, double beta2, void* workspace, size_t workspace_bytes,
                  rcc_stream_t stream, rcc_adamw* out) {
  const rcc_status bad = RCC_ERR_INVALID_ARGUMENT;
  if (!out) return fail(bad, "out is NULL");
  *out = nullptr;
  if (!tensors || n < 1) return fail(bad, "tensors and num_tensors >= 1 are required");
  const uint64_t items = count_items(tensors, n);
  if (!items)
    return fail(bad, "a tensor has no elements or over 2^40, or there are over 2^31 pieces of %d",
                kAdamWItem);
  if (step < 0) return fail(bad, "step must be >= 0");
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0))
    return fail(bad, "betas must lie in [0, 1)");
  const bool eight = tensors[0].exp_avg_scale != nullptr;
  for (int i = 0; i < n; ++i) {
    const rcc_status st = check_tensor(tensors[i], i, eight);
    if (st != RCC_OK) return st;
  }
  if (!workspace || !on(workspace, 256))
    return fail(bad, "workspace must be given, 256-byte aligned");
  const int sms = adamw_sms();
  const Layout l = layout_of(n, items, adamw_rows(sms));
  if (workspace_bytes < l.bytes)
    return fail(RCC_ERR_SHAPE_MISMATCH, "the workspace has %zu bytes, %zu are needed",
                workspace_bytes, l.bytes);
  std::vector<RwSpan> spans;
  spans.reserve((size_t)n * 7 + 1);
  auto add = [&](const void* p, size_t bytes, bool written) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (p) spans.push_back({at, at + bytes, written});
  };
  add(workspace, l.bytes, true);
  for (int i = 0; i < n; ++i) {
    const rcc_adamw_tensor& t = tensors[i];
    const size_t state = t.numel * (eight ? 1 : 4), scales = (t.numel + 127) / 128 * 4;
    add(t.grad, t.numel * (t.grad_type == RCC_BF16 ? 2 : 4), false);
    add(t.param, t.numel * 4, true);
    add(t.exp_avg, state, true);
    add(t.exp_avg_sq, state, true);
    add(t.exp_avg_scale, scales, true);
    add(t.exp_avg_sq_scale, scales, true);
    add(t.copy, t.numel * 2, true);
  }
  if (written_overlap(std::move(spans)))
    return fail(bad, "a buffer that a step writes overlaps another buffer");

  // the status, the tensors and the items, as they lie in the workspace
  std::vector<char> first(kRowsAt, 0), tables(l.bytes - l.tensors_at, 0);
  auto* status = reinterpret_cast<rcc_adamw_status*>(first.data());
  status->step = step;
  status->beta1_power = std::pow(beta1, (double)step);
  status->beta2_power = std::pow(beta2, (double)step);
  status->clip_coef = 1.f;
  bool all_bf16 = true;
  for (int i = 0; i < n; ++i) all_bf16 = all_bf16 && tensors[i].grad_type == RCC_BF16;
  auto* table = reinterpret_cast<AdamWTensor*>(tables.data());
  auto* item = reinterpret_cast<AdamWItem*>(tables.data() + (l.items_at - l.tensors_at));
  for (int i = 0; i < n; ++i) {
    const rcc_adamw_tensor& t = tensors[i];
    AdamWTensor& d = table[i];
    d.grad = t.grad;
    d.param = t.param;
    d.m = t.exp_avg;
    d.v = t.exp_avg_sq;
    d.m_scales = t.exp_avg_scale;
    d.v_scales = t.exp_avg_sq_scale;
    d.copy = static_cast<__nv_bfloat16*>(t.copy);
    d.numel = t.numel;
    d.bf16 = t.grad_type == RCC_BF16;
    d.vec = vectors_of(t, eight, 16);
    d.wide = vectors_of(t, eight, 32);
    d.bulk = d.vec && on(t.exp_avg, 16) && on(t.exp_avg_sq, 16);
    const size_t chunks = (t.numel + kAdamWItem - 1) / kAdamWItem;
    for (size_t c = 0; c < chunks; ++c) *item++ = {(uint32_t)i, (uint32_t)c};
  }

  Plan p;
  p.workspace = static_cast<char*>(workspace);
  p.tensors_at = l.tensors_at;
  p.items_at = l.items_at;
  p.items = items;
  p.sms = sms;
  p.seed = seed;
  p.eight = eight;
  p.all_bf16 = all_bf16;
  cudaError_t e = cudaGetDevice(&p.device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  e = cudaStreamIsCapturing(cs, &capture);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  if (capture != cudaStreamCaptureStatusNone)
    return fail(bad, "a plan cannot be made while its stream is capturing");
  // from pageable memory: the call returns once the bytes have been taken
  e = cudaMemcpyAsync(p.workspace, first.data(), first.size(), cudaMemcpyHostToDevice, cs);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(p.workspace + l.tensors_at, tables.data(), tables.size(),
                        cudaMemcpyHostToDevice, cs);
  if (e != cudaSuccess) return cuda_fail(e, "rcc_adamw_create");
  std::lock_guard<std::mutex> lock(g_plans_mu);
  const uintptr_t id = ++g_next_plan;
  g_plans.emplace(id, p);
  *out = reinterpret_cast<rcc_adamw>(id);
  return RCC_OK;
}

bool finite_pos(double x) { return std::isfinite(x) && x > 0.0; }

}  // namespace

extern "C" {

size_t rcc_adamw_workspace(const rcc_adamw_tensor* tensors, int num_tensors) {
  const uint64_t items = count_items(tensors, num_tensors);
  return items ? layout_of(num_tensors, items, adamw_rows(adamw_sms())).bytes : 0;
}

rcc_status rcc_adamw_create(const rcc_adamw_tensor* tensors, int num_tensors, uint32_t seed,
                            int64_t step, double beta1, double beta2, void* workspace,
                            size_t workspace_bytes, rcc_stream_t stream, rcc_adamw* out) {
  rcc::NvtxRange nvtx_range("rcc_adamw_create");
  try {
    t_err.clear();
    return create(tensors, num_tensors, seed, step, beta1, beta2, workspace, workspace_bytes,
                  stream, out);
  } catch (const std::exception&) {
    return fail(RCC_ERR_INVALID_ARGUMENT, "no host memory for the plan's tables");
  }
}

rcc_status rcc_adamw_step(rcc_adamw plan, const rcc_adamw_cfg* cfg, double scale,
                          rcc_stream_t stream) {
  rcc::NvtxRange nvtx_range("rcc_adamw_step");
  t_err.clear();
  const rcc_status bad = RCC_ERR_INVALID_ARGUMENT;
  Plan p;
  {
    std::lock_guard<std::mutex> lock(g_plans_mu);
    const auto found = g_plans.find(reinterpret_cast<uintptr_t>(plan));
    if (found == g_plans.end())
      return fail(RCC_ERR_MISSING_REGISTRATION, "no such plan, or it has been destroyed");
    p = found->second;
  }
  if (!cfg) return fail(bad, "cfg is NULL");
  if (cfg->replicas != 1) return fail(bad, "replicas %d must be 1", cfg->replicas);
  if (cfg->flags) return fail(bad, "flags 0x%x must be 0", cfg->flags);
  if (!finite_pos(cfg->lr) && cfg->lr != 0.0) return fail(bad, "lr must be finite and >= 0");
  if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0 && cfg->beta2 >= 0.0 && cfg->beta2 < 1.0))
    return fail(bad, "betas must lie in [0, 1)");
  if (!(cfg->eps > 0.0) || !std::isnormal((float)cfg->eps))
    return fail(bad, "eps must be > 0 and a normal fp32 number");
  if (!std::isfinite(cfg->weight_decay) || !std::isfinite(cfg->max_grad_norm))
    return fail(bad, "weight_decay and max_grad_norm must be finite");
  if (!finite_pos(scale) || !std::isnormal((float)(1.0 / scale)))
    return fail(bad, "scale must be > 0, and 1 / scale a normal fp32 number");
  rcc_status st = check_device(p.device);
  if (st != RCC_OK) return st;
  AdamWArgs a = {};
  a.tensors = reinterpret_cast<const AdamWTensor*>(p.workspace + p.tensors_at);
  a.items = reinterpret_cast<const AdamWItem*>(p.workspace + p.items_at);
  a.rows = reinterpret_cast<AdamWRow*>(p.workspace + kRowsAt);
  a.status = reinterpret_cast<rcc_adamw_status*>(p.workspace);
  a.decision = reinterpret_cast<AdamWDecision*>(p.workspace + kDecisionAt);
  a.arrived = reinterpret_cast<uint32_t*>(p.workspace + kArrivedAt);
  a.num_items = p.items;
  a.sms = p.sms;
  a.all_bf16 = p.all_bf16;
  a.seed = p.seed;
  a.inv_scale64 = 1.0 / scale;
  a.max_norm = cfg->max_grad_norm;
  a.lr = cfg->lr;
  a.beta1 = cfg->beta1;
  a.beta2 = cfg->beta2;
  a.inv_scale = (float)(1.0 / scale);
  a.b1 = (float)cfg->beta1;
  a.one_minus_b1 = (float)(1.0 - cfg->beta1);
  a.b2 = (float)cfg->beta2;
  a.one_minus_b2 = (float)(1.0 - cfg->beta2);
  a.eps = (float)cfg->eps;
  a.decay = (float)(1.0 - cfg->lr * cfg->weight_decay);
  a.one = 1.f;
  uint64_t launches = 0;
  const cudaError_t e = launch_adamw(a, p.eight, reinterpret_cast<cudaStream_t>(stream), &launches);
  rcc::add_launches(launches);
  return e == cudaSuccess ? RCC_OK : cuda_fail(e, "rcc_adamw_step");
}

rcc_status rcc_adamw_destroy(rcc_adamw plan) {
  t_err.clear();
  std::lock_guard<std::mutex> lock(g_plans_mu);
  if (!g_plans.erase(reinterpret_cast<uintptr_t>(plan)))
    return fail(RCC_ERR_MISSING_REGISTRATION, "no such plan, or it has been destroyed");
  return RCC_OK;
}

}  // extern "C"
