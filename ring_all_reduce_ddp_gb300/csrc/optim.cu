// The C ABI (include/ddp_ring.h): the operators between a gradient sync and
// the next forward (ddp_optim_*). A handle holds one gradient set's tile
// tables and workspace in device memory, planned once.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <exception>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "host.h"
#include "optim.cuh"

using namespace ddp;
using namespace ddp::host;

struct ddp_optim {
  int32_t k = 0;
  ddp_dtype dt = DDP_FLOAT32;
  std::vector<const void*> grads;
  std::vector<int64_t> numel;
  struct Table {
    void* mem = nullptr;
    OptimTable t{};
  };
  Table norm, clip, update;  // tiles cut at the gradients', the outputs' and the state's 8-element boundaries
  void* work_mem = nullptr;
  OptimWork work{};
  ddp_dtype param_dt = DDP_FLOAT32;
  bool has_master = false;
  int64_t* step = nullptr;
};

namespace {

constexpr int64_t kMaxNumel = int64_t(1) << 48;  // byte counts and tile arithmetic stay far inside 64 bits

using Ranges = std::vector<std::pair<uintptr_t, uintptr_t>>;

int phase(const void* ptr, int es, int vec = kOptimVec) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(ptr) / es % vec);
}

ddp_status check_tensor(const void* ptr, int es, const char* what, int64_t i) {
  DDP_CHECK(ptr != nullptr, DDP_ERR_ARG, std::string(what) + "[" + std::to_string(i) + "] is null");
  DDP_CHECK(reinterpret_cast<uintptr_t>(ptr) % es == 0, DDP_ERR_ALIGN,
            std::string(what) + "[" + std::to_string(i) + "] is not aligned to its element size");
  return DDP_OK;
}

// Add [count] tensors of numel elements each (cycling over the k sizes) to r,
// checked; tensors of no elements are skipped, their pointers may be null.
ddp_status add_ranges(Ranges& r, const void* const* v, int64_t count, const std::vector<int64_t>& numel, int es,
                      const char* what) {
  DDP_CHECK(v != nullptr, DDP_ERR_ARG, std::string(what) + " array is null");
  const int64_t k = static_cast<int64_t>(numel.size());
  for (int64_t i = 0; i < count; ++i) {
    if (numel[i % k] == 0) continue;
    DDP_TRY(check_tensor(v[i], es, what, i));
    r.push_back(range_of(v[i], numel[i % k] * es));
  }
  return DDP_OK;
}

// The tensors' records, their tiles of `elems` elements as a prefix, and the p
// outputs of each, in one device allocation. recs[j].f gives tensor j's tile boundaries.
ddp_status build_table(const std::vector<OptimTensor>& recs, int elems, const void* const* outs, int32_t p,
                       ddp_optim::Table* out) {
  const size_t k = recs.size();
  std::vector<int32_t> tile0{0};
  for (const OptimTensor& t : recs) {
    const int64_t c = t.n > 0 ? (t.n + t.f + elems - 1) / elems : 0;
    DDP_CHECK(tile0.back() + c <= 0x7FFFFFFF, DDP_ERR_ARG, "gradient set too large for one launch");
    tile0.push_back(static_cast<int32_t>(tile0.back() + c));
  }
  std::vector<void*> ptrs(k * p);  // tensor-major: one tensor's p outputs together
  for (int32_t r = 0; r < p; ++r)
    for (size_t j = 0; j < k; ++j) ptrs[j * p + r] = const_cast<void*>(outs[r * k + j]);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t o_outs = up(k * sizeof(OptimTensor)), o_tile0 = o_outs + up(ptrs.size() * sizeof(void*)),
               total = o_tile0 + up((k + 1) * sizeof(int32_t));
  std::vector<unsigned char> host(total, 0);
  std::memcpy(host.data(), recs.data(), k * sizeof(OptimTensor));
  if (!ptrs.empty()) std::memcpy(host.data() + o_outs, ptrs.data(), ptrs.size() * sizeof(void*));
  std::memcpy(host.data() + o_tile0, tile0.data(), (k + 1) * sizeof(int32_t));
  void* mem = nullptr;
  DDP_TRY(alloc_device(&mem, total, "optim tile table"));
  const ddp_status st = upload(mem, host.data(), total, "optim tile table upload");
  if (st != DDP_OK) {
    (void)cudaFree(mem);
    return st;
  }
  unsigned char* d = static_cast<unsigned char*>(mem);
  out->mem = mem;
  out->t.tensors = reinterpret_cast<const OptimTensor*>(d);
  out->t.outs = reinterpret_cast<void* const*>(d + o_outs);
  out->t.ntiles = tile0.back();
  out->t.p = p;
  out->t.k = static_cast<int32_t>(k);
  out->t.tile0 = reinterpret_cast<const int32_t*>(d + o_tile0);
  return DDP_OK;
}

// Put a new table in the place of an old one that launches in flight may read.
ddp_status replace_table(ddp_optim::Table* old, const ddp_optim::Table& now) {
  void* gone = old->mem;
  *old = now;
  if (gone) {
    DDP_CUDA(cudaDeviceSynchronize(), "synchronize before releasing the previous tile table");
    DDP_CUDA(cudaFree(gone), "release of the previous tile table");
  }
  return DDP_OK;
}

cudaError_t optim_free_device(ddp_optim* h) {
  cudaError_t first = cudaSuccess;
  for (void* m : {h->norm.mem, h->clip.mem, h->update.mem, h->work_mem}) {
    const cudaError_t e = m ? cudaFree(m) : cudaSuccess;
    if (first == cudaSuccess) first = e;
  }
  return first;
}

ddp_status create_impl(ddp_optim* h, int32_t k, const void* const* grads, const int64_t* numel, ddp_dtype dtype) {
  const int es = esize(dtype);
  h->k = k;
  h->dt = dtype;
  for (int32_t j = 0; j < k; ++j)
    DDP_CHECK(numel[j] >= 0 && numel[j] <= kMaxNumel, DDP_ERR_ARG, "numel must be in [0, 2^48]");
  h->numel.assign(numel, numel + k);
  h->grads.assign(grads, grads + k);
  Ranges r;
  DDP_TRY(add_ranges(r, grads, k, h->numel, es, "grads"));
  DDP_CHECK(disjoint(r), DDP_ERR_ARG, "gradient tensors overlap");
  std::vector<OptimTensor> recs(k);
  for (int32_t j = 0; j < k; ++j) {
    recs[j] = OptimTensor{};
    recs[j].grad = grads[j];
    recs[j].n = numel[j];
    recs[j].f = phase(grads[j], es, 32 / es);
    recs[j].aligned = recs[j].grad_aligned = 1;
  }
  DDP_TRY(build_table(recs, kNormTileBytes / es, nullptr, 0, &h->norm));
  h->work.norm_blocks = optim_norm_blocks(h->norm.t.ntiles);
  const size_t blocks = h->work.norm_blocks, head = 256 + kScalarCopies * sizeof(StepScalars),
               bytes = head + (2 * blocks + k) * sizeof(double);
  DDP_TRY(alloc_device(&h->work_mem, bytes, "optim workspace"));
  DDP_CUDA(cudaMemset(h->work_mem, 0, bytes), "optim workspace");
  DDP_CUDA(cudaDeviceSynchronize(), "optim workspace");
  unsigned char* d = static_cast<unsigned char*>(h->work_mem);
  h->work.ticket = reinterpret_cast<unsigned int*>(d);
  h->work.scalars = reinterpret_cast<StepScalars*>(d + 256);
  h->work.block_sum = reinterpret_cast<double*>(d + head);
  h->work.part_sum = h->work.block_sum + blocks;
  return DDP_OK;
}

ddp_status set_outputs_impl(ddp_optim* h, int32_t p, void* const* outs) {
  const int es = esize(h->dt), vec = 32 / es;
  const int64_t k = h->k;
  Ranges all, apart;
  DDP_TRY(add_ranges(all, outs, p * k, h->numel, es, "outs"));
  DDP_CHECK(disjoint(all), DDP_ERR_ARG, "outputs overlap");
  for (int64_t i = 0; i < p * k; ++i)  // an output may be its own gradient, and overlap no other
    if (h->numel[i % k] > 0 && outs[i] != h->grads[i % k]) apart.push_back(range_of(outs[i], h->numel[i % k] * es));
  for (int64_t j = 0; j < k; ++j)
    if (h->numel[j] > 0) apart.push_back(range_of(h->grads[j], h->numel[j] * es));
  DDP_CHECK(disjoint(apart), DDP_ERR_ARG, "an output overlaps a gradient and is not the same tensor");
  std::vector<OptimTensor> recs(k);
  for (int64_t j = 0; j < k; ++j) {
    OptimTensor& t = recs[j] = OptimTensor{};
    t.grad = h->grads[j];
    t.n = h->numel[j];
    t.f = phase(outs[j], es, vec);
    t.grad_aligned = phase(t.grad, es, vec) == t.f;
    t.aligned = 1;
    for (int32_t r = 1; r < p; ++r) t.aligned &= phase(outs[r * k + j], es, vec) == t.f;
  }
  ddp_optim::Table now;
  DDP_TRY(build_table(recs, scale_tile_bytes(p) / es, outs, p, &now));
  return replace_table(&h->clip, now);
}

ddp_status set_params_impl(ddp_optim* h, int32_t p, void* const* params, ddp_dtype param_dtype, float* const* master,
                           float* const* exp_avg, float* const* exp_avg_sq, int64_t* step) {
  const int ps = esize(param_dtype);
  const int64_t k = h->k;
  auto any = [](float* const* v) { return reinterpret_cast<const void* const*>(v); };
  Ranges all;
  DDP_TRY(add_ranges(all, params, p * k, h->numel, ps, "params"));
  if (master) DDP_TRY(add_ranges(all, any(master), k, h->numel, 4, "master"));
  DDP_TRY(add_ranges(all, any(exp_avg), k, h->numel, 4, "exp_avg"));
  DDP_TRY(add_ranges(all, any(exp_avg_sq), k, h->numel, 4, "exp_avg_sq"));
  DDP_TRY(add_ranges(all, h->grads.data(), k, h->numel, esize(h->dt), "grads"));
  all.push_back(range_of(step, sizeof(int64_t)));
  DDP_CHECK(disjoint(all), DDP_ERR_ARG, "parameters, state, step and gradients overlap");
  std::vector<OptimTensor> recs(k);
  for (int64_t j = 0; j < k; ++j) {
    OptimTensor& t = recs[j] = OptimTensor{};
    t.grad = h->grads[j];
    t.m = exp_avg[j];
    t.v = exp_avg_sq[j];
    t.master = master ? master[j] : nullptr;
    t.n = h->numel[j];
    t.f = phase(t.m, 4);
    t.grad_aligned = phase(t.grad, esize(h->dt)) == t.f;
    t.aligned = phase(t.v, 4) == t.f && (!master || phase(t.master, 4) == t.f);
    for (int32_t r = 0; r < p; ++r) t.aligned &= phase(params[r * k + j], ps) == t.f;
  }
  ddp_optim::Table now;
  DDP_TRY(build_table(recs, kOptimTile, params, p, &now));
  h->param_dt = param_dtype;
  h->has_master = master != nullptr;
  h->step = step;
  return replace_table(&h->update, now);
}

// The planners allocate host memory: no exception leaves a C entry point.
template <typename F>
ddp_status no_throw(F&& f) {
  try {
    return f();
  } catch (const std::exception&) {  // bad_alloc, length_error
    return fail(DDP_ERR_NOMEM, "host memory for the tile table");
  }
}

ddp_status check_scalar(const void* ptr, size_t align, const char* what) {
  DDP_CHECK(ptr != nullptr, DDP_ERR_ARG, std::string(what) + " is null");
  DDP_CHECK(reinterpret_cast<uintptr_t>(ptr) % align == 0, DDP_ERR_ALIGN, std::string(what) + " is not aligned");
  return DDP_OK;
}

ddp_status check_kind(ddp_norm kind) {
  DDP_CHECK(kind == DDP_NORM_L2 || kind == DDP_NORM_INF, DDP_ERR_ARG, "unknown norm");
  return DDP_OK;
}

ddp_status check_max_norm(float max_norm) {
  DDP_CHECK(max_norm > 0.0f, DDP_ERR_ARG, "max_norm must be positive");
  return DDP_OK;
}

}  // namespace

extern "C" {

ddp_status ddp_optim_create(ddp_optim** handle, int32_t k, const void* const* grads, const int64_t* numel,
                            ddp_dtype dtype) {
  DDP_CHECK(handle != nullptr, DDP_ERR_ARG, "handle pointer is null");
  *handle = nullptr;
  DDP_TRY(check_common(1, 0, dtype));
  DDP_CHECK(k >= 1 && numel && grads, DDP_ERR_ARG, "need k >= 1 tensors, numel and grads");
  ddp_optim* h = new (std::nothrow) ddp_optim();
  DDP_CHECK(h != nullptr, DDP_ERR_NOMEM, "host memory for the handle");
  const ddp_status st = no_throw([&] { return create_impl(h, k, grads, numel, dtype); });
  if (st != DDP_OK) {
    (void)optim_free_device(h);
    delete h;
    return st;
  }
  *handle = h;
  return DDP_OK;
}

ddp_status ddp_optim_destroy(ddp_optim* h) {
  if (!h) return DDP_OK;
  const cudaError_t e = optim_free_device(h);
  delete h;
  if (e != cudaSuccess) return cuda_fail(e, "optim release");
  return DDP_OK;
}

ddp_status ddp_optim_norm(ddp_optim* h, ddp_norm kind, float* norm, float* each, cudaStream_t stream) {
  DDP_NVTX("ddp_optim_norm");
  DDP_CHECK(h != nullptr, DDP_ERR_ARG, "handle is null");
  DDP_TRY(check_kind(kind));
  DDP_TRY(check_scalar(norm, sizeof(float), "norm"));
  if (each) DDP_TRY(check_scalar(each, sizeof(float), "each"));
  DDP_CUDA(launch_optim_norm(h->norm.t, h->work, h->dt, kind, norm, each, stream), "norm launch");
  return DDP_OK;
}

ddp_status ddp_optim_set_outputs(ddp_optim* h, int32_t p, void* const* outs) {
  DDP_CHECK(h != nullptr, DDP_ERR_ARG, "handle is null");
  DDP_TRY(check_common(p, 0, h->dt));
  DDP_CHECK(outs != nullptr, DDP_ERR_ARG, "outs array is null");
  return no_throw([&] { return set_outputs_impl(h, p, outs); });
}

ddp_status ddp_optim_clip(ddp_optim* h, ddp_norm kind, float max_norm, float* norm, cudaStream_t stream) {
  DDP_NVTX("ddp_optim_clip");
  DDP_CHECK(h != nullptr, DDP_ERR_ARG, "handle is null");
  DDP_TRY(check_kind(kind));
  DDP_TRY(check_max_norm(max_norm));
  DDP_TRY(check_scalar(norm, sizeof(float), "norm"));
  DDP_CHECK(h->clip.mem != nullptr, DDP_ERR_STATE, "no outputs: call ddp_optim_set_outputs first");
  DDP_CUDA(launch_optim_norm(h->norm.t, h->work, h->dt, kind, norm, nullptr, stream), "norm launch");
  DDP_CUDA(launch_optim_scale(h->clip.t, h->dt, norm, max_norm, stream), "clip launch");
  return DDP_OK;
}

ddp_status ddp_optim_set_params(ddp_optim* h, int32_t p, void* const* params, ddp_dtype param_dtype,
                                float* const* master, float* const* exp_avg, float* const* exp_avg_sq, int64_t* step) {
  DDP_CHECK(h != nullptr, DDP_ERR_ARG, "handle is null");
  DDP_TRY(check_common(p, 0, param_dtype));
  DDP_CHECK(params && exp_avg && exp_avg_sq, DDP_ERR_ARG, "params, exp_avg or exp_avg_sq array is null");
  DDP_CHECK(!(master && param_dtype == DDP_FLOAT32), DDP_ERR_DTYPE,
            "fp32 parameters take no master copy: they are the master");
  DDP_TRY(check_scalar(step, sizeof(int64_t), "step"));
  return no_throw([&] { return set_params_impl(h, p, params, param_dtype, master, exp_avg, exp_avg_sq, step); });
}

ddp_status ddp_optim_adamw(ddp_optim* h, double lr, double beta1, double beta2, double eps, double weight_decay,
                           const float* norm, float max_norm, cudaStream_t stream) {
  DDP_NVTX("ddp_optim_adamw");
  DDP_CHECK(h != nullptr, DDP_ERR_ARG, "handle is null");
  DDP_CHECK(std::isfinite(lr) && lr >= 0.0, DDP_ERR_ARG, "lr must be finite and >= 0");
  DDP_CHECK(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0, DDP_ERR_ARG, "betas must be in [0, 1)");
  DDP_CHECK(std::isfinite(eps) && eps >= 0.0, DDP_ERR_ARG, "eps must be finite and >= 0");
  DDP_CHECK(std::isfinite(weight_decay) && weight_decay >= 0.0, DDP_ERR_ARG, "weight_decay must be finite and >= 0");
  if (norm) {
    DDP_TRY(check_max_norm(max_norm));
    DDP_TRY(check_scalar(norm, sizeof(float), "norm"));
  }
  DDP_CHECK(h->update.mem != nullptr, DDP_ERR_STATE, "no parameters: call ddp_optim_set_params first");
  AdamwArgs a;
  a.lr = static_cast<float>(lr);
  a.log_beta1 = std::log(beta1);
  a.log_beta2 = std::log(beta2);
  a.beta2 = static_cast<float>(beta2);
  a.one_minus_beta1 = static_cast<float>(1.0 - beta1);
  a.one_minus_beta2 = static_cast<float>(1.0 - beta2);
  a.eps = static_cast<float>(eps);
  a.decay = static_cast<float>(lr * weight_decay);
  a.max_norm = max_norm;
  a.norm = norm;
  a.step = h->step;
  DDP_CUDA(launch_optim_adamw(h->update.t, h->work, h->dt, h->param_dt, h->has_master, a, stream), "AdamW launch");
  return DDP_OK;
}

}  // extern "C"
