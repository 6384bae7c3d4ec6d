// Host side of the operators around the root unit declared in
// include/zero_flat.h: argument checks, kernel arguments, launches.  Like the
// rest of the library it allocates no memory, and keeps nothing of a call but what
// the device answered (its SMs, a kernel's attributes and resident clusters).
#include <atomic>
#include <cmath>
#include <cstdint>
#include <limits>

#include "zero_flat.h"
#include "zero_ops.cuh"
#include "zero_status.cuh"

static_assert(zf::kMaxNormDim == ZERO_MAX_NORM_DIM, "layer norm width limit mismatch");
static_assert(zf::kMaxTeacher == ZERO_MAX_TEACHER, "teacher entry limit mismatch");

namespace zf {

cudaError_t device_sms(int* sms) {
    static std::atomic<int> known[64];          // 0: not looked up
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        const cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        known[dev].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return cudaSuccess;
}

}  // namespace zf

namespace {

using zf::cuda_call;
using zf::fail;
using zf::ok;

constexpr int64_t kMax32 = std::numeric_limits<int32_t>::max();

int check_type(int32_t bytes, const char* name) {
    if (bytes != 2 && bytes != 4)
        return fail(ZERO_ERR_INVALID_ARG, "%s = %d (2: bf16, 4: fp32)", name, bytes);
    return ZERO_OK;
}

// A device array of elements of `bytes` bytes: aligned to its element type.
int check_array(const void* p, int32_t bytes, const char* name) {
    if (p == nullptr) return fail(ZERO_ERR_INVALID_ARG, "%s is NULL", name);
    if (!zf::aligned_to(p, bytes))
        return fail(ZERO_ERR_MISALIGNED, "%s is not aligned to its element type", name);
    return ZERO_OK;
}

// Rows of `dim` elements `stride` apart, n of them.
int check_rows(const void* p, int64_t n, int64_t dim, int64_t stride, int32_t bytes,
               const char* name) {
    if (n > 0) {
        if (int rc = check_array(p, bytes, name)) return rc;
    }
    if (stride < dim)
        return fail(ZERO_ERR_SIZE, "%s: row stride %lld < %lld", name, (long long)stride,
                    (long long)dim);
    if (n > 0 && stride > std::numeric_limits<int64_t>::max() / 8 / n)
        return fail(ZERO_ERR_SIZE, "%s: size overflows int64", name);
    return ZERO_OK;
}

// An output in place of an input: where rows have different strides, one row's
// result would lie on another's input.
int check_in_place(const void* out, int64_t out_stride, const void* in, int64_t in_stride,
                   int64_t n, const char* name) {
    if (out == in && out_stride != in_stride && n > 1)
        return fail(ZERO_ERR_SIZE, "%s in place of an input needs the same row stride", name);
    return ZERO_OK;
}

// A scalar that the kernels use in fp32.
bool finite_f32(double x) { return std::isfinite(static_cast<float>(x)); }

int check_table(int64_t n_tokens, int64_t vocab, int64_t dim, double scale) {
    if (!finite_f32(scale)) return fail(ZERO_ERR_INVALID_ARG, "scale must be finite in fp32");
    if (n_tokens < 0 || vocab < 1 || dim < 1)
        return fail(ZERO_ERR_INVALID_ARG, "n_tokens >= 0, vocab >= 1 and dim >= 1 are needed");
    if (n_tokens > kMax32 || vocab > kMax32 - 1 || dim > kMax32)
        return fail(ZERO_ERR_SIZE, "n_tokens, vocab and dim must fit 32 bits");
    if (vocab > std::numeric_limits<int64_t>::max() / 8 / dim)
        return fail(ZERO_ERR_SIZE, "the table's size overflows int64");
    // the gradient's sum launch: 8 groups of 256 columns a block row
    if (dim > 8 * 256 * int64_t{65535})
        return fail(ZERO_ERR_SIZE, "dim = %lld is too large", (long long)dim);
    return ZERO_OK;
}

int check_ids(const void* ids, int32_t id_bytes, int64_t n_tokens) {
    if (id_bytes != 4 && id_bytes != 8)
        return fail(ZERO_ERR_INVALID_ARG, "id_bytes = %d (4 or 8)", id_bytes);
    return n_tokens > 0 ? check_array(ids, id_bytes, "ids") : ZERO_OK;
}

int check_workspace(const void* workspace, int64_t bytes, int64_t need) {
    if (need == 0) return ZERO_OK;
    if (workspace == nullptr) return fail(ZERO_ERR_INVALID_ARG, "workspace is NULL");
    if (!zf::aligned_to(workspace, 16))
        return fail(ZERO_ERR_MISALIGNED, "workspace is not 16-byte aligned");
    if (bytes < need)
        return fail(ZERO_ERR_SIZE, "workspace of %lld bytes: %lld are needed", (long long)bytes,
                    (long long)need);
    return ZERO_OK;
}

int64_t norm_workspace(int64_t n_rows, int64_t dim) {
    return static_cast<int64_t>(zf::norm_grad_ctas(n_rows, dim)) * 2 * dim * 4;
}

int check_norm(int64_t n_rows, int64_t dim, int32_t act_bytes, int32_t param_bytes) {
    if (n_rows < 0 || dim < 1)
        return fail(ZERO_ERR_INVALID_ARG, "n_rows >= 0 and dim >= 1 are needed");
    if (dim > ZERO_MAX_NORM_DIM)
        return fail(ZERO_ERR_SIZE, "dim = %lld exceeds %d", (long long)dim, ZERO_MAX_NORM_DIM);
    if (int rc = check_type(act_bytes, "act_bytes")) return rc;
    return check_type(param_bytes, "param_bytes");
}

int check_optional(const void* p, int32_t bytes, const char* name) {
    return p == nullptr ? ZERO_OK : check_array(p, bytes, name);
}

int distill(const void* logits, int32_t logits_bytes, int64_t n_rows, int64_t vocab,
            int64_t logits_stride, const int32_t* ids, const void* teacher, int32_t teacher_bytes,
            int64_t top, const float* weights, double temperature, float* loss, void* grad,
            int64_t grad_stride, bool with_grad, void* stream) {
    if (n_rows < 0 || vocab < 1 || top < 1)
        return fail(ZERO_ERR_INVALID_ARG, "n_rows >= 0, vocab >= 1 and top >= 1 are needed");
    if (n_rows > kMax32 || vocab > kMax32)
        return fail(ZERO_ERR_SIZE, "n_rows and vocab must fit 32 bits");
    if (top > ZERO_MAX_TEACHER)
        return fail(ZERO_ERR_SIZE, "top = %lld exceeds %d", (long long)top, ZERO_MAX_TEACHER);
    if (!(temperature > 0.0) || !std::isfinite(temperature) ||
        !finite_f32(1.4426950408889634 / temperature) || !finite_f32(temperature * temperature))
        return fail(ZERO_ERR_INVALID_ARG, "temperature must be positive and finite");
    if (int rc = check_type(logits_bytes, "logits_bytes")) return rc;
    if (int rc = check_type(teacher_bytes, "teacher_bytes")) return rc;
    if (int rc = check_rows(logits, n_rows, vocab, logits_stride, logits_bytes, "logits"))
        return rc;
    if (with_grad) {
        if (int rc = check_rows(grad, n_rows, vocab, grad_stride, logits_bytes, "grad_logits"))
            return rc;
        if (int rc = check_in_place(grad, grad_stride, logits, logits_stride, n_rows, "grad_logits"))
            return rc;
    }
    if (n_rows == 0) return ok();
    if (int rc = check_array(ids, 4, "teacher_ids")) return rc;
    if (int rc = check_array(teacher, teacher_bytes, "teacher_logits")) return rc;
    if (int rc = check_array(loss, 4, "loss")) return rc;
    if (int rc = check_optional(weights, 4, "weights")) return rc;
    zf::DistillArgs a{};
    a.logits = logits;
    a.grad = with_grad ? grad : nullptr;
    a.ids = ids;
    a.teacher = teacher;
    a.weights = weights;
    a.loss = loss;
    a.n_rows = n_rows;
    a.logits_stride = logits_stride;
    a.grad_stride = grad_stride;
    a.vocab = vocab;
    a.top = static_cast<int32_t>(top);
    a.teacher_f32 = teacher_bytes == 4;
    a.c = static_cast<float>(1.4426950408889634 / temperature);
    a.tau = static_cast<float>(temperature);
    return cuda_call(with_grad ? "distillation loss and gradient launch"
                               : "distillation loss launch",
                     [&] {
                         return zf::launch_distill(a, logits_bytes,
                                                   static_cast<cudaStream_t>(stream));
                     });
}

}  // namespace

ZERO_API int zero_embedding(const void* ids, int32_t id_bytes, int64_t n_tokens,
                            const void* weight, int32_t weight_bytes, int64_t vocab, int64_t dim,
                            double scale, void* out, int32_t out_bytes, int64_t out_stride,
                            void* stream) {
    if (int rc = check_table(n_tokens, vocab, dim, scale)) return rc;
    if (int rc = check_ids(ids, id_bytes, n_tokens)) return rc;
    if (int rc = check_type(weight_bytes, "weight_bytes")) return rc;
    if (int rc = check_type(out_bytes, "out_bytes")) return rc;
    if (int rc = check_rows(weight, vocab, dim, dim, weight_bytes, "weight")) return rc;
    if (int rc = check_rows(out, n_tokens, dim, out_stride, out_bytes, "out")) return rc;
    if (n_tokens == 0) return ok();
    zf::EmbedArgs a{};
    a.ids = ids;
    a.weight = weight;
    a.out = out;
    a.n_tokens = n_tokens;
    a.vocab = vocab;
    a.dim = dim;
    a.out_stride = out_stride;
    a.id64 = id_bytes == 8;
    a.scale = static_cast<float>(scale);
    return cuda_call("embedding launch", [&] {
        return zf::launch_embed(a, weight_bytes, out_bytes, static_cast<cudaStream_t>(stream));
    });
}

ZERO_API int zero_embedding_grad_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t dim,
                                                 int64_t* bytes) {
    if (bytes == nullptr) return fail(ZERO_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_table(n_tokens, vocab, dim, 1.0)) return rc;
    *bytes = zf::embed_grad_workspace(n_tokens, vocab, dim);
    return ok();
}

ZERO_API int zero_embedding_grad(const void* ids, int32_t id_bytes, int64_t n_tokens,
                                 const void* grad_out, int32_t grad_out_bytes,
                                 int64_t grad_out_stride, double scale, void* grad_weight,
                                 int32_t grad_weight_bytes, int64_t vocab, int64_t dim,
                                 int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
    if (int rc = check_table(n_tokens, vocab, dim, scale)) return rc;
    if (int rc = check_ids(ids, id_bytes, n_tokens)) return rc;
    if (int rc = check_type(grad_out_bytes, "grad_out_bytes")) return rc;
    if (int rc = check_type(grad_weight_bytes, "grad_weight_bytes")) return rc;
    if (int rc = check_rows(grad_out, n_tokens, dim, grad_out_stride, grad_out_bytes, "grad_out"))
        return rc;
    if (int rc = check_rows(grad_weight, vocab, dim, dim, grad_weight_bytes, "grad_weight"))
        return rc;
    if (accumulate != 0 && accumulate != 1)
        return fail(ZERO_ERR_INVALID_ARG, "accumulate = %d (0 or 1)", accumulate);
    if (int rc = check_workspace(workspace, workspace_bytes,
                                 zf::embed_grad_workspace(n_tokens, vocab, dim)))
        return rc;
    if (n_tokens == 0 && accumulate) return ok();
    zf::EmbedGradArgs a{};
    a.ids = ids;
    a.grad_out = grad_out;
    a.grad_weight = grad_weight;
    a.n_tokens = n_tokens;
    a.vocab = vocab;
    a.dim = dim;
    a.grad_stride = grad_out_stride;
    a.id64 = id_bytes == 8;
    a.accumulate = accumulate;
    a.scale = static_cast<float>(scale);
    a.workspace = workspace;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (zf::embed_grad_in_one(n_tokens, vocab, dim))
        return cuda_call("embedding gradient launch", [&] {
            return zf::launch_embed_buckets(a, grad_out_bytes, grad_weight_bytes, s);
        });
    if (int rc = cuda_call("embedding gradient sort launch",
                           [&] { return zf::launch_embed_sort(a, grad_weight_bytes, s); }))
        return rc;
    if (n_tokens == 0) return ok();
    return cuda_call("embedding gradient sum launch", [&] {
        return zf::launch_embed_sum(a, grad_out_bytes, grad_weight_bytes, s);
    });
}

ZERO_API int zero_layer_norm(const void* x, int32_t act_bytes, int64_t n_rows, int64_t dim,
                             int64_t x_stride, const void* weight, const void* bias,
                             int32_t param_bytes, double eps, void* out, int64_t out_stride,
                             float* mean, float* rstd, void* stream) {
    if (int rc = check_norm(n_rows, dim, act_bytes, param_bytes)) return rc;
    if (!(eps >= 0.0) || !finite_f32(eps))
        return fail(ZERO_ERR_INVALID_ARG, "eps must be >= 0 and finite in fp32");
    if (int rc = check_rows(x, n_rows, dim, x_stride, act_bytes, "x")) return rc;
    if (int rc = check_rows(out, n_rows, dim, out_stride, act_bytes, "out")) return rc;
    if (int rc = check_in_place(out, out_stride, x, x_stride, n_rows, "out")) return rc;
    if (int rc = check_optional(weight, param_bytes, "weight")) return rc;
    if (int rc = check_optional(bias, param_bytes, "bias")) return rc;
    if (int rc = check_optional(mean, 4, "mean")) return rc;
    if (int rc = check_optional(rstd, 4, "rstd")) return rc;
    if (n_rows == 0) return ok();
    zf::NormArgs a{};
    a.x = x;
    a.out = out;
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    a.n_rows = n_rows;
    a.x_stride = x_stride;
    a.out_stride = out_stride;
    a.dim = static_cast<int32_t>(dim);
    a.param_f32 = param_bytes == 4;
    a.eps = static_cast<float>(eps);
    return cuda_call("layer norm launch", [&] {
        return zf::launch_norm(a, act_bytes, static_cast<cudaStream_t>(stream));
    });
}

ZERO_API int zero_layer_norm_grad_workspace_bytes(int64_t n_rows, int64_t dim, int64_t* bytes) {
    if (bytes == nullptr) return fail(ZERO_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_norm(n_rows, dim, 2, 2)) return rc;
    *bytes = norm_workspace(n_rows, dim);
    return ok();
}

ZERO_API int zero_layer_norm_grad(const void* grad_out, const void* x, int32_t act_bytes,
                                  int64_t n_rows, int64_t dim, int64_t grad_out_stride,
                                  int64_t x_stride, const void* weight, int32_t param_bytes,
                                  const float* mean, const float* rstd, void* grad_x,
                                  int64_t grad_x_stride, void* grad_weight, void* grad_bias,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    if (int rc = check_norm(n_rows, dim, act_bytes, param_bytes)) return rc;
    if (int rc = check_rows(grad_out, n_rows, dim, grad_out_stride, act_bytes, "grad_out"))
        return rc;
    if (int rc = check_rows(x, n_rows, dim, x_stride, act_bytes, "x")) return rc;
    if (int rc = check_rows(grad_x, n_rows, dim, grad_x_stride, act_bytes, "grad_x")) return rc;
    if (int rc = check_in_place(grad_x, grad_x_stride, grad_out, grad_out_stride, n_rows, "grad_x"))
        return rc;
    if (int rc = check_in_place(grad_x, grad_x_stride, x, x_stride, n_rows, "grad_x")) return rc;
    if (int rc = check_optional(weight, param_bytes, "weight")) return rc;
    if (int rc = check_optional(grad_weight, param_bytes, "grad_weight")) return rc;
    if (int rc = check_optional(grad_bias, param_bytes, "grad_bias")) return rc;
    if (n_rows > 0) {
        if (int rc = check_array(mean, 4, "mean")) return rc;
        if (int rc = check_array(rstd, 4, "rstd")) return rc;
    }
    if (int rc = check_workspace(workspace, workspace_bytes, norm_workspace(n_rows, dim)))
        return rc;
    const bool params = grad_weight != nullptr || grad_bias != nullptr;
    if (n_rows == 0 && !params) return ok();
    zf::NormArgs a{};
    a.x = x;
    a.grad_out = grad_out;
    a.out = grad_x;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.grad_weight = grad_weight;
    a.grad_bias = grad_bias;
    a.partials = static_cast<float*>(workspace);
    a.n_rows = n_rows;
    a.x_stride = x_stride;
    a.grad_out_stride = grad_out_stride;
    a.out_stride = grad_x_stride;
    a.dim = static_cast<int32_t>(dim);
    a.param_f32 = param_bytes == 4;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = cuda_call("layer norm gradient launch",
                           [&] { return zf::launch_norm_grad(a, act_bytes, s); }))
        return rc;
    if (!params) return ok();
    return cuda_call("layer norm gradient reduction launch",
                     [&] { return zf::launch_norm_grad_reduce(a, act_bytes, s); });
}

ZERO_API int zero_distill_loss(const void* logits, int32_t logits_bytes, int64_t n_rows,
                               int64_t vocab, int64_t logits_stride, const int32_t* teacher_ids,
                               const void* teacher_logits, int32_t teacher_bytes, int64_t top,
                               const float* weights, double temperature, float* loss,
                               void* stream) {
    return distill(logits, logits_bytes, n_rows, vocab, logits_stride, teacher_ids, teacher_logits,
                   teacher_bytes, top, weights, temperature, loss, nullptr, 0, false, stream);
}

ZERO_API int zero_distill_loss_grad(const void* logits, int32_t logits_bytes, int64_t n_rows,
                                    int64_t vocab, int64_t logits_stride,
                                    const int32_t* teacher_ids, const void* teacher_logits,
                                    int32_t teacher_bytes, int64_t top, const float* weights,
                                    double temperature, float* loss, void* grad_logits,
                                    int64_t grad_logits_stride, void* stream) {
    return distill(logits, logits_bytes, n_rows, vocab, logits_stride, teacher_ids, teacher_logits,
                   teacher_bytes, top, weights, temperature, loss, grad_logits, grad_logits_stride,
                   true, stream);
}
