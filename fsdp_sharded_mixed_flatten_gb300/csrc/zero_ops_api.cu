// Host side of the operators around the root unit declared in
// include/zero_flat.h: argument checks, kernel arguments, launches.  Like the
// rest of the library it allocates no memory, and keeps nothing of a call but what
// the device answered (its SMs, a kernel's attributes and resident clusters).
#include <atomic>
#include <cmath>
#include <cstdint>
#include <limits>

#include "zero_flat.h"
#include "zero_head.cuh"
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

namespace {

constexpr int64_t kBlock = 128;             // columns of a scale

int check_eight(const void* codes, const void* scales, int64_t n, int64_t dim, int64_t stride,
                const char* name) {
    if (int rc = check_rows(codes, n, dim, stride, 1, name)) return rc;
    if (n > 0) {
        if (scales == nullptr) return fail(ZERO_ERR_INVALID_ARG, "%s: its scales are NULL", name);
        if (!zf::aligned_to(scales, 4))
            return fail(ZERO_ERR_MISALIGNED, "%s: its scales are not aligned", name);
    }
    return ZERO_OK;
}

// An optional matrix: nothing, or rows.
int check_maybe_rows(const void* p, int64_t n, int64_t dim, int64_t stride, int32_t bytes,
                     const char* name) {
    return p == nullptr ? ZERO_OK : check_rows(p, n, dim, stride, bytes, name);
}

int eight(const void* x, void* out, int32_t bytes, int64_t n_rows, int64_t dim, int64_t stride,
          uint8_t* codes, int64_t codes_stride, float* scales, void* stream) {
    const bool pack = out == nullptr;
    if (n_rows < 0 || dim < 1)
        return fail(ZERO_ERR_INVALID_ARG, "n_rows >= 0 and dim >= 1 are needed");
    // as many CTAs as a launch takes, of eight warps that take 512 columns at least
    if (n_rows > kMax32 || dim > kMax32 - 1024 || n_rows * ((dim + 511) / 512) > kMax32)
        return fail(ZERO_ERR_SIZE, "n_rows * ceil(dim / 512) must fit 32 bits");
    if (int rc = check_type(bytes, pack ? "x_bytes" : "out_bytes")) return rc;
    if (int rc = check_rows(pack ? x : out, n_rows, dim, stride, bytes, pack ? "x" : "out"))
        return rc;
    if (int rc = check_eight(codes, scales, n_rows, dim, codes_stride, "codes")) return rc;
    if (n_rows == 0) return ok();
    zf::EightArgs a{};
    a.x = x;
    a.out = out;
    a.codes = codes;
    a.scales = scales;
    a.n_rows = n_rows;
    a.dim = dim;
    a.blocks = (dim + kBlock - 1) / kBlock;
    a.x_stride = stride;
    a.codes_stride = codes_stride;
    return cuda_call(pack ? "row packing launch" : "row unpacking launch", [&] {
        return zf::launch_eight(a, bytes, static_cast<cudaStream_t>(stream));
    });
}

}  // namespace

ZERO_API int zero_pack_rows(const void* x, int32_t x_bytes, int64_t n_rows, int64_t dim,
                            int64_t x_stride, uint8_t* codes, int64_t codes_stride, float* scales,
                            void* stream) {
    return eight(x, nullptr, x_bytes, n_rows, dim, x_stride, codes, codes_stride, scales, stream);
}

ZERO_API int zero_unpack_rows(const uint8_t* codes, int64_t codes_stride, const float* scales,
                              int64_t n_rows, int64_t dim, void* out, int32_t out_bytes,
                              int64_t out_stride, void* stream) {
    if (out == nullptr && n_rows > 0) return fail(ZERO_ERR_INVALID_ARG, "out is NULL");
    return eight(nullptr, out, out_bytes, n_rows, dim, out_stride, const_cast<uint8_t*>(codes),
                 codes_stride, const_cast<float*>(scales), stream);
}

ZERO_API int zero_rms_norm(const void* x, const void* residual, int32_t act_bytes, int64_t n_rows,
                           int64_t dim, int64_t x_stride, int64_t residual_stride,
                           const void* weight, int32_t param_bytes, double eps, void* out,
                           int64_t out_stride, void* total, int64_t total_stride, uint8_t* out8,
                           int64_t out8_stride, float* out8_scales, uint8_t* total8,
                           int64_t total8_stride, float* total8_scales, float* rstd,
                           void* stream) {
    if (int rc = check_norm(n_rows, dim, act_bytes, param_bytes)) return rc;
    if (!(eps >= 0.0) || !finite_f32(eps))
        return fail(ZERO_ERR_INVALID_ARG, "eps must be >= 0 and finite in fp32");
    if (int rc = check_rows(x, n_rows, dim, x_stride, act_bytes, "x")) return rc;
    if (int rc = check_maybe_rows(residual, n_rows, dim, residual_stride, act_bytes, "residual"))
        return rc;
    if (int rc = check_maybe_rows(out, n_rows, dim, out_stride, act_bytes, "out")) return rc;
    if (int rc = check_maybe_rows(total, n_rows, dim, total_stride, act_bytes, "total")) return rc;
    if (out8 != nullptr || out8_scales != nullptr) {
        if (int rc = check_eight(out8, out8_scales, n_rows, dim, out8_stride, "out8")) return rc;
    }
    if (total8 != nullptr || total8_scales != nullptr) {
        if (int rc = check_eight(total8, total8_scales, n_rows, dim, total8_stride, "total8"))
            return rc;
    }
    if (n_rows > 0 && total != nullptr && total == out)
        return fail(ZERO_ERR_INVALID_ARG, "total and out are the same array");
    if (out != nullptr && out == residual && n_rows > 0)
        return fail(ZERO_ERR_INVALID_ARG, "out and residual are the same array");
    if (total != nullptr) {
        if (int rc = check_in_place(total, total_stride, x, x_stride, n_rows, "total")) return rc;
        if (int rc = check_in_place(total, total_stride, residual, residual_stride, n_rows,
                                    "total"))
            return rc;
    }
    if (out != nullptr) {
        if (int rc = check_in_place(out, out_stride, x, x_stride, n_rows, "out")) return rc;
    }
    if (int rc = check_optional(weight, param_bytes, "weight")) return rc;
    if (int rc = check_optional(rstd, 4, "rstd")) return rc;
    if (n_rows == 0) return ok();
    zf::RmsArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.total = total;
    a.out = out;
    a.out8 = out8;
    a.out8_scales = out8_scales;
    a.total8 = total8;
    a.total8_scales = total8_scales;
    a.rstd = rstd;
    a.n_rows = n_rows;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.total_stride = total_stride;
    a.out_stride = out_stride;
    a.out8_stride = out8_stride;
    a.total8_stride = total8_stride;
    a.dim = static_cast<int32_t>(dim);
    a.blocks = static_cast<int32_t>((dim + kBlock - 1) / kBlock);
    a.param_f32 = param_bytes == 4;
    a.eps = static_cast<float>(eps);
    return cuda_call("rms norm launch", [&] {
        return zf::launch_rms_norm(a, act_bytes, static_cast<cudaStream_t>(stream));
    });
}

ZERO_API int zero_rms_norm_grad_workspace_bytes(int64_t n_rows, int64_t dim, int64_t* bytes) {
    if (bytes == nullptr) return fail(ZERO_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_norm(n_rows, dim, 2, 2)) return rc;
    *bytes = static_cast<int64_t>(zf::rms_grad_ctas(n_rows)) * dim * 4;
    return ok();
}

ZERO_API int zero_rms_norm_grad(const void* grad_out, const void* total, const uint8_t* total8,
                                int64_t total8_stride, const float* total8_scales,
                                int32_t act_bytes, int64_t n_rows, int64_t dim,
                                int64_t grad_out_stride, int64_t total_stride, const void* weight,
                                int32_t param_bytes, const float* rstd, const void* grad_total,
                                int64_t grad_total_stride, void* grad_x, int64_t grad_x_stride,
                                void* grad_weight, void* out, int64_t out_stride, void* workspace,
                                int64_t workspace_bytes, void* stream) {
    if (int rc = check_norm(n_rows, dim, act_bytes, param_bytes)) return rc;
    if (int rc = check_rows(grad_out, n_rows, dim, grad_out_stride, act_bytes, "grad_out"))
        return rc;
    if (total != nullptr) {
        if (total8 != nullptr || total8_scales != nullptr)
            return fail(ZERO_ERR_INVALID_ARG, "total and total8: one of the two is needed");
        if (int rc = check_rows(total, n_rows, dim, total_stride, act_bytes, "total")) return rc;
    } else if (n_rows > 0) {
        if (total8 == nullptr) return fail(ZERO_ERR_INVALID_ARG, "total and total8 are NULL");
        if (int rc = check_eight(total8, total8_scales, n_rows, dim, total8_stride, "total8"))
            return rc;
    }
    if (int rc = check_maybe_rows(grad_total, n_rows, dim, grad_total_stride, act_bytes,
                                  "grad_total"))
        return rc;
    if (int rc = check_rows(grad_x, n_rows, dim, grad_x_stride, act_bytes, "grad_x")) return rc;
    if (int rc = check_maybe_rows(out, n_rows, dim, out_stride, act_bytes, "out")) return rc;
    if (int rc = check_in_place(grad_x, grad_x_stride, grad_out, grad_out_stride, n_rows, "grad_x"))
        return rc;
    if (int rc = check_in_place(grad_x, grad_x_stride, total, total_stride, n_rows, "grad_x"))
        return rc;
    if (int rc = check_in_place(grad_x, grad_x_stride, grad_total, grad_total_stride, n_rows,
                                "grad_x"))
        return rc;
    if (n_rows > 0 && out != nullptr && (out == grad_x || out == grad_out || out == grad_total ||
                                         out == total))
        return fail(ZERO_ERR_INVALID_ARG, "out is another array of the call");
    if (int rc = check_optional(weight, param_bytes, "weight")) return rc;
    if (int rc = check_optional(grad_weight, param_bytes, "grad_weight")) return rc;
    if (n_rows > 0) {
        if (int rc = check_array(rstd, 4, "rstd")) return rc;
    }
    if (int rc = check_workspace(
            workspace, workspace_bytes,
            grad_weight == nullptr ? 0
                                   : static_cast<int64_t>(zf::rms_grad_ctas(n_rows)) * dim * 4))
        return rc;
    if (n_rows == 0 && grad_weight == nullptr) return ok();
    zf::RmsArgs a{};
    a.x = total;
    a.grad_out = grad_out;
    a.grad_total = grad_total;
    a.weight = weight;
    a.out = out;
    a.grad_x = grad_x;
    a.grad_weight = grad_weight;
    a.total8 = const_cast<uint8_t*>(total8);
    a.total8_scales = const_cast<float*>(total8_scales);
    a.rstd = const_cast<float*>(rstd);
    a.partials = static_cast<float*>(workspace);
    a.n_rows = n_rows;
    a.x_stride = total_stride;
    a.grad_out_stride = grad_out_stride;
    a.grad_total_stride = grad_total_stride;
    a.out_stride = out_stride;
    a.grad_x_stride = grad_x_stride;
    a.total8_stride = total8_stride;
    a.dim = static_cast<int32_t>(dim);
    a.blocks = static_cast<int32_t>((dim + kBlock - 1) / kBlock);
    a.param_f32 = param_bytes == 4;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = cuda_call("rms norm gradient launch",
                           [&] { return zf::launch_rms_norm_grad(a, act_bytes, s); }))
        return rc;
    if (grad_weight == nullptr) return ok();
    return cuda_call("rms norm gradient reduction launch",
                     [&] { return zf::launch_rms_reduce(a, act_bytes, s); });
}

namespace {

int check_head(int64_t n_tokens, int64_t vocab, int64_t dim) {
    if (n_tokens < 0 || vocab < 1 || dim < 1)
        return fail(ZERO_ERR_INVALID_ARG, "n_tokens >= 0, vocab >= 1 and dim >= 1 are needed");
    if (n_tokens > ZERO_MAX_HEAD_TOKENS || vocab > ZERO_MAX_HEAD_VOCAB || dim > ZERO_MAX_HEAD_DIM)
        return fail(ZERO_ERR_SIZE, "n_tokens, vocab or dim is too large (at most %d, %d, %d)",
                    ZERO_MAX_HEAD_TOKENS, ZERO_MAX_HEAD_VOCAB, ZERO_MAX_HEAD_DIM);
    return ZERO_OK;
}

// What both passes read.
int head_call(zf::HeadCall& c, const uint16_t* hidden, int64_t n_tokens, int64_t dim,
              int64_t hidden_stride, const uint16_t* table, int64_t vocab, const void* labels,
              int32_t label_bytes) {
    if (int rc = check_head(n_tokens, vocab, dim)) return rc;
    if (int rc = check_rows(hidden, n_tokens, dim, hidden_stride, 2, "hidden")) return rc;
    if (int rc = check_array(table, 2, "table")) return rc;
    if (label_bytes != 4 && label_bytes != 8)
        return fail(ZERO_ERR_INVALID_ARG, "label_bytes = %d (4 or 8)", label_bytes);
    if (n_tokens > 0) {
        if (int rc = check_array(labels, label_bytes, "labels")) return rc;
    }
    c.hidden = hidden;
    c.table = table;
    c.labels = labels;
    c.n_tokens = n_tokens;
    c.vocab = vocab;
    c.dim = dim;
    c.hidden_stride = hidden_stride;
    c.label64 = label_bytes == 8;
    return ZERO_OK;
}

// Wherever the table lies, or of one that is read in place.
int head_workspace(int64_t n_tokens, int64_t vocab, int64_t dim, bool back, bool in_place,
                   int64_t* bytes) {
    if (bytes == nullptr) return fail(ZERO_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = check_head(n_tokens, vocab, dim)) return rc;
    if (in_place && dim % 8 != 0)
        return fail(ZERO_ERR_INVALID_ARG, "a table is read in place where dim is a multiple of 8");
    int64_t need = dim % 8 == 0 ? zf::head_bytes(n_tokens, vocab, dim, back, true) : 0;
    if (!in_place) {
        const int64_t copied = zf::head_bytes(n_tokens, vocab, dim, back, false);
        if (copied > need) need = copied;
    }
    *bytes = need;
    return ok();
}

}  // namespace

ZERO_API int zero_head_loss_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t dim,
                                            int64_t* bytes) {
    return head_workspace(n_tokens, vocab, dim, false, false, bytes);
}

ZERO_API int zero_head_loss_grad_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t dim,
                                                 int64_t* bytes) {
    return head_workspace(n_tokens, vocab, dim, true, false, bytes);
}

ZERO_API int zero_head_loss_in_place_workspace_bytes(int64_t n_tokens, int64_t vocab, int64_t dim,
                                                     int64_t* bytes) {
    return head_workspace(n_tokens, vocab, dim, false, true, bytes);
}

ZERO_API int zero_head_loss_grad_in_place_workspace_bytes(int64_t n_tokens, int64_t vocab,
                                                          int64_t dim, int64_t* bytes) {
    return head_workspace(n_tokens, vocab, dim, true, true, bytes);
}

ZERO_API int zero_head_loss(const uint16_t* hidden, int64_t n_tokens, int64_t dim,
                            int64_t hidden_stride, const uint16_t* table, int64_t vocab,
                            const void* labels, int32_t label_bytes, float* loss, float* lse,
                            void* workspace, int64_t workspace_bytes, void* stream) {
    zf::HeadCall c{};
    if (int rc = head_call(c, hidden, n_tokens, dim, hidden_stride, table, vocab, labels,
                           label_bytes))
        return rc;
    if (n_tokens > 0) {
        if (int rc = check_array(loss, 4, "loss")) return rc;
    }
    if (int rc = check_optional(lse, 4, "lse")) return rc;
    if (n_tokens == 0) return ok();
    const zf::HeadPlan p = zf::head_plan(n_tokens, vocab, dim, false, zf::head_table_in_place(c));
    if (int rc = check_workspace(workspace, workspace_bytes, p.bytes)) return rc;
    c.loss = loss;
    c.lse = lse;
    c.workspace = workspace;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!zf::head_rows_as_they_are(c)) {
        if (int rc = cuda_call("head rows launch",
                               [&] { return zf::launch_head_rows(c, p, false, s); }))
            return rc;
        if (int rc =
                cuda_call("head gather launch", [&] { return zf::launch_head_gather(c, p, s); }))
            return rc;
    }
    for (int64_t first = 0; first < vocab; first += p.piece) {
        if (int rc = cuda_call("head loss launch",
                               [&] { return zf::launch_head_loss(c, p, first, s); }))
            return rc;
    }
    return cuda_call("head join launch", [&] { return zf::launch_head_join(c, p, s); });
}

ZERO_API int zero_head_loss_grad(const uint16_t* hidden, int64_t n_tokens, int64_t dim,
                                 int64_t hidden_stride, const uint16_t* table, int64_t vocab,
                                 const void* labels, int32_t label_bytes, const float* lse,
                                 const float* grad_loss, uint16_t* grad_hidden,
                                 int64_t grad_hidden_stride, uint16_t* grad_table,
                                 int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
    zf::HeadCall c{};
    if (int rc = head_call(c, hidden, n_tokens, dim, hidden_stride, table, vocab, labels,
                           label_bytes))
        return rc;
    if (n_tokens > 0) {
        if (int rc = check_array(lse, 4, "lse")) return rc;
        if (int rc = check_array(grad_loss, 4, "grad_loss")) return rc;
    }
    if (int rc = check_maybe_rows(grad_hidden, n_tokens, dim, grad_hidden_stride, 2, "grad_hidden"))
        return rc;
    if (grad_hidden != nullptr) {
        if (int rc = check_in_place(grad_hidden, grad_hidden_stride, hidden, hidden_stride,
                                    n_tokens, "grad_hidden"))
            return rc;
    }
    if (int rc = check_optional(grad_table, 2, "grad_table")) return rc;
    if (grad_table != nullptr && grad_table == table)
        return fail(ZERO_ERR_INVALID_ARG, "grad_table and table are the same array");
    if (accumulate != 0 && accumulate != 1)
        return fail(ZERO_ERR_INVALID_ARG, "accumulate = %d (0 or 1)", accumulate);
    const bool rows = grad_hidden != nullptr && n_tokens > 0;
    if (!rows && (grad_table == nullptr || (n_tokens == 0 && accumulate))) return ok();
    const zf::HeadPlan p = zf::head_plan(n_tokens, vocab, dim, true, zf::head_table_in_place(c));
    if (int rc = check_workspace(workspace, workspace_bytes, p.bytes)) return rc;
    c.lse = const_cast<float*>(lse);
    c.grad_loss = grad_loss;
    c.grad_hidden = grad_hidden;
    c.grad_hidden_stride = grad_hidden_stride;
    c.grad_table = grad_table;
    c.accumulate = accumulate;
    c.workspace = workspace;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = cuda_call("head rows launch", [&] { return zf::launch_head_rows(c, p, true, s); }))
        return rc;
    if (int rc = cuda_call("head gather launch", [&] { return zf::launch_head_gather(c, p, s); }))
        return rc;
    for (int64_t first = 0; first < vocab; first += p.piece) {
        if (int rc = cuda_call("head logits' gradient launch",
                               [&] { return zf::launch_head_dz(c, p, first, s); }))
            return rc;
        if (int rc = cuda_call("head gradients launch",
                               [&] { return zf::launch_head_products(c, p, first, s); }))
            return rc;
    }
    if (!rows) return ok();
    return cuda_call("head gradient rows launch",
                     [&] { return zf::launch_head_finish(c, p, s); });
}
