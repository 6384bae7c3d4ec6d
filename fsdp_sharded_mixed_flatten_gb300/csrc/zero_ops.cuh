// Argument blocks, launchers and element access of the operators around the
// root unit: token table (zero_embed.cu), layer norm (zero_norm.cu) and
// distillation loss (zero_distill.cu).
//
// bf16 values travel as uint16_t.  A parameter or its gradient may be a piece
// of a flat buffer that starts at any element, and rows may have any stride,
// so every kernel comes in a form with vector accesses (VEC elements, up to 16
// bytes) and one with single elements (VEC = 1); the host picks the first where
// every address and stride of the call allows it.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zero_common.cuh"

namespace zf {

// ------------------------------------------------------ element access ------

template <class T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t x) { return bf16_to_float(x); }

template <class T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float x) { return float_to_bf16_rn(x); }

// VEC consecutive elements, loaded and stored as one word.
template <class T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T x[VEC];
};

template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> ld_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, VEC>*>(p);
}

template <class T, int VEC>
__device__ __forceinline__ void st_pack(T* p, const Pack<T, VEC>& v) {
    *reinterpret_cast<Pack<T, VEC>*>(p) = v;
}

template <class T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack(const float* x) {
    Pack<T, VEC> v;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v.x[e] = narrow<T>(x[e]);
    return v;
}

// One parameter value of an array whose type is known at run time.
__device__ __forceinline__ float ld_param(const void* p, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i]
               : bf16_to_float(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ void st_param(void* p, bool f32, int64_t i, float x) {
    if (f32) {
        static_cast<float*>(p)[i] = x;
    } else {
        static_cast<uint16_t*>(p)[i] = float_to_bf16_rn(x);
    }
}

// Pairs of fp32 in one 64-bit register, from end to end, so that no moves
// form them.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 unpair(Pair p) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair p;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
    return p;
}
// Two bf16 of a word (the lower one first) as fp32, and back.
__device__ __forceinline__ Pair widen2(uint32_t w) {
    Pair p;
    asm("{\n\t.reg .b32 lo, hi;\n\t"
        "shl.b32 lo, %1, 16;\n\t"
        "and.b32 hi, %1, 0xFFFF0000;\n\t"
        "mov.b64 %0, {lo, hi};\n\t}"
        : "=l"(p)
        : "r"(w));
    return p;
}
__device__ __forceinline__ uint32_t narrow2(Pair p) {
    uint32_t w;
    asm("{\n\t.reg .f32 a, b;\n\t"
        "mov.b64 {a, b}, %1;\n\t"
        "cvt.rn.bf16x2.f32 %0, b, a;\n\t}"
        : "=r"(w)
        : "l"(p));
    return w;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}

// --------------------------------------------------------- token table ------

struct EmbedArgs {
    const void* ids;          // int32 or int64, n_tokens
    const void* weight;       // [vocab][dim]
    void* out;                // rows of out_stride elements
    int64_t n_tokens;
    int64_t vocab;
    int64_t dim;
    int64_t out_stride;
    int32_t id64;
    float scale;
};

cudaError_t launch_embed(const EmbedArgs& a, int weight_bytes, int out_bytes, cudaStream_t stream);

struct EmbedGradArgs {
    const void* ids;
    const void* grad_out;     // rows of grad_stride elements
    void* grad_weight;        // [vocab][dim]
    int64_t n_tokens;
    int64_t vocab;
    int64_t dim;
    int64_t grad_stride;
    int32_t id64;
    int32_t accumulate;
    float scale;
    void* workspace;
};

int64_t embed_grad_workspace(int64_t n_tokens, int64_t vocab, int64_t dim);
// One launch (few tokens), or a sort launch and a sum launch over a workspace.
bool embed_grad_in_one(int64_t n_tokens, int64_t vocab, int64_t dim);
cudaError_t launch_embed_buckets(const EmbedGradArgs& a, int grad_bytes, int grad_weight_bytes,
                                 cudaStream_t stream);
cudaError_t launch_embed_sort(const EmbedGradArgs& a, int grad_weight_bytes, cudaStream_t stream);
cudaError_t launch_embed_sum(const EmbedGradArgs& a, int grad_bytes, int grad_weight_bytes,
                             cudaStream_t stream);

// ---------------------------------------------------------- layer norm ------

constexpr int64_t kMaxNormDim = 16384;

struct NormArgs {
    const void* x;            // rows of x_stride elements
    const void* grad_out;     // backward only
    void* out;                // the output, or grad_x
    const void* weight;       // dim values, or null (ones)
    const void* bias;         // dim values, or null (zeros); forward only
    float* mean;              // n_rows; may be null in the forward
    float* rstd;
    void* grad_weight;        // dim values, or null
    void* grad_bias;
    float* partials;          // [CTAs][2][dim] column sums of the backward
    int64_t n_rows;
    int64_t x_stride;
    int64_t grad_out_stride;
    int64_t out_stride;
    int32_t dim;
    int32_t param_f32;        // weight, bias and their gradients are fp32
    int32_t group_threads;    // threads that hold a row (set by the launch)
    float eps;
};

// CTAs of the backward launch at most, which writes one pair of partial column
// sums each.
int norm_grad_ctas(int64_t n_rows, int64_t dim);
cudaError_t launch_norm(const NormArgs& a, int act_bytes, cudaStream_t stream);
cudaError_t launch_norm_grad(const NormArgs& a, int act_bytes, cudaStream_t stream);
cudaError_t launch_norm_grad_reduce(const NormArgs& a, int act_bytes, cudaStream_t stream);

// --------------------------------------------------- distillation loss ------

constexpr int64_t kMaxTeacher = 1024;

struct DistillArgs {
    const void* logits;       // rows of logits_stride elements
    void* grad;               // rows of grad_stride elements, or null
    const int32_t* ids;       // [n_rows][top] contiguous
    const void* teacher;      // [n_rows][top] contiguous
    const float* weights;     // n_rows, or null (ones)
    float* loss;              // n_rows
    int64_t n_rows;
    int64_t logits_stride;
    int64_t grad_stride;
    int64_t vocab;
    int32_t top;
    int32_t teacher_f32;
    float c;                  // log2(e) / temperature
    float tau;
    int32_t ranks;            // CTAs of a row, a power of two (set by the launch)
    int32_t rank_shift;
    int32_t stage_words;      // 16-byte words of a row that a CTA keeps
    int32_t section;          // words a thread of one of its copy groups
};

cudaError_t launch_distill(const DistillArgs& a, int logits_bytes, cudaStream_t stream);

// ------------------------------------------------------------ launches ------

inline bool aligned_to(const void* p, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

// SMs of the current device (looked up once per device).  Launches take the
// form that reports a failed look-up; plans without a launch count one SM then.
cudaError_t device_sms(int* sms);
inline int device_sms() {
    int sms = 0;
    return device_sms(&sms) == cudaSuccess ? sms : 1;
}

}  // namespace zf
