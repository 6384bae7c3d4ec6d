// Root-mean-square norm over rows of `dim` values, with the residual's addition:
//   s = x + res,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w,
// and its backward pass for xh = s r, g = dy w, dt the gradient that reaches s past the
// norm:
//   dx = dt + r (g - xh mean(g xh)),  dw = sum_rows dy xh.
// y and s may be written in 8 bits (zero_eight.cuh), and the backward pass reads s from
// them, so that a training step keeps a byte an element of it.
//
// A row lives in the registers of a group of threads, 8 K elements each; a CTA holds
// several groups, which work through the rows independently, the next row's loads under
// way while a row is worked on.  The backward pass keeps its columns of dw in registers
// over all rows; each CTA writes one partial row, which a second launch adds up in CTA
// order.
#include "zero_eight.cuh"
#include "zero_ops.cuh"

namespace zf {

namespace {

constexpr int kRmsWarps = 32;          // of a CTA, at most

// The group of threads that holds a row.
struct RmsGroup {
    int threads, warps, index, per_cta, t;
    __device__ explicit RmsGroup(int group_threads)
        : threads(group_threads),
          warps(group_threads / 32),
          index(threadIdx.x / group_threads),
          per_cta(blockDim.x / group_threads),
          t(threadIdx.x - (threadIdx.x / group_threads) * group_threads) {}
    __device__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
    }
};

// Sum over a group, in a fixed order.  `red` has two halves used in turn: one barrier a
// call is enough.
__device__ __forceinline__ float rms_group_sum(const RmsGroup& g, float v,
                                               float (*red)[kRmsWarps], int& half) {
    v = warp_sum(v);
    if (g.warps == 1) return v;
    const int lane = threadIdx.x % 32, w0 = g.index * g.warps;
    if (lane == 0) red[half][w0 + g.t / 32] = v;
    g.sync();
    v = warp_sum(lane < g.warps ? red[half][w0 + lane] : 0.0f);
    half ^= 1;
    return v;
}

template <class T, int K, bool WIDE>
__global__ void __launch_bounds__(K == 4 ? 512 : 1024)
rms_norm_kernel(const __grid_constant__ RmsArgs a) {
    __shared__ float red[2][kRmsWarps];
    int half = 0;
    const RmsGroup g(a.group_threads);
    const Octets<WIDE, K> c(g.t, g.threads, a.dim);
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index;
    Octet<T> x[K], res[K];
    auto load = [&](int64_t at) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = c.template load<T>(static_cast<const T*>(a.x) + at * a.x_stride, k);
            if (a.residual != nullptr)
                res[k] = c.template load<T>(static_cast<const T*>(a.residual) +
                                            at * a.residual_stride, k);
        }
    };
    if (row < a.n_rows) load(row);
    for (; row < a.n_rows; row += step) {
        float s[K][8];
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[k][e] = widen<T>(x[k].x[e]);
                if (a.residual != nullptr) s[k][e] = __fadd_rn(s[k][e], widen<T>(res[k].x[e]));
                q = __fmaf_rn(s[k][e], s[k][e], q);
            }
        }
        if (row + step < a.n_rows) load(row + step);
        if (a.total != nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                c.template store<T>(static_cast<T*>(a.total) + row * a.total_stride, k, s[k]);
        }
        if (a.total8 != nullptr) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                c.store_eight(a.total8 + row * a.total8_stride, a.total8_scales + row * a.blocks,
                              k, s[k]);
        }
        const float r = inv_sqrt(__fmaf_rn(rms_group_sum(g, q, red, half), inv_d, a.eps));
        if (g.t == 0 && a.rstd != nullptr) a.rstd[row] = r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[8];
            c.params(w, a.weight, a.param_f32, k);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = s[k][e] * r * w[e];
            if (a.out != nullptr)
                c.template store<T>(static_cast<T*>(a.out) + row * a.out_stride, k, w);
            if (a.out8 != nullptr)
                c.store_eight(a.out8 + row * a.out8_stride, a.out8_scales + row * a.blocks, k, w);
        }
    }
}

// EIGHT: s comes in 8 bits.
template <class T, int K, bool WIDE, bool EIGHT>
__global__ void __launch_bounds__(K == 4 ? 512 : 1024)
rms_norm_grad_kernel(const __grid_constant__ RmsArgs a) {
    extern __shared__ float cols[];                  // [groups][dim] at the end
    __shared__ float red[2][kRmsWarps];
    int half = 0;
    const RmsGroup g(a.group_threads);
    const Octets<WIDE, K> c(g.t, g.threads, a.dim);
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index;
    float dw[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[k][e] = 0.0f;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (; row < a.n_rows; row += step) {
        float xh[K][8], gr[K][8];
        const float r = a.rstd[row];
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (EIGHT) {
                c.load_eight(xh[k], a.total8 + row * a.total8_stride,
                             a.total8_scales + row * a.blocks, k);
            } else {
                const Octet<T> v =
                    c.template load<T>(static_cast<const T*>(a.x) + row * a.x_stride, k);
#pragma unroll
                for (int e = 0; e < 8; ++e) xh[k][e] = widen<T>(v.x[e]);
            }
            const Octet<T> dy =
                c.template load<T>(static_cast<const T*>(a.grad_out) + row * a.grad_out_stride, k);
            float w[8];
            c.params(w, a.weight, a.param_f32, k);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = widen<T>(dy.x[e]);
                xh[k][e] *= r;
                gr[k][e] = d * w[e];
                dw[k][e] = __fmaf_rn(d, xh[k][e], dw[k][e]);
                q = __fmaf_rn(gr[k][e], xh[k][e], q);
                w[e] *= xh[k][e];
            }
            if (a.out != nullptr)
                c.template store<T>(static_cast<T*>(a.out) + row * a.out_stride, k, w);
        }
        const float m = -rms_group_sum(g, q, red, half) * inv_d;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Octet<T> t{};
            if (a.grad_total != nullptr)
                t = c.template load<T>(static_cast<const T*>(a.grad_total) +
                                       row * a.grad_total_stride, k);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = r * __fmaf_rn(xh[k][e], m, gr[k][e]);
                if (a.grad_total != nullptr) y[e] += widen<T>(t.x[e]);
            }
            c.template store<T>(static_cast<T*>(a.grad_x) + row * a.grad_x_stride, k, y);
        }
    }
    if (a.grad_weight == nullptr) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c.ok(k, e)) cols[g.index * a.dim + c.at(k, e)] = dw[k][e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.dim; i += blockDim.x) {
        float t = 0.0f;
        for (int j = 0; j < g.per_cta; ++j) t += cols[j * a.dim + i];
        if (gridDim.x == 1) st_param(a.grad_weight, a.param_f32, i, t);
        else a.partials[static_cast<int64_t>(blockIdx.x) * a.dim + i] = t;
    }
}

// Column sums over the CTAs' partial rows: 32 columns a block, 32 strands of CTAs, joined
// in a fixed order.
constexpr int kRmsStrands = 32;

__global__ void __launch_bounds__(32 * kRmsStrands)
rms_reduce_kernel(const __grid_constant__ RmsArgs a, int n_parts) {
    __shared__ float sum[kRmsStrands][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");       // the partial rows are there
    const int lane = threadIdx.x % 32, strand = threadIdx.x / 32;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (c < a.dim) {
#pragma unroll 4
        for (int i = strand; i < n_parts; i += kRmsStrands)
            t += a.partials[static_cast<int64_t>(i) * a.dim + c];
    }
    sum[strand][lane] = t;
    __syncthreads();
    t = warp_sum(sum[lane][strand]);
    const int to = blockIdx.x * 32 + strand;
    if (lane == 0 && to < a.dim) st_param(a.grad_weight, a.param_f32, to, t);
}

// Rows of any width in 8 bits and back: a warp takes up to 1024 columns of a row.
constexpr int kEightWarps = 8;
constexpr int kEightOctets = 4;

template <class T, bool WIDE>
__global__ void __launch_bounds__(32 * kEightWarps)
pack_kernel(const __grid_constant__ EightArgs a) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kEightWarps + threadIdx.x / 32;
    const int64_t row = id / a.sections;
    if (row >= a.n_rows) return;
    const int64_t first = (id - row * a.sections) * a.section;
    const int64_t rest = a.dim - first;
    const Octets<WIDE, kEightOctets> c(threadIdx.x % 32, 32,
                                       static_cast<int>(rest < a.section ? rest : a.section));
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + first;
    Octet<T> v[kEightOctets];
#pragma unroll
    for (int k = 0; k < kEightOctets; ++k) v[k] = c.template load<T>(x, k);
#pragma unroll
    for (int k = 0; k < kEightOctets; ++k) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = widen<T>(v[k].x[e]);
        c.store_eight(a.codes + row * a.codes_stride + first,
                      a.scales + row * a.blocks + first / kEightBlock, k, f);
    }
}

template <class T, bool WIDE>
__global__ void __launch_bounds__(32 * kEightWarps)
unpack_kernel(const __grid_constant__ EightArgs a) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kEightWarps + threadIdx.x / 32;
    const int64_t row = id / a.sections;
    if (row >= a.n_rows) return;
    const int64_t first = (id - row * a.sections) * a.section;
    const int64_t rest = a.dim - first;
    const Octets<WIDE, kEightOctets> c(threadIdx.x % 32, 32,
                                       static_cast<int>(rest < a.section ? rest : a.section));
    float f[kEightOctets][8];
#pragma unroll
    for (int k = 0; k < kEightOctets; ++k)
        c.load_eight(f[k], a.codes + row * a.codes_stride + first,
                     a.scales + row * a.blocks + first / kEightBlock, k);
#pragma unroll
    for (int k = 0; k < kEightOctets; ++k)
        c.template store<T>(static_cast<T*>(a.out) + row * a.x_stride + first, k, f[k]);
}

// How rows are held: octets a thread, threads of a group, groups of a CTA.
struct RmsShape {
    int k, group, per_cta;
};

RmsShape rms_shape(int64_t dim) {
    const int k = dim <= 4096 ? 1 : dim <= 8192 ? 2 : 4;
    const int group = static_cast<int>((dim + 256 * k - 1) / (256 * k) * 32);
    int per_cta = 512 / group;
    if (per_cta > 8) per_cta = 8;               // 16 hardware barriers a CTA
    return {k, group, per_cta};
}

int64_t rms_grid(const RmsShape& s, int64_t rows, int64_t per_sm) {
    const int64_t need = (rows + s.per_cta - 1) / s.per_cta;
    const int64_t most = static_cast<int64_t>(device_sms()) * per_sm;
    return need < 1 ? 1 : need < most ? need : most;
}

int64_t rms_forward_grid(const RmsShape& s, int64_t rows) {
    return rms_grid(s, rows, s.k == 4 ? 1 : 1024 / (s.group * s.per_cta));
}

int64_t rms_backward_grid(const RmsShape& s, int64_t rows) { return rms_grid(s, rows, 1); }

template <class F>
cudaError_t by_k(int k, F&& f) {
    if (k == 1) return f(std::integral_constant<int, 1>{});
    if (k == 2) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 4>{});
}

template <class F>
cudaError_t by_type(int bytes, F&& f) {
    return bytes == 4 ? f(float{}) : f(uint16_t{});
}

bool wide_rows(const void* p, int64_t stride, int bytes) {
    return p == nullptr || (aligned_to(p, 16) && stride * bytes % 16 == 0);
}

// Codes are reached 8 bytes at a time.
bool wide_codes(const void* p, int64_t stride) {
    return p == nullptr || (aligned_to(p, 8) && stride % 8 == 0);
}

}  // namespace

int rms_grad_ctas(int64_t n_rows, int64_t dim) {
    return static_cast<int>(rms_backward_grid(rms_shape(dim), n_rows));
}

cudaError_t launch_rms_norm(RmsArgs a, int act_bytes, cudaStream_t stream) {
    const RmsShape s = rms_shape(a.dim);
    a.group_threads = s.group;
    const bool wide = wide_rows(a.x, a.x_stride, act_bytes) &&
                      wide_rows(a.residual, a.residual_stride, act_bytes) &&
                      wide_rows(a.total, a.total_stride, act_bytes) &&
                      wide_rows(a.out, a.out_stride, act_bytes) &&
                      wide_codes(a.out8, a.out8_stride) && wide_codes(a.total8, a.total8_stride);
    const unsigned grid = static_cast<unsigned>(rms_forward_grid(s, a.n_rows));
    return by_type(act_bytes, [&](auto t) {
        using T = decltype(t);
        return by_k(s.k, [&](auto k) {
            if (wide) rms_norm_kernel<T, k.value, true><<<grid, s.group * s.per_cta, 0, stream>>>(a);
            else rms_norm_kernel<T, k.value, false><<<grid, s.group * s.per_cta, 0, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_rms_norm_grad(RmsArgs a, int act_bytes, cudaStream_t stream) {
    const RmsShape s = rms_shape(a.dim);
    a.group_threads = s.group;
    const bool wide = wide_rows(a.x, a.x_stride, act_bytes) &&
                      wide_rows(a.grad_out, a.grad_out_stride, act_bytes) &&
                      wide_rows(a.grad_total, a.grad_total_stride, act_bytes) &&
                      wide_rows(a.grad_x, a.grad_x_stride, act_bytes) &&
                      wide_rows(a.out, a.out_stride, act_bytes) &&
                      wide_codes(a.total8, a.total8_stride);
    const unsigned grid = static_cast<unsigned>(rms_backward_grid(s, a.n_rows));
    const size_t smem = sizeof(float) * s.per_cta * a.dim;
    return by_type(act_bytes, [&](auto t) {
        using T = decltype(t);
        return by_k(s.k, [&](auto k) {
            constexpr int K = k.value;
            const auto kernel = a.total8 != nullptr
                                    ? (wide ? rms_norm_grad_kernel<T, K, true, true>
                                            : rms_norm_grad_kernel<T, K, false, true>)
                                    : (wide ? rms_norm_grad_kernel<T, K, true, false>
                                            : rms_norm_grad_kernel<T, K, false, false>);
            // at most 64 KB: 4 groups of 4096 columns, 1 of 16384
            if (cudaError_t e = cudaFuncSetAttribute(
                    kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
                e != cudaSuccess)
                return e;
            kernel<<<grid, s.group * s.per_cta, smem, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_rms_reduce(const RmsArgs& a, cudaStream_t stream) {
    const int64_t parts = rms_backward_grid(rms_shape(a.dim), a.n_rows);
    if (parts == 1) return cudaSuccess;                      // the sums themselves are there
    // its blocks may be set up while the partial rows are still being added up
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((a.dim + 31) / 32));
    cfg.blockDim = dim3(32 * kRmsStrands);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rms_reduce_kernel, a, static_cast<int>(parts));
}

cudaError_t launch_eight(EightArgs a, int act_bytes, cudaStream_t stream) {
    a.section = 256 * kEightOctets;
    a.sections = (a.dim + a.section - 1) / a.section;
    const bool pack = a.out == nullptr;
    const void* act = pack ? a.x : a.out;
    const bool wide = wide_rows(act, a.x_stride, act_bytes) && wide_codes(a.codes, a.codes_stride);
    const int64_t ctas = (a.n_rows * a.sections + kEightWarps - 1) / kEightWarps;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(ctas);
    return by_type(act_bytes, [&](auto t) {
        using T = decltype(t);
        const auto kernel = pack ? (wide ? pack_kernel<T, true> : pack_kernel<T, false>)
                                 : (wide ? unpack_kernel<T, true> : unpack_kernel<T, false>);
        kernel<<<grid, 32 * kEightWarps, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace zf
