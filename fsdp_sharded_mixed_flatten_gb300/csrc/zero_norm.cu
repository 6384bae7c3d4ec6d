// Layer norm over rows of `dim` values:
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r,
//   y = xh w + b,
// and its backward pass for g = dy w:
//   dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// A row lives in registers, E elements a thread: a warp holds a row of up to
// 32 E elements, a block of up to 1024 threads a longer one, so that every
// byte of x, dy and the output crosses memory once and the variance is the
// two-pass one.  The backward pass keeps each thread's columns of dw and db in
// registers over all rows of its CTA; each CTA writes one pair of partial
// rows, which a second launch adds up in CTA order.
#include "zero_ops.cuh"

namespace zf {

namespace {

// Sum of a pair over the threads that hold a row (WARP: one warp; else the
// block, through `red`, 2 x 32 floats used in turn).
template <bool WARP>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red, int& phase) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (WARP) {
        return make_float2(a, b);
    } else {
        float2* slot = red + 32 * phase;
        phase ^= 1;
        const int n_warps = blockDim.x / 32;
        if (threadIdx.x % 32 == 0) slot[threadIdx.x / 32] = make_float2(a, b);
        __syncthreads();
        float2 t = make_float2(0.0f, 0.0f);
        if (threadIdx.x % 32 < n_warps) t = slot[threadIdx.x % 32];
        return make_float2(warp_sum(t.x), warp_sum(t.y));
    }
}

// Rows in flight: the warps of the grid (WARP) or its blocks; lanes of a row.
template <bool WARP>
struct RowGroup {
    int64_t first, step;
    int lane, lanes;
    __device__ RowGroup() {
        if constexpr (WARP) {
            const int warps = blockDim.x / 32;
            first = static_cast<int64_t>(blockIdx.x) * warps + threadIdx.x / 32;
            step = static_cast<int64_t>(gridDim.x) * warps;
            lane = threadIdx.x % 32;
            lanes = 32;
        } else {
            first = blockIdx.x;
            step = gridDim.x;
            lane = threadIdx.x;
            lanes = blockDim.x;
        }
    }
};

template <class T, int VEC, int E, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int N = E / VEC;
    __shared__ float2 red[64];
    int phase = 0;
    const RowGroup<WARP> g;
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    for (int64_t row = g.first; row < a.n_rows; row += g.step) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        float v[E];
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int col = (n * g.lanes + g.lane) * VEC;
            if (col < a.dim) {
                const Pack<T, VEC> p = ld_pack<T, VEC>(x + col);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[n * VEC + e] = widen<T>(p.x[e]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[n * VEC + e] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) sum += v[i];
        const float mu = row_sum2<WARP>(sum, 0.0f, red, phase).x * inv_d;
        float sq = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int col = (n * g.lanes + g.lane) * VEC;
            if (col < a.dim) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = v[n * VEC + e] - mu;
                    sq += d * d;
                }
            }
        }
        const float var = row_sum2<WARP>(sq, 0.0f, red, phase).x * inv_d;
        const float r = 1.0f / sqrtf(var + a.eps);
        if (g.lane == 0) {
            if (a.mean != nullptr) a.mean[row] = mu;
            if (a.rstd != nullptr) a.rstd[row] = r;
        }
        T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int col = (n * g.lanes + g.lane) * VEC;
            if (col < a.dim) {
                float y[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float w =
                        a.weight != nullptr ? ld_param(a.weight, a.param_f32, col + e) : 1.0f;
                    const float b = a.bias != nullptr ? ld_param(a.bias, a.param_f32, col + e)
                                                      : 0.0f;
                    y[e] = (v[n * VEC + e] - mu) * r * w + b;
                }
                st_pack<T, VEC>(out + col, pack<T, VEC>(y));
            }
        }
    }
}

template <class T, int VEC, int E, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024)
norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int N = E / VEC;
    extern __shared__ float cols[];      // WARP: [warps][dim]
    __shared__ float2 red[64];
    int phase = 0;
    const RowGroup<WARP> g;
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    float dw[E], db[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.0f;
    for (int64_t row = g.first; row < a.n_rows; row += g.step) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* dy = static_cast<const T*>(a.grad_out) + row * a.grad_out_stride;
        const float mu = a.mean[row], r = a.rstd[row];
        Pack<T, VEC> px[N], py[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int col = (n * g.lanes + g.lane) * VEC;
            if (col < a.dim) {
                px[n] = ld_pack<T, VEC>(x + col);
                py[n] = ld_pack<T, VEC>(dy + col);
            }
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int col = (n * g.lanes + g.lane) * VEC;
            if (col < a.dim) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (widen<T>(px[n].x[e]) - mu) * r, d = widen<T>(py[n].x[e]);
                    const float w =
                        a.weight != nullptr ? ld_param(a.weight, a.param_f32, col + e) : 1.0f;
                    dw[n * VEC + e] += d * xh;
                    db[n * VEC + e] += d;
                    s1 += d * w;
                    s2 += d * w * xh;
                }
            }
        }
        const float2 s = row_sum2<WARP>(s1, s2, red, phase);
        const float m1 = s.x * inv_d, m2 = s.y * inv_d;
        T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int col = (n * g.lanes + g.lane) * VEC;
            if (col < a.dim) {
                float y[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (widen<T>(px[n].x[e]) - mu) * r, d = widen<T>(py[n].x[e]);
                    const float w =
                        a.weight != nullptr ? ld_param(a.weight, a.param_f32, col + e) : 1.0f;
                    y[e] = r * (d * w - m1 - xh * m2);
                }
                st_pack<T, VEC>(out + col, pack<T, VEC>(y));
            }
        }
    }
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.dim;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float* acc = which == 0 ? dw : db;
        float* to = WARP ? cols + (threadIdx.x / 32) * a.dim : part + which * a.dim;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int col = (n * g.lanes + g.lane) * VEC;
            if (col < a.dim) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) to[col + e] = acc[n * VEC + e];
            }
        }
        if constexpr (WARP) {
            __syncthreads();
            const int warps = blockDim.x / 32;
            for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
                float t = 0.0f;
                for (int k = 0; k < warps; ++k) t += cols[k * a.dim + c];
                part[which * a.dim + c] = t;
            }
            __syncthreads();
        }
    }
}

// Column sums over the CTAs' partial rows: 32 columns a block, 16 strands of
// CTAs each, joined in a fixed order.
constexpr int kStrands = 16;

__global__ void __launch_bounds__(32 * kStrands)
norm_grad_reduce_kernel(const __grid_constant__ NormArgs a, int n_parts) {
    __shared__ float sum[kStrands][33];
    const int lane = threadIdx.x % 32, strand = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;   // of 2 dim columns
    const int64_t width = 2 * static_cast<int64_t>(a.dim);
    float t = 0.0f;
    if (c < width) {
        for (int i = strand; i < n_parts; i += kStrands) t += a.partials[i * width + c];
    }
    sum[strand][lane] = t;
    __syncthreads();
    if (strand == 0 && c < width) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < kStrands; ++i) t += sum[i][lane];
        void* to = c < a.dim ? a.grad_weight : a.grad_bias;
        if (to != nullptr) st_param(to, a.param_f32, c < a.dim ? c : c - a.dim, t);
    }
}

// How a row is held: elements per thread, and threads (32: a warp a row).
struct Shape {
    int e, threads;
    bool warp;
};

Shape shape_for(int64_t dim) {
    if (dim <= 256) return {8, 256, true};
    if (dim <= 512) return {16, 256, true};
    if (dim <= 768) return {24, 256, true};
    if (dim <= 1024) return {32, 256, true};
    return {16, static_cast<int>((dim + 511) / 512 * 32), false};
}

int64_t row_blocks(const Shape& s, int64_t rows) {
    return s.warp ? (rows + s.threads / 32 - 1) / (s.threads / 32) : rows;
}

// Elements of one access that every row of a matrix allows.
int row_vec(int want, int elem, const void* p, int64_t stride, int64_t dim) {
    return aligned_to(p, static_cast<int64_t>(want) * elem) && stride % want == 0 &&
                   dim % want == 0
               ? want
               : 1;
}

template <class T, int VEC, bool BACK>
cudaError_t launch_shape(const NormArgs& a, cudaStream_t stream) {
    const Shape s = shape_for(a.dim);
    int64_t blocks = row_blocks(s, a.n_rows);
    size_t smem = 0;
    if (BACK) {
        blocks = norm_grad_ctas(a.n_rows, a.dim);
        if (s.warp) smem = static_cast<size_t>(s.threads / 32) * a.dim * sizeof(float);
    } else if (blocks > (int64_t{1} << 30)) {
        blocks = int64_t{1} << 30;
    }
    const unsigned g = static_cast<unsigned>(blocks);
#define ZF_NORM(E, WARP)                                                                   \
    do {                                                                                   \
        if constexpr (BACK)                                                                \
            norm_grad_kernel<T, VEC, E, WARP><<<g, s.threads, smem, stream>>>(a);          \
        else                                                                               \
            norm_kernel<T, VEC, E, WARP><<<g, s.threads, 0, stream>>>(a);                  \
        return cudaGetLastError();                                                         \
    } while (0)
    if (s.warp) {
        if (s.e == 8) ZF_NORM(8, true);
        if (s.e == 16) ZF_NORM(16, true);
        if (s.e == 24) ZF_NORM(24, true);
        ZF_NORM(32, true);
    }
    ZF_NORM(16, false);
#undef ZF_NORM
}

template <bool BACK>
cudaError_t dispatch(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    const int want = 16 / act_bytes;
    int vec = row_vec(want, act_bytes, a.x, a.x_stride, a.dim);
    if (row_vec(want, act_bytes, a.out, a.out_stride, a.dim) == 1) vec = 1;
    if (BACK && row_vec(want, act_bytes, a.grad_out, a.grad_out_stride, a.dim) == 1) vec = 1;
    if (act_bytes == 4)
        return vec == 4 ? launch_shape<float, 4, BACK>(a, stream)
                        : launch_shape<float, 1, BACK>(a, stream);
    return vec == 8 ? launch_shape<uint16_t, 8, BACK>(a, stream)
                    : launch_shape<uint16_t, 1, BACK>(a, stream);
}

}  // namespace

int norm_grad_ctas(int64_t n_rows, int64_t dim) {
    const Shape s = shape_for(dim);
    const int64_t blocks = row_blocks(s, n_rows);
    const int64_t most = static_cast<int64_t>(device_sms()) * (s.warp ? 2 : 1);
    return static_cast<int>(blocks < most ? (blocks > 0 ? blocks : 1) : most);
}

cudaError_t launch_norm(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    return dispatch<false>(a, act_bytes, stream);
}

cudaError_t launch_norm_grad(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    return dispatch<true>(a, act_bytes, stream);
}

cudaError_t launch_norm_grad_reduce(const NormArgs& a, cudaStream_t stream) {
    const int64_t width = 2 * static_cast<int64_t>(a.dim);
    norm_grad_reduce_kernel<<<static_cast<unsigned>((width + 31) / 32), 32 * kStrands, 0, stream>>>(
        a, norm_grad_ctas(a.n_rows, a.dim));
    return cudaGetLastError();
}

}  // namespace zf
