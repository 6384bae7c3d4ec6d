// Layer norm over rows of `dim` values:
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r,
//   y = xh w + b,
// and its backward pass for g = dy w:
//   dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// A row lives in the registers of a group of threads, E elements each, so that
// every byte of x, dy and the output crosses memory once.  A CTA holds several
// groups, which work through the rows independently, kBatch rows at a time:
// one group barrier then serves the sums of several rows, and the next batch's
// loads are under way meanwhile.  The parameters stay in registers over all
// rows, and so do the backward pass's columns of dw and db; each CTA writes
// one pair of partial rows, which a second launch adds up in CTA order.
//
// The variance is taken about a mean at every step: a warp's squares about the
// warp's mean, then sum (M2_w + n_w (mean_w - mu)^2) over the warps of the
// row, so that a mean far from zero costs no digits and one exchange is enough.
#include "zero_ops.cuh"

namespace zf {

namespace {

constexpr int kNormThreads = 512;      // of a CTA, at most
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kSmallThreads = 384;     // of the forward pass at E = 8: 768 an SM, 80 registers

// Rows per batch, as far as 128 registers a thread go.
__host__ __device__ constexpr int batch_of(int e) { return e == 8 ? 2 : 1; }

// The group of threads that holds a row.
struct Group {
    int threads, warps;        // of a group
    int index, per_cta;        // this group's place in its CTA
    int t;                     // this thread's place in its group
    __device__ explicit Group(int group_threads)
        : threads(group_threads),
          warps(group_threads / 32),
          index(threadIdx.x / group_threads),
          per_cta(blockDim.x / group_threads),
          t(threadIdx.x - (threadIdx.x / group_threads) * group_threads) {}
    __device__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
    }
};

// This thread's columns: pack n holds columns n * group * VEC + t * VEC ...;
// `ok` says which packs there are.
template <int VEC, int E>
struct Columns {
    static constexpr int N = E / VEC;
    int first, step;
    bool ok[N];
    __device__ Columns(const Group& g, int dim) : first(g.t * VEC), step(g.threads * VEC) {
#pragma unroll
        for (int n = 0; n < N; ++n) ok[n] = first + n * step < dim;
    }
    __device__ __forceinline__ int at(int n) const { return first + n * step; }
};

// A row's E elements as loaded, zeros where there are none.
template <class T, int VEC, int E>
struct Row {
    static constexpr int N = E / VEC;
    Pack<T, VEC> p[N];
    __device__ __forceinline__ void load(const T* at, bool in, const Columns<VEC, E>& c) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            p[n] = Pack<T, VEC>{};
            if (in && c.ok[n]) p[n] = ld_pack<T, VEC>(at + n * c.step);
        }
    }
    // element pairs (2 i, 2 i + 1) in fp32
    __device__ __forceinline__ Pair operator[](int i) const {
        if constexpr (VEC == 1) {
            return pair(widen<T>(p[2 * i].x[0]), widen<T>(p[2 * i + 1].x[0]));
        } else if constexpr (sizeof(T) == 2) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&p[2 * i / VEC])[i % (VEC / 2)];
            return widen2(w);
        } else {
            const auto& v = p[2 * i / VEC];
            return pair(widen<T>(v.x[2 * i % VEC]), widen<T>(v.x[2 * i % VEC + 1]));
        }
    }
};

template <class T, int VEC, int E>
__device__ __forceinline__ void store_row(T* at, const Pair (&y)[E / 2], const Columns<VEC, E>& c) {
#pragma unroll
    for (int n = 0; n < E / VEC; ++n) {
        if (!c.ok[n]) continue;
        Pack<T, VEC> v;
        if constexpr (VEC == 1) {
            const float2 f = unpair(y[n / 2]);
            v.x[0] = narrow<T>(n % 2 == 0 ? f.x : f.y);
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i)
                reinterpret_cast<uint32_t*>(&v)[i] = narrow2(y[n * VEC / 2 + i]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 f = unpair(y[n * VEC / 2 + i]);
                v.x[2 * i] = narrow<T>(f.x);
                v.x[2 * i + 1] = narrow<T>(f.y);
            }
        }
        st_pack<T, VEC>(at + n * c.step, v);
    }
}

// The parameters of this thread's columns (`missing` where there is no array
// or no column).
template <int VEC, int E>
__device__ __forceinline__ void ld_params(Pair (&w)[E / 2], const void* p, bool f32,
                                          const Columns<VEC, E>& c, float missing) {
    float v[E];
#pragma unroll
    for (int n = 0; n < E / VEC; ++n) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            v[n * VEC + e] = p != nullptr && c.ok[n] ? ld_param(p, f32, c.at(n) + e) : missing;
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = pair(v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ float both(Pair p) {
    const float2 v = unpair(p);
    return v.x + v.y;
}

__device__ __forceinline__ Pair splat(float x) { return pair(x, x); }

// Sums of K pairs of values over a group, in a fixed order: lanes, then warps.
// `red` has two halves that are used in turn: one barrier a call is enough.
template <int K>
__device__ __forceinline__ void group_sum(const Group& g, float2 (&x)[K],
                                          float2 (*red)[K][kNormWarps], int& half) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = make_float2(warp_sum(x[k].x), warp_sum(x[k].y));
    if (g.warps == 1) return;
    float2(*slot)[kNormWarps] = red[half];
    half ^= 1;
    const int w0 = g.index * g.warps, lane = threadIdx.x % 32;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) slot[k][w0 + g.t / 32] = x[k];
    }
    g.sync();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const float2 v = lane < g.warps ? slot[k][w0 + lane] : make_float2(0.0f, 0.0f);
        x[k] = make_float2(warp_sum(v.x), warp_sum(v.y));
    }
}

template <class T, int VEC, int E>
__global__ void __launch_bounds__(E == 8 ? kSmallThreads : kNormThreads, E == 8 ? 2 : 1)
norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kBatch = batch_of(E), P = E / 2;
    __shared__ float2 red[2][kBatch][kNormWarps];
    int half = 0;
    const Group g(a.group_threads);
    const Columns<VEC, E> c(g, a.dim);
    const int lane = threadIdx.x % 32;
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    // columns of this warp, and of the warp `lane` of the group
    auto columns_of = [&](int w) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < E / VEC; ++k)
            n += min(max(a.dim - (k * g.threads + w * 32) * VEC, 0), 32 * VEC);
        return static_cast<float>(n);
    };
    const float inv_n = 1.0f / fmaxf(columns_of(g.t / 32), 1.0f);
    const float lane_n = columns_of(lane);
    const float lane_inv_n = 1.0f / fmaxf(lane_n, 1.0f);
    Pair w[P], b[P];
    ld_params<VEC, E>(w, a.weight, a.param_f32, c, 1.0f);
    ld_params<VEC, E>(b, a.bias, a.param_f32, c, 0.0f);
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta * kBatch;
    int64_t row = (static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index) * kBatch;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + c.first;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + c.first;
    Row<T, VEC, E> next[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) next[i].load(x + i * a.x_stride, row + i < a.n_rows, c);
    for (; row < a.n_rows; row += step, out += step * a.out_stride) {
        Pair v[kBatch][P];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
#pragma unroll
            for (int j = 0; j < P; ++j) v[i][j] = next[i][j];
        }
        x += step * a.x_stride;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            next[i].load(x + i * a.x_stride, row + step + i < a.n_rows, c);
        float2 s[kBatch];        // a warp's sum, and its squares about its mean
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            Pair t = v[i][0];
#pragma unroll
            for (int j = 1; j < P; ++j) t = add2(t, v[i][j]);
            s[i].x = warp_sum(both(t));
            const Pair m = splat(-s[i].x * inv_n);
            Pair q = 0;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                Pair d = add2(v[i][j], m);
                if constexpr (VEC == 1) {
                    const float2 f = unpair(d);
                    d = pair(c.ok[2 * j] ? f.x : 0.0f, c.ok[2 * j + 1] ? f.y : 0.0f);
                } else {
                    d = c.ok[2 * j / VEC] ? d : 0;
                }
                q = fma2(d, d, q);
            }
            s[i].y = warp_sum(both(q));
        }
        if (g.warps > 1) {
            const int w0 = g.index * g.warps;
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) red[half][i][w0 + g.t / 32] = s[i];
            }
            g.sync();
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float2 o =
                    lane < g.warps ? red[half][i][w0 + lane] : make_float2(0.0f, 0.0f);
                s[i].x = warp_sum(o.x);
                const float d = __fmaf_rn(o.x, lane_inv_n, -s[i].x * inv_d);
                s[i].y = warp_sum(lane < g.warps ? __fmaf_rn(lane_n * d, d, o.y) : 0.0f);
            }
            half ^= 1;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (row + i >= a.n_rows) break;
            const float mu = s[i].x * inv_d;
            const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fmaf_rn(s[i].y, inv_d, a.eps)));
            if (g.t == 0) {
                if (a.mean != nullptr) a.mean[row + i] = mu;
                if (a.rstd != nullptr) a.rstd[row + i] = r;
            }
            const Pair m2 = splat(-mu), r2 = splat(r);
#pragma unroll
            for (int j = 0; j < P; ++j) v[i][j] = fma2(mul2(add2(v[i][j], m2), r2), w[j], b[j]);
            store_row<T, VEC, E>(out + i * a.out_stride, v[i], c);
        }
    }
}

template <class T, int VEC, int E>
__global__ void __launch_bounds__(kNormThreads, 1)
norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kBatch = batch_of(E), P = E / 2;
    extern __shared__ float cols[];          // [groups][dim] where a CTA has several
    __shared__ float2 red[2][kBatch][kNormWarps];
    int half = 0;
    const Group g(a.group_threads);
    const Columns<VEC, E> c(g, a.dim);
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    Pair w[P], dw[P], db[P];
    ld_params<VEC, E>(w, a.weight, a.param_f32, c, 1.0f);
#pragma unroll
    for (int j = 0; j < P; ++j) dw[j] = db[j] = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta * kBatch;
    int64_t row = (static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index) * kBatch;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + c.first;
    const T* dy = static_cast<const T*>(a.grad_out) + row * a.grad_out_stride + c.first;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + c.first;
    Row<T, VEC, E> next_x[kBatch], next_y[kBatch];
    float next_mu[kBatch], next_r[kBatch];
    auto load = [&](int64_t at) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const bool in = at + i < a.n_rows;
            next_x[i].load(x + i * a.x_stride, in, c);
            next_y[i].load(dy + i * a.grad_out_stride, in, c);
            next_mu[i] = in ? a.mean[at + i] : 0.0f;
            next_r[i] = in ? a.rstd[at + i] : 0.0f;
        }
    };
    load(row);
    for (; row < a.n_rows; row += step, out += step * a.out_stride) {
        Pair xh[kBatch][P], gr[kBatch][P];
        float r[kBatch];
        float2 s[kBatch];
        // dy is 0 where there is no row or column, and adds nothing there
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const Pair m2 = splat(-next_mu[i]), r2 = splat(next_r[i]);
            r[i] = next_r[i];
            Pair s1 = 0, s2 = 0;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const Pair d = next_y[i][j];
                xh[i][j] = mul2(add2(next_x[i][j], m2), r2);
                gr[i][j] = mul2(d, w[j]);
                dw[j] = fma2(d, xh[i][j], dw[j]);
                db[j] = add2(db[j], d);
                s1 = add2(s1, gr[i][j]);
                s2 = fma2(gr[i][j], xh[i][j], s2);
            }
            s[i] = make_float2(both(s1), both(s2));
        }
        x += step * a.x_stride;
        dy += step * a.grad_out_stride;
        load(row + step);
        group_sum<kBatch>(g, s, red, half);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (row + i >= a.n_rows) break;
            const Pair r2 = splat(r[i]), m1 = splat(-s[i].x * inv_d * r[i]);
            const Pair m2 = splat(-s[i].y * inv_d * r[i]);
#pragma unroll
            for (int j = 0; j < P; ++j)
                gr[i][j] = fma2(xh[i][j], m2, fma2(gr[i][j], r2, m1));
            store_row<T, VEC, E>(out + i * a.out_stride, gr[i], c);
        }
    }
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.dim;
    auto put = [&](const Pair (&acc)[P], float* to) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float2 f = unpair(acc[j]);
            const int n0 = 2 * j / VEC, n1 = (2 * j + 1) / VEC;
            if (c.ok[n0]) to[c.at(n0) + 2 * j % VEC] = f.x;
            if (c.ok[n1]) to[c.at(n1) + (2 * j + 1) % VEC] = f.y;
        }
    };
    if (g.per_cta == 1) {
        put(dw, part);
        put(db, part + a.dim);
        return;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        put(which == 0 ? dw : db, cols + g.index * a.dim);
        __syncthreads();
        for (int k = threadIdx.x; k < a.dim; k += blockDim.x) {
            float t = 0.0f;
            for (int i = 0; i < g.per_cta; ++i) t += cols[i * a.dim + k];
            part[which * a.dim + k] = t;
        }
    }
}

// Column sums over the CTAs' partial rows: 32 columns a block, 32 strands of
// CTAs each with several loads in flight, joined in a fixed order.
constexpr int kStrands = 32;
constexpr int kStrandLoads = 5;

__global__ void __launch_bounds__(32 * kStrands)
norm_grad_reduce_kernel(const __grid_constant__ NormArgs a, int n_parts) {
    __shared__ float sum[kStrands][33];
    const int lane = threadIdx.x % 32, strand = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;   // of 2 dim columns
    const int64_t width = 2 * static_cast<int64_t>(a.dim);
    float t = 0.0f;
    if (c < width) {
        const float* p = a.partials + c;
        for (int i = strand; i < n_parts; i += kStrands * kStrandLoads) {
            float v[kStrandLoads];
#pragma unroll
            for (int u = 0; u < kStrandLoads; ++u) {
                const int at = i + u * kStrands;
                v[u] = at < n_parts ? p[at * width] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < kStrandLoads; ++u) t += v[u];
        }
    }
    sum[strand][lane] = t;
    __syncthreads();
    // warp s adds up column s over the strands
    t = warp_sum(sum[lane][strand]);
    const int64_t to_c = static_cast<int64_t>(blockIdx.x) * 32 + strand;
    if (lane == 0 && to_c < width) {
        void* to = to_c < a.dim ? a.grad_weight : a.grad_bias;
        if (to != nullptr) st_param(to, a.param_f32, to_c < a.dim ? to_c : to_c - a.dim, t);
    }
}

// How rows are held: elements per thread, threads of a group, groups of a CTA.
struct Shape {
    int e, group, per_cta;
};

Shape shape_for(int64_t dim, bool back) {
    const int e = dim <= 2048 ? 8 : dim <= 16 * kNormThreads ? 16 : 32;
    const int group = static_cast<int>((dim + e * 32 - 1) / (e * 32) * 32);
    int per_cta = (back || e != 8 ? kNormThreads : kSmallThreads) / group;
    if (per_cta > 8) per_cta = 8;               // 16 hardware barriers a CTA
    return {e, group, per_cta};
}

int64_t ctas_for(const Shape& s, int64_t rows, bool back) {
    const int threads = s.group * s.per_cta;
    const int per_sm = back || s.e != 8 ? kNormThreads / threads : 2 * kSmallThreads / threads;
    const int64_t per = static_cast<int64_t>(s.per_cta) * batch_of(s.e);
    const int64_t need = rows > 0 ? (rows + per - 1) / per : 1;
    const int64_t most = static_cast<int64_t>(device_sms()) * per_sm;
    return need < most ? need : most;
}

// Whether every row of a matrix allows accesses of 16 bytes.
bool wide_rows(int elem, const void* p, int64_t stride, int64_t dim) {
    const int want = 16 / elem;
    return aligned_to(p, 16) && stride % want == 0 && dim % want == 0;
}

template <class T, int VEC, bool BACK>
cudaError_t launch_shape(NormArgs a, cudaStream_t stream) {
    const Shape s = shape_for(a.dim, BACK);
    a.group_threads = s.group;
    const unsigned g = static_cast<unsigned>(ctas_for(s, a.n_rows, BACK));
    const int threads = s.group * s.per_cta;
    const size_t smem =
        BACK && s.per_cta > 1 ? static_cast<size_t>(s.per_cta) * a.dim * sizeof(float) : 0;
#define ZF_NORM(E)                                                            \
    do {                                                                      \
        if constexpr (BACK)                                                   \
            norm_grad_kernel<T, VEC, E><<<g, threads, smem, stream>>>(a);     \
        else                                                                  \
            norm_kernel<T, VEC, E><<<g, threads, 0, stream>>>(a);             \
        return cudaGetLastError();                                            \
    } while (0)
    if (s.e == 8) ZF_NORM(8);
    if (s.e == 16) ZF_NORM(16);
    ZF_NORM(32);
#undef ZF_NORM
}

template <bool BACK>
cudaError_t dispatch(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    const bool wide = wide_rows(act_bytes, a.x, a.x_stride, a.dim) &&
                      wide_rows(act_bytes, a.out, a.out_stride, a.dim) &&
                      (!BACK || wide_rows(act_bytes, a.grad_out, a.grad_out_stride, a.dim));
    if (act_bytes == 4)
        return wide ? launch_shape<float, 4, BACK>(a, stream)
                    : launch_shape<float, 1, BACK>(a, stream);
    return wide ? launch_shape<uint16_t, 8, BACK>(a, stream)
                : launch_shape<uint16_t, 1, BACK>(a, stream);
}

}  // namespace

int norm_grad_ctas(int64_t n_rows, int64_t dim) {
    return static_cast<int>(ctas_for(shape_for(dim, true), n_rows, true));
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
