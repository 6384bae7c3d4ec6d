// Layer norm over rows of `dim` values:
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r,
//   y = xh w + b,
// and its backward pass for g = dy w:
//   dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// A row lives in the registers of a group of threads, E elements each, so that
// every byte of x, dy and the output crosses memory once.  A CTA holds several
// groups, which work through the rows independently; the next row's loads are
// under way while a row is worked on.  The parameters stay in registers or, to
// leave room for more warps, in shared memory (each thread its own columns: no
// barrier), and the backward pass's columns of dw and db in registers over all
// rows; each CTA writes one pair of partial rows, which a second launch adds up
// in CTA order.
//
// The variance is taken about a mean at every step: a warp's squares about the
// warp's mean, then sum (M2_w + n_w (mean_w - mu)^2) over the warps of the
// row, so that a mean far from zero costs no digits and one exchange is enough.
#include "zero_ops.cuh"

#include <mutex>

namespace zf {

namespace {

constexpr int kNormThreads = 512;      // of a CTA, at most
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kGradThreads = 384;      // of the backward pass at E = 8, two CTAs an SM

// Rows worked on at a time.
__host__ __device__ constexpr int batch_of(int) { return 1; }

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

// This thread's columns: pack n holds columns n * group * VEC + t * VEC ..., of
// which the first left[n] exist.
template <int VEC, int E>
struct Columns {
    static constexpr int N = E / VEC;
    int first, step;
    int left[N];
    __device__ Columns(const Group& g, int dim) : first(g.t * VEC), step(g.threads * VEC) {
#pragma unroll
        for (int n = 0; n < N; ++n) left[n] = min(max(dim - at(n), 0), VEC);
    }
    __device__ __forceinline__ int at(int n) const { return first + n * step; }
    __device__ __forceinline__ bool ok(int n, int e) const { return e < left[n]; }
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
            if (in && c.left[n] == VEC) p[n] = ld_pack<T, VEC>(at + n * c.step);
            if constexpr (VEC > 1) {
                if (in && c.left[n] > 0 && c.left[n] < VEC) {     // the row's last elements
#pragma unroll
                    for (int e = 0; e < VEC - 1; ++e) {
                        if (e < c.left[n]) p[n].x[e] = at[n * c.step + e];
                    }
                }
            }
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
        if (c.left[n] == 0) continue;
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
        if (c.left[n] == VEC) {
            st_pack<T, VEC>(at + n * c.step, v);
        } else if constexpr (VEC > 1) {
#pragma unroll
            for (int e = 0; e < VEC - 1; ++e) {
                if (e < c.left[n]) at[n * c.step + e] = v.x[e];
            }
        }
    }
}

// The parameters of this thread's columns (`missing` where there is no array
// or no column).  Loads without conditions, at a clamped place, so that all are
// under way at once.
template <class PT, int VEC, int E>
__device__ __forceinline__ void ld_params_as(float (&v)[E], const void* p, int dim,
                                             const Columns<VEC, E>& c) {
    PT raw[E];
#pragma unroll
    for (int i = 0; i < E; ++i)
        raw[i] = static_cast<const PT*>(p)[min(c.at(i / VEC) + i % VEC, dim - 1)];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = widen<PT>(raw[i]);
}

template <int VEC, int E>
__device__ __forceinline__ void ld_params(Pair (&w)[E / 2], const void* p, const NormArgs& a,
                                          const Columns<VEC, E>& c, float missing) {
    float v[E];
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = missing;
    } else if (a.param_f32) {
        ld_params_as<float>(v, p, a.dim, c);
    } else {
        ld_params_as<uint16_t>(v, p, a.dim, c);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = c.ok(i / VEC, i % VEC) ? v[i] : missing;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = pair(v[2 * i], v[2 * i + 1]);
}

// Pairs of this thread's columns in shared memory, 16 bytes a thread at a time.
template <int E>
struct Kept {
    ulonglong2* at;
    int step;
    __device__ Kept(void* base, int array)
        : at(static_cast<ulonglong2*>(base) + array * (E / 4) * blockDim.x + threadIdx.x),
          step(blockDim.x) {}
    __device__ __forceinline__ void put(const Pair (&w)[E / 2]) const {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) at[i * step] = make_ulonglong2(w[2 * i], w[2 * i + 1]);
    }
    __device__ __forceinline__ ulonglong2 operator[](int i) const { return at[i * step]; }
};

__device__ __forceinline__ float both(Pair p) {
    const float2 v = unpair(p);
    return v.x + v.y;
}

__device__ __forceinline__ Pair splat(float x) { return pair(x, x); }

// 1 / sqrt(x): the approximation and one Newton step.
__device__ __forceinline__ float inv_sqrt(float x) {
    const float y = rsqrtf(x);
    const float z = y * __fmaf_rn(-0.5f * x * y, y, 1.5f);
    return y == __builtin_huge_valf() ? y : z;
}

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
__global__ void __launch_bounds__(kNormThreads, E == 32 ? 1 : 2)
norm_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) char params[];           // weight, bias
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
    const Kept<E> w(params, 0), b(params, 1);
    {
        Pair v[P];
        ld_params<VEC, E>(v, a.weight, a, c, 1.0f);
        w.put(v);
        ld_params<VEC, E>(v, a.bias, a, c, 0.0f);
        b.put(v);
    }
    const bool ragged = a.dim % VEC != 0;
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
                if (VEC == 1 || ragged) {
                    const float2 f = unpair(d);
                    d = pair(c.ok(2 * j / VEC, 2 * j % VEC) ? f.x : 0.0f,
                             c.ok((2 * j + 1) / VEC, (2 * j + 1) % VEC) ? f.y : 0.0f);
                } else {
                    d = c.left[2 * j / VEC] != 0 ? d : 0;
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
            const float r = inv_sqrt(__fmaf_rn(s[i].y, inv_d, a.eps));
            if (g.t == 0) {
                if (a.mean != nullptr) a.mean[row + i] = mu;
                if (a.rstd != nullptr) a.rstd[row + i] = r;
            }
            const Pair m2 = splat(-mu), r2 = splat(r);
#pragma unroll
            for (int j = 0; j < P / 2; ++j) {
                const ulonglong2 wj = w[j], bj = b[j];
                Pair *y0 = &v[i][2 * j], *y1 = &v[i][2 * j + 1];
                *y0 = fma2(mul2(add2(*y0, m2), r2), wj.x, bj.x);
                *y1 = fma2(mul2(add2(*y1, m2), r2), wj.y, bj.y);
            }
            store_row<T, VEC, E>(out + i * a.out_stride, v[i], c);
        }
    }
}

template <class T, int VEC, int E>
__global__ void __launch_bounds__(E == 8 ? kGradThreads : kNormThreads, E == 8 ? 2 : 1)
norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kBatch = 1, P = E / 2;
    constexpr bool kKeep = E > 8;            // the weight in shared memory
    extern __shared__ __align__(16) char dyn[];
    float* cols = reinterpret_cast<float*>(dyn);     // [groups][dim] where a CTA has several;
                                                     // before, the weight
    __shared__ float2 red[2][kBatch][kNormWarps];
    int half = 0;
    const Group g(a.group_threads);
    const Columns<VEC, E> c(g, a.dim);
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    Pair w[P], dw[P], db[P];
    ld_params<VEC, E>(w, a.weight, a, c, 1.0f);
    const Kept<E> kept(dyn, 0);
    if (kKeep) kept.put(w);
#pragma unroll
    for (int j = 0; j < P; ++j) dw[j] = db[j] = 0;
    // the reduction's launch may be set up from now on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
                Pair wj = w[j];
                if (kKeep) wj = j % 2 == 0 ? kept[j / 2].x : kept[j / 2].y;
                xh[i][j] = mul2(add2(next_x[i][j], m2), r2);
                gr[i][j] = mul2(d, wj);
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
            if (c.ok(n0, 2 * j % VEC)) to[c.at(n0) + 2 * j % VEC] = f.x;
            if (c.ok(n1, (2 * j + 1) % VEC)) to[c.at(n1) + (2 * j + 1) % VEC] = f.y;
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
    asm volatile("griddepcontrol.wait;" ::: "memory");       // the partial rows are there
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
    int per_cta = (back && e == 8 ? kGradThreads : kNormThreads) / group;
    if (per_cta > 8) per_cta = 8;               // 16 hardware barriers a CTA
    return {e, group, per_cta};
}

// CTAs: what the registers of an SM hold (launch bounds), or what the rows need.
int64_t ctas_for(const Shape& s, int64_t rows, bool back) {
    const int threads = s.group * s.per_cta;
    const int per_sm = back ? (s.e == 8 ? 2 * kGradThreads / threads : 1)
                            : (s.e == 32 ? 1 : 2 * kNormThreads / threads);
    const int64_t per = static_cast<int64_t>(s.per_cta) * (back ? 1 : batch_of(s.e));
    const int64_t need = rows > 0 ? (rows + per - 1) / per : 1;
    const int64_t most = static_cast<int64_t>(device_sms()) * per_sm;
    return need < most ? need : most;
}

// Whether every row of a matrix starts on a 16-byte boundary.
bool wide_rows(int elem, const void* p, int64_t stride) {
    return aligned_to(p, 16) && stride % (16 / elem) == 0;
}

template <class T, int VEC, int E, bool BACK>
cudaError_t launch_e(const NormArgs& a, unsigned grid, int threads, size_t smem,
                     cudaStream_t stream) {
    const auto kernel = BACK ? norm_grad_kernel<T, VEC, E> : norm_kernel<T, VEC, E>;
    // more than 48 KB of shared memory need asking for
    static std::once_flag once[64];
    static cudaError_t set[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        2 * sizeof(float) * E * kNormThreads);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    kernel<<<grid, threads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <class T, int VEC, bool BACK>
cudaError_t launch_shape(NormArgs a, cudaStream_t stream) {
    const Shape s = shape_for(a.dim, BACK);
    a.group_threads = s.group;
    const unsigned g = static_cast<unsigned>(ctas_for(s, a.n_rows, BACK));
    const int threads = s.group * s.per_cta;
    size_t smem = 0;
    if (BACK) {
        const size_t kept = s.e > 8 ? sizeof(float) * s.e * threads : 0;
        const size_t cols = s.per_cta > 1 ? sizeof(float) * s.per_cta * a.dim : 0;
        smem = kept > cols ? kept : cols;
    } else {
        smem = 2 * sizeof(float) * s.e * threads;
    }
    if (s.e == 8) return launch_e<T, VEC, 8, BACK>(a, g, threads, smem, stream);
    if (s.e == 16) return launch_e<T, VEC, 16, BACK>(a, g, threads, smem, stream);
    return launch_e<T, VEC, 32, BACK>(a, g, threads, smem, stream);
}

template <bool BACK>
cudaError_t dispatch(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    const bool wide = wide_rows(act_bytes, a.x, a.x_stride) &&
                      wide_rows(act_bytes, a.out, a.out_stride) &&
                      (!BACK || wide_rows(act_bytes, a.grad_out, a.grad_out_stride));
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
    // its blocks may be set up while the partial rows are still being added up
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((width + 31) / 32));
    cfg.blockDim = dim3(32 * kStrands);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_grad_reduce_kernel, a, norm_grad_ctas(a.n_rows, a.dim));
}

}  // namespace zf
