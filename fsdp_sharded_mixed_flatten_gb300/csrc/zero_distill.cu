// Distillation from a teacher's top logits.  For a row of student logits z
// over the vocabulary and the teacher's entries (id_k, l_k):
//   p = softmax(l / tau) over the entries,  q = softmax(z / tau) over the row,
//   loss = w tau^2 sum_k p_k (log p_k - log q_{id_k}),
//   dloss/dz_v = w tau (q_v - sum_{k: id_k = v} p_k).
//
// One pass over the row keeps each thread's running maximum m and the sum of
// exp((z - m) / tau), rescaled when the maximum grows; the gradient pass
// reads the row again, which by then is in L2, so that DRAM sees one read and
// one write of the logits.  Exponentials are 2^((z - m) c), c = log2(e) / tau:
// the difference is taken first, so that a row of the type's lowest values
// is a row of equal ones.
#include "zero_ops.cuh"

namespace zf {

namespace {

constexpr int kThreads_ = 512;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (z - m) c with the maximum of an all-masked part taken as 0, so that its
// terms are 2^-inf = 0 and not NaN.
__device__ __forceinline__ float finite_max(float m) { return m == -kInf ? 0.0f : m; }

struct Running {
    float m, s;
    __device__ __forceinline__ void add(const Running& o, float c) {
        const float top = fmaxf(m, o.m), t = finite_max(top);
        s = s * ex2((m - t) * c) + o.s * ex2((o.m - t) * c);
        m = top;
    }
};

template <int N>
__device__ __forceinline__ void accumulate(Running& r, const float (&x)[N], float c) {
    float top = r.m;
#pragma unroll
    for (int e = 0; e < N; ++e) top = fmaxf(top, x[e]);
    const float t = finite_max(top);
    float s = r.s * ex2((r.m - t) * c);
#pragma unroll
    for (int e = 0; e < N; ++e) s += ex2((x[e] - t) * c);
    r.s = s;
    r.m = top;
}

// A row from its first 16-byte boundary on; `head` single elements before.
template <class T>
struct RowSplit {
    static constexpr int kV = 16 / sizeof(T);
    int head;
    int64_t n_vec;
    __device__ RowSplit(const T* p, int64_t n, bool vec) {
        if (!vec) {
            head = 0;
            n_vec = 0;
            return;
        }
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16) / sizeof(T);
        head = mis == 0 ? 0 : kV - mis;
        if (head > n) head = static_cast<int>(n);
        n_vec = (n - head) / kV;
    }
    __device__ int64_t tail() const { return head + n_vec * kV; }
};

template <class T, bool GRAD>
__global__ void __launch_bounds__(kThreads_) distill_kernel(const __grid_constant__ DistillArgs a) {
    constexpr int kV = 16 / sizeof(T);
    constexpr int kWarps = kThreads_ / 32;
    extern __shared__ float dyn[];
    float* p_s = dyn;                                    // teacher probabilities
    float* z_s = dyn + a.top;                            // the student's logits there
    int32_t* id_s = reinterpret_cast<int32_t*>(dyn + 2 * a.top);
    __shared__ Running part[kWarps];
    __shared__ float terms[2];                           // sum p (log p - z / tau), any entry

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const float w = a.weights != nullptr ? a.weights[row] : 1.0f;
    const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
    T* dz = GRAD ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
    const bool vec = !GRAD || ((reinterpret_cast<uintptr_t>(z) ^
                                reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
    const RowSplit<T> split(z, a.vocab, vec);
    bool live = w != 0.0f;

    Running r{-kInf, 0.0f};
    if (live) {
        if (warp == 0) {
            const int32_t* ids = a.ids + row * a.top;
            const int64_t t0 = row * a.top;
            float best = -kInf;
            for (int k = lane; k < a.top; k += 32) {
                const int32_t id = ids[k];
                const bool in = id >= 0 && id < a.vocab;
                const float l = in ? ld_param(a.teacher, a.teacher_f32, t0 + k) * a.inv_tau : -kInf;
                id_s[k] = in ? id : -1;
                z_s[k] = in ? widen<T>(z[id]) : 0.0f;
                p_s[k] = l;
                best = fmaxf(best, l);
            }
            best = warp_max(best);
            const float t = finite_max(best);
            float sum = 0.0f;
            for (int k = lane; k < a.top; k += 32) sum += expf(p_s[k] - t);
            sum = warp_sum(sum);
            const float log_sum = logf(sum), inv = 1.0f / sum;
            float acc = 0.0f;
            for (int k = lane; k < a.top; k += 32) {
                const float l = p_s[k] - t;
                const float p = best == -kInf ? 0.0f : expf(l) * inv;
                if (p != 0.0f) acc += p * (l - log_sum);
                p_s[k] = p;
            }
            acc = warp_sum(acc);
            if (lane == 0) {
                terms[0] = acc;
                terms[1] = best == -kInf ? 0.0f : 1.0f;
            }
        }
        for (int64_t i = tid; i < split.n_vec; i += kThreads_) {
            const Pack<T, kV> v = ld_pack<T, kV>(z + split.head + i * kV);
            float x[kV];
#pragma unroll
            for (int e = 0; e < kV; ++e) x[e] = widen<T>(v.x[e]);
            accumulate(r, x, a.c);
        }
        for (int64_t i = tid; i < split.head; i += kThreads_) {
            const float x[1] = {widen<T>(z[i])};
            accumulate(r, x, a.c);
        }
        for (int64_t i = split.tail() + tid; i < a.vocab; i += kThreads_) {
            const float x[1] = {widen<T>(z[i])};
            accumulate(r, x, a.c);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Running other{__shfl_xor_sync(0xFFFFFFFFu, r.m, o),
                          __shfl_xor_sync(0xFFFFFFFFu, r.s, o)};
            r.add(other, a.c);
        }
        if (lane == 0) part[warp] = r;
    }
    __syncthreads();
    if (live) {
        live = terms[1] != 0.0f;
        r = part[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) r.add(part[i], a.c);
    }
    const float m = finite_max(r.m);
    if (warp == 0) {
        float loss = 0.0f;
        if (live) {
            // sum_k p_k (log p_k - (z_k - m) / tau) + log sum
            float acc = 0.0f;
            for (int k = lane; k < a.top; k += 32) {
                if (p_s[k] != 0.0f) acc += p_s[k] * (z_s[k] - m) * a.inv_tau;
            }
            acc = warp_sum(acc);
            loss = w * a.tau2 * (terms[0] - acc + logf(r.s));
        }
        if (lane == 0) a.loss[row] = loss;
    }
    if constexpr (GRAD) {
        const float f = live ? a.tau * w / r.s : 0.0f;
        for (int64_t i = tid; i < split.n_vec; i += kThreads_) {
            T* at = dz + split.head + i * kV;
            float y[kV];
            if (live) {
                const Pack<T, kV> v = ld_pack<T, kV>(z + split.head + i * kV);
#pragma unroll
                for (int e = 0; e < kV; ++e) y[e] = ex2((widen<T>(v.x[e]) - m) * a.c) * f;
            } else {
#pragma unroll
                for (int e = 0; e < kV; ++e) y[e] = 0.0f;
            }
            st_pack<T, kV>(at, pack<T, kV>(y));
        }
        for (int64_t i = tid; i < split.head; i += kThreads_) {
            dz[i] = narrow<T>(live ? ex2((widen<T>(z[i]) - m) * a.c) * f : 0.0f);
        }
        for (int64_t i = split.tail() + tid; i < a.vocab; i += kThreads_) {
            dz[i] = narrow<T>(live ? ex2((widen<T>(z[i]) - m) * a.c) * f : 0.0f);
        }
        __syncthreads();
        if (live) {
            // the teacher's entries: one warp each; equal ids add up in the
            // order of the entries, and the first of them writes
            for (int k = warp; k < a.top; k += kWarps) {
                const int32_t id = id_s[k];
                if (id < 0) continue;
                float p = 0.0f;
                bool earlier = false;
                for (int j = lane; j < a.top; j += 32) {
                    if (id_s[j] == id) {
                        p += p_s[j];
                        earlier |= j < k;
                    }
                }
                p = warp_sum(p);
                if (__any_sync(0xFFFFFFFFu, earlier)) continue;
                if (lane == 0) {
                    const float q = ex2((z_s[k] - m) * a.c) / r.s;
                    dz[id] = narrow<T>(a.tau * w * (q - p));
                }
            }
        }
    }
}

template <class T>
cudaError_t launch(const DistillArgs& a, cudaStream_t stream) {
    const size_t smem = 3 * sizeof(float) * static_cast<size_t>(a.top);
    const unsigned grid = static_cast<unsigned>(a.n_rows);
    if (a.grad != nullptr) {
        distill_kernel<T, true><<<grid, kThreads_, smem, stream>>>(a);
    } else {
        distill_kernel<T, false><<<grid, kThreads_, smem, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int logits_bytes, cudaStream_t stream) {
    return logits_bytes == 4 ? launch<float>(a, stream) : launch<uint16_t>(a, stream);
}

}  // namespace zf
