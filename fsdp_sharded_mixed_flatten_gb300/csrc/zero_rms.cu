// Root-mean-square norm over rows of `dim` values, with the residual's addition:
//   s = x + res,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w,
// and its backward pass for xh = s r, g = dy w, dt the gradient that reaches s past the
// norm:
//   dx = dt + r (g - xh mean(g xh)),  dw = sum_rows dy xh.
// y and s may be written in 8 bits (zero_eight.cuh), and the backward pass reads s from
// them, so that a training step keeps a byte an element of it.
//
// A row lives in the registers of a group of threads, 8 K elements each; a CTA holds
// several groups, which work through the rows independently, the next rows' loads under
// way while a row is worked on: into rings in shared memory (rms_rows_kernel,
// rms_rows_grad_kernel), or, for what those do not take, straight to registers.  The
// backward pass keeps its columns of dw in registers over all rows; each CTA writes one
// partial row, which a second launch adds up in CTA order.
//
// Bound by memory where rows are many: 16384 x 4096 bf16 with residual 85 us (6.3 TB/s), with
// the sum in 8 bits 99 us; backward of 8192 x 4096 49 us (5.5 TB/s, 5 us of it the second
// launch), of 16384 x 4096 from 8 bits with the output once more 102 us (5.9 TB/s); 16384 x
// 14336 bf16 packed and unpacked 207 us (6.9 TB/s).  Few rows take as long as the host's call
// (4 x 4096: 9 us).
#include "zero_eight.cuh"

#include <mutex>

#include "zero_kernels.cuh"
#include "zero_ops.cuh"
#include "zero_status.cuh"
#include "zero_tile.cuh"

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

// 1 / sqrt(mean(s^2) + eps) of a row whose squares this thread has added up to q.  Where the
// row's sum leaves fp32 (values of 1e17 and more), it is made once more of values times 2^-72:
// the largest, 2^128, then have squares of 2^112 and 16384 of them a sum that fp32 holds, and
// what is small beside them counts for nothing.
template <int K>
__device__ __forceinline__ float row_rstd(const RmsGroup& g, const float (&s)[K][8], float q,
                                          float inv_d, float eps, float (*red)[kRmsWarps],
                                          int& half) {
    float r = inv_sqrt(__fmaf_rn(rms_group_sum(g, q, red, half), inv_d, eps));
    if (__builtin_expect(r == 0.0f, 0)) {
        constexpr float kBy = 0x1p-72f;
        q = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) q = __fmaf_rn(s[k][e] * kBy, s[k][e] * kBy, q);
        }
        q = rms_group_sum(g, q, red, half);
        r = inv_sqrt(__fmaf_rn(q, inv_d, eps * kBy * kBy)) * kBy;
    }
    return r;
}

template <class T, int K, bool WIDE>
__global__ void __launch_bounds__(512, K == 1 ? 2 : 1)
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
    constexpr bool kHeld = K <= 2;           // the weight in registers
    float held[kHeld ? K : 1][8];
    if constexpr (kHeld) {
#pragma unroll
        for (int k = 0; k < K; ++k) c.params(held[k], a.weight, a.param_f32, k);
    }
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
        const float r = row_rstd(g, s, q, inv_d, a.eps, red, half);
        if (g.t == 0 && a.rstd != nullptr) a.rstd[row] = r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[8];
            if constexpr (!kHeld) c.params(w, a.weight, a.param_f32, k);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = s[k][e] * r * (kHeld ? held[kHeld ? k : 0][e] : w[e]);
            if (a.out != nullptr)
                c.template store<T>(static_cast<T*>(a.out) + row * a.out_stride, k, w);
            if (a.out8 != nullptr)
                c.store_eight(a.out8 + row * a.out8_stride, a.out8_scales + row * a.blocks, k, w);
        }
    }
}

// The backward pass of rows of which shared memory holds less than two: from 8225 columns on,
// of fp32 (with s in 8 bits from 10465 on), of bf16 with an fp32 weight from 14393 on.
// EIGHT: s comes in 8 bits.
constexpr int kWideOctets = 4;
template <class T, bool WIDE, bool EIGHT>
__global__ void __launch_bounds__(512, 1)
rms_norm_grad_kernel(const __grid_constant__ RmsArgs a) {
    constexpr int K = kWideOctets;
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

// The same through shared memory: every group has a ring of slots, one row's arrays each,
// that its first thread fills by bulk copies, so that several rows a group are on their way
// whatever the registers hold.  A slot is filled again when the group's next exchange shows
// that all have done with it.
//
// Threads of a CTA at most: more where a thread has one octet and few registers (forward of
// 8192 rows of bf16: 768 columns 15.1 us, by 512 threads 16.7; 2048 28.0 / 32.0; but 16384 x
// 1024 fp32 55.7 / 48.6).
__host__ __device__ constexpr int rows_threads(int k, int elem, bool back) {
    return k == 1 && elem == 2 && !back ? 768 : 512;
}
constexpr uint64_t kRowsWaitNs = 2000000000ull;

struct RowsRing {
    char* base;
    uint32_t slot_bytes, bars;
    int slots, at;
    uint32_t phase;
    int* stop;
    int* status;
    __device__ __forceinline__ const char* here() const { return base + at * slot_bytes; }
    __device__ __forceinline__ uint32_t bar(int s) const { return bars + 8 * s; }
    // The slot's row has come.  When a wait runs out the launch goes on with what is there
    // (no group is left waiting for a part of itself) and the status tells.
    __device__ __forceinline__ void wait() const {
        const uint32_t b = bar(at);
        if (!tile::bar_try(b, phase)) tile::bar_wait(b, phase, stop, status, kRowsWaitNs);
    }
    __device__ __forceinline__ void next() {
        if (++at == slots) {
            at = 0;
            phase ^= 1;
        }
    }
};

template <class T>
__device__ __forceinline__ Octet<T> octet_at(const char* p) {
    return *reinterpret_cast<const Octet<T>*>(p);
}

// A row's array in a slot: the aligned words that hold it, which start up to 15 bytes before
// (WIDE: rows on the 16-byte grid, of whole octets).
template <bool WIDE, class T>
__device__ __forceinline__ uint32_t row_bytes(const T* row, int dim) {
    const int bytes = dim * static_cast<int>(sizeof(T));
    return WIDE ? bytes : (off_16(row) + bytes + 15) / 16 * 16;
}
// ... of an array of rows at most
__host__ __device__ constexpr int64_t row_room(int64_t dim, int64_t elem, bool wide) {
    return wide ? dim * elem : (dim * elem + 15) / 16 * 16 + 16;
}
template <bool WIDE, class T>
__device__ __forceinline__ void fetch_row(uint32_t to, const T* row, int dim, uint32_t bar) {
    tile::bulk_load(to, reinterpret_cast<const char*>(row) - (WIDE ? 0 : off_16(row)),
                    row_bytes<WIDE>(row, dim), bar);
}
// This thread's values of octet k of it; zeros where there are no columns, but for WIDE,
// where those are some of the row's.
template <class T, bool WIDE, int K>
__device__ __forceinline__ Octet<T> octet_of(const char* array, int mis, const Octets<WIDE, K>& c,
                                             int k) {
    if constexpr (WIDE) {
        return octet_at<T>(array + (c.at(k, 0) < c.dim ? c.at(k, 0) : 0) * sizeof(T));
    } else {
        Octet<T> v{};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c.ok(k, e)) v.x[e] = reinterpret_cast<const T*>(array + mis)[c.at(k, e)];
        }
        return v;
    }
}

// The weight: this thread's octets in registers, or, where there are four of them, all of
// it in shared memory as it is.
template <bool WIDE, int K>
struct Weight {
    float held[K <= 2 ? K : 1][8];
    const char* at;
    bool f32;
    __device__ __forceinline__ void octet(float (&w)[8], int k, const Octets<WIDE, K>& c) const {
        const int column = WIDE && c.at(k, 0) < c.dim ? c.at(k, 0) : 0;
        if constexpr (K <= 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = held[k][e];
        } else if constexpr (!WIDE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = c.ok(k, e) ? ld_param(at, f32, c.at(k, e)) : 1.0f;
        } else if (f32) {
            const Octet<float> v = octet_at<float>(at + 4 * column);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = v.x[e];
        } else {
            const Octet<uint16_t> v = octet_at<uint16_t>(at + 2 * column);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = widen<uint16_t>(v.x[e]);
        }
    }
};

// Bytes of shared memory a column for it.
__host__ __device__ constexpr int weight_bytes(int k, bool f32) { return k <= 2 ? 0 : f32 ? 4 : 2; }

// Sets up the CTA's rings, and the weight after them.
template <bool WIDE, int K>
__device__ __forceinline__ RowsRing rows_begin(const RmsArgs& a, const RmsGroup& g,
                                               const Octets<WIDE, K>& c, char* dyn,
                                               Weight<WIDE, K>& weight, int* stop) {
    RowsRing r;
    r.slots = a.slots;
    r.slot_bytes = a.slot_bytes;
    r.base = dyn + g.index * a.slots * a.slot_bytes;
    char* after = dyn + g.per_cta * a.slots * a.slot_bytes;
    weight.at = after;
    weight.f32 = a.weight != nullptr && a.param_f32;
    const int padded = (a.dim + 7) / 8 * 8;
    r.bars = tile::smem_address(after + weight_bytes(K, weight.f32) * padded) + g.index * a.slots * 8;
    r.at = 0;
    r.phase = 0;
    r.stop = stop;
    r.status = a.status;
    if (threadIdx.x == 0) *stop = 0;
    if (g.t == 0) {
        for (int s = 0; s < r.slots; ++s) tile::bar_init(r.bar(s), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if constexpr (K <= 2) {
#pragma unroll
        for (int k = 0; k < K; ++k) c.params(weight.held[k], a.weight, a.param_f32, k);
    } else {
        for (int i = threadIdx.x; i < a.dim; i += blockDim.x) {
            if (weight.f32)
                reinterpret_cast<float*>(after)[i] = static_cast<const float*>(a.weight)[i];
            else
                reinterpret_cast<uint16_t*>(after)[i] =
                    a.weight == nullptr ? 0x3F80 : static_cast<const uint16_t*>(a.weight)[i];
        }
    }
    __syncthreads();
    return r;
}

__device__ __forceinline__ void rows_end(const int* stop) {
    if (*static_cast<const volatile int*>(stop)) {         // copies under way get time to come
        const uint64_t t0 = tile::now_ns();
        while (tile::now_ns() - t0 < 20000000ull) {}
    }
}

// (Rows off the 16-byte grid go straight to registers: 8192 x 4001 bf16 60 us, through shared
// memory by single elements 62, with the sum in 8 bits 79 / 88.)
template <class T, int K>
__global__ void __launch_bounds__(rows_threads(K, sizeof(T), false), 1)
rms_rows_kernel(const __grid_constant__ RmsArgs a) {
    extern __shared__ __align__(128) char dyn[];
    __shared__ float red[2][kRmsWarps];
    __shared__ int stop;
    int half = 0;
    const RmsGroup g(a.group_threads);
    const Octets<true, K> c(g.t, g.threads, a.dim);
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    Weight<true, K> weight;
    RowsRing ring = rows_begin(a, g, c, dyn, weight, &stop);
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index;
    const uint32_t second = row_room(a.dim, sizeof(T), true);
    auto x_row = [&](int64_t at) { return static_cast<const T*>(a.x) + at * a.x_stride; };
    auto residual_row = [&](int64_t at) {
        return static_cast<const T*>(a.residual) + at * a.residual_stride;
    };
    auto fill = [&](int64_t at, int s) {
        if (at >= a.n_rows) return;
        const uint32_t to = tile::smem_address(ring.base + s * ring.slot_bytes), bar = ring.bar(s);
        const bool two = a.residual != nullptr;
        tile::bar_expect(bar, row_bytes<true>(x_row(at), a.dim) +
                                  (two ? row_bytes<true>(residual_row(at), a.dim) : 0));
        fetch_row<true>(to, x_row(at), a.dim, bar);
        if (two) fetch_row<true>(to + second, residual_row(at), a.dim, bar);
    };
    if (g.t == 0) {
        for (int s = 0; s < ring.slots; ++s) fill(row + s * step, s);
    }
    for (; row < a.n_rows; row += step) {
        ring.wait();
        const char* from = ring.here();
        float s[K][8];
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Octet<T> x = octet_of<T>(from, 0, c, k);
            if (a.residual != nullptr) {
                const Octet<T> r = octet_of<T>(from + second, 0, c, k);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[k][e] = __fadd_rn(widen<T>(x.x[e]), widen<T>(r.x[e]));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) s[k][e] = widen<T>(x.x[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c.at(k, 0) >= a.dim) s[k][e] = 0.0f;
                q = __fmaf_rn(s[k][e], s[k][e], q);
            }
        }
        const float r = row_rstd(g, s, q, inv_d, a.eps, red, half);
        if (g.t == 0) {
            fill(row + ring.slots * step, ring.at);
            if (a.rstd != nullptr) a.rstd[row] = r;
        }
        ring.next();
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
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[8], y[8];
            weight.octet(w, k, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = s[k][e] * r * w[e];
            if (a.out != nullptr)
                c.template store<T>(static_cast<T*>(a.out) + row * a.out_stride, k, y);
            if (a.out8 != nullptr)
                c.store_eight(a.out8 + row * a.out8_stride, a.out8_scales + row * a.blocks, k, y);
        }
    }
    __syncthreads();
    rows_end(&stop);
}

template <class T, int K, bool WIDE, bool EIGHT>
__global__ void __launch_bounds__(rows_threads(K, sizeof(T), true), 1)
rms_rows_grad_kernel(const __grid_constant__ RmsArgs a) {
    // a row's values stay in registers as they come; four octets of them do not fit (held
    // all the same, 8192 x 8192 bf16 162 us, read twice 116) and are read from the slot
    // twice, which is filled again a row later
    constexpr bool kHeld = K <= 2;
    extern __shared__ __align__(128) char dyn[];
    __shared__ float red[2][kRmsWarps];
    __shared__ int stop;
    int half = 0;
    const RmsGroup g(a.group_threads);
    const Octets<WIDE, K> c(g.t, g.threads, a.dim);
    const float inv_d = 1.0f / static_cast<float>(a.dim);
    Weight<WIDE, K> weight;
    RowsRing ring = rows_begin(a, g, c, dyn, weight, &stop);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index;
    const uint32_t first = row_room(a.dim, EIGHT ? 1 : sizeof(T), WIDE);
    const uint32_t second = first + row_room(a.dim, sizeof(T), WIDE);
    auto x_row = [&](int64_t at) { return static_cast<const T*>(a.x) + at * a.x_stride; };
    auto codes_row = [&](int64_t at) { return a.total8 + at * a.total8_stride; };
    auto dy_row = [&](int64_t at) {
        return static_cast<const T*>(a.grad_out) + at * a.grad_out_stride;
    };
    auto dt_row = [&](int64_t at) {
        return static_cast<const T*>(a.grad_total) + at * a.grad_total_stride;
    };
    auto fill = [&](int64_t at, int s) {
        if (at >= a.n_rows) return;
        const uint32_t to = tile::smem_address(ring.base + s * ring.slot_bytes), bar = ring.bar(s);
        const bool dt = a.grad_total != nullptr;
        uint32_t bytes =
            row_bytes<WIDE>(dy_row(at), a.dim) + (dt ? row_bytes<WIDE>(dt_row(at), a.dim) : 0);
        if constexpr (EIGHT) bytes += row_bytes<WIDE>(codes_row(at), a.dim);
        else bytes += row_bytes<WIDE>(x_row(at), a.dim);
        tile::bar_expect(bar, bytes);
        if constexpr (EIGHT) fetch_row<WIDE>(to, codes_row(at), a.dim, bar);
        else fetch_row<WIDE>(to, x_row(at), a.dim, bar);
        fetch_row<WIDE>(to + first, dy_row(at), a.dim, bar);
        if (dt) fetch_row<WIDE>(to + second, dt_row(at), a.dim, bar);
    };
    if (g.t == 0) {
        for (int s = 0; s < ring.slots; ++s) fill(row + s * step, s);
    }
    float dw[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[k][e] = 0.0f;
    }
    constexpr int kScales = WIDE ? 1 : 2;
    float next_r = 0.0f, scale[K][kScales], next_scale[K][kScales];
    auto load_small = [&](int64_t at) {
        if (at >= a.n_rows) return;
        next_r = a.rstd[at];
        if constexpr (EIGHT) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int b = 0; b < kScales; ++b) {
                    // (the other mapping's octets are of two blocks)
                    const int col = c.at(k, 4 * b);
                    next_scale[k][b] =
                        col < a.dim ? a.total8_scales[at * a.blocks + col / kEightBlock] : 0.0f;
                }
            }
        }
    };
    load_small(row);
    int64_t before = -1;                       // the row before, whose slot is to be filled
    for (; row < a.n_rows; row += step) {
        ring.wait();
        const char* from = ring.here();
        const float r = next_r;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int b = 0; b < kScales; ++b) scale[k][b] = next_scale[k][b];
        }
        load_small(row + step);
        struct Raw {
            Octet<T> x, dy, dt;
            uint2 codes;
        } raw[kHeld ? K : 1];
        const int x_mis = WIDE ? 0 : EIGHT ? off_16(codes_row(row)) : off_16(x_row(row));
        const int dy_mis = WIDE ? 0 : off_16(dy_row(row));
        const int dt_mis = WIDE || a.grad_total == nullptr ? 0 : off_16(dt_row(row));
        auto fetch = [&](Raw& v, int k, bool with_dt) {
            if constexpr (!EIGHT) {
                v.x = octet_of<T>(from, x_mis, c, k);
            } else if constexpr (WIDE) {
                v.codes = *reinterpret_cast<const uint2*>(from + (c.at(k, 0) < a.dim ? c.at(k, 0) : 0));
            } else {
                const Octet<uint8_t> q = octet_of<uint8_t>(from, x_mis, c, k);
                v.codes = *reinterpret_cast<const uint2*>(&q);
            }
            v.dy = octet_of<T>(from + first, dy_mis, c, k);
            if (with_dt && a.grad_total != nullptr)
                v.dt = octet_of<T>(from + second, dt_mis, c, k);
        };
        // xh, dy (0 where there are no columns) and the weight
        auto open = [&](const Raw& v, int k, float (&xh)[8], float (&d)[8], float (&w)[8]) {
            if constexpr (EIGHT) {
                values_of(xh, v.codes, 1.0f);
#pragma unroll
                for (int e = 0; e < 8; ++e) xh[e] *= scale[k][WIDE ? 0 : e / 4] * r;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) xh[e] = widen<T>(v.x.x[e]) * r;
            }
            weight.octet(w, k, c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d[e] = !WIDE || c.at(k, 0) < a.dim ? widen<T>(v.dy.x[e]) : 0.0f;
        };
        float q = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Raw& v = raw[kHeld ? k : 0];
            fetch(v, k, kHeld);
            float xh[8], d[8], w[8];
            open(v, k, xh, d, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[k][e] = __fmaf_rn(d[e], xh[e], dw[k][e]);
                q = __fmaf_rn(d[e] * w[e], xh[e], q);
            }
        }
        const float m = -rms_group_sum(g, q, red, half) * inv_d;
        if (g.t == 0) {
            if constexpr (kHeld) {
                fill(row + ring.slots * step, ring.at);
            } else if (before >= 0) {
                fill(before + ring.slots * step, ring.at == 0 ? ring.slots - 1 : ring.at - 1);
            }
        }
        before = row;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Raw& v = raw[kHeld ? k : 0];
            if constexpr (!kHeld) fetch(v, k, true);
            float xh[8], d[8], w[8], y[8];
            open(v, k, xh, d, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r * __fmaf_rn(xh[e], m, d[e] * w[e]);
            if (a.grad_total != nullptr) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += widen<T>(v.dt.x[e]);
            }
            c.template store<T>(static_cast<T*>(a.grad_x) + row * a.grad_x_stride, k, y);
            if (a.out != nullptr) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = xh[e] * w[e];
                c.template store<T>(static_cast<T*>(a.out) + row * a.out_stride, k, y);
            }
        }
        ring.next();
    }
    __syncthreads();                           // the rings and the weight have been used up
    rows_end(&stop);
    if (a.grad_weight == nullptr) return;
    float* cols = reinterpret_cast<float*>(dyn);         // [groups][dim]
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (WIDE && c.at(k, 0) < a.dim) {
            float4* to = reinterpret_cast<float4*>(cols + g.index * a.dim + c.at(k, 0));
            to[0] = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
            to[1] = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
        } else if (!WIDE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c.ok(k, e)) cols[g.index * a.dim + c.at(k, e)] = dw[k][e];
            }
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
constexpr int kPackOctets = 4, kUnpackOctets = 2;

template <class T, bool WIDE>
__global__ void __launch_bounds__(32 * kEightWarps)
pack_kernel(const __grid_constant__ EightArgs a) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kEightWarps + threadIdx.x / 32;
    const int64_t row = id / a.sections;
    if (row >= a.n_rows) return;
    const int64_t first = (id - row * a.sections) * a.section;
    const int64_t rest = a.dim - first;
    // rows off the 16-byte grid: bf16 by shifted words (8192 x 4001 42 us, by single elements
    // 55), fp32 by single elements (5003 x 1501 13.9 us, by shifted words 15.5)
    constexpr bool kShift = !WIDE && sizeof(T) == 2;
    const Octets<WIDE || kShift, kPackOctets> c(threadIdx.x % 32, 32,
                                       static_cast<int>(rest < a.section ? rest : a.section));
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + first;
    Octet<T> v[kPackOctets];
#pragma unroll
    for (int k = 0; k < kPackOctets; ++k) {
        if constexpr (kShift) v[k] = c.template load_any<T>(x, k);
        else v[k] = c.template load<T>(x, k);
    }
#pragma unroll
    for (int k = 0; k < kPackOctets; ++k) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = widen<T>(v[k].x[e]);
        uint8_t* const codes = a.codes + row * a.codes_stride + first;
        float* const scales = a.scales + row * a.blocks + first / kEightBlock;
        if constexpr (kShift) c.store_eight_any(codes, scales, k, f);
        else c.store_eight(codes, scales, k, f);
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
    const Octets<WIDE, kUnpackOctets> c(threadIdx.x % 32, 32,
                                       static_cast<int>(rest < a.section ? rest : a.section));
    float f[kUnpackOctets][8];
#pragma unroll
    for (int k = 0; k < kUnpackOctets; ++k)
        c.load_eight(f[k], a.codes + row * a.codes_stride + first,
                     a.scales + row * a.blocks + first / kEightBlock, k);
#pragma unroll
    for (int k = 0; k < kUnpackOctets; ++k)
        c.template store<T>(static_cast<T*>(a.out) + row * a.x_stride + first, k, f[k]);
}

// The same with 16 columns a lane, by 32-byte words: a block of 128 is 8 lanes.
constexpr int kWideUnits = 2;              // times 512 columns a warp
struct alignas(32) Words {
    uint32_t w[8];
};
__device__ __forceinline__ Words ld_words(const void* p) {
    Words v;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]),
                   "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void st_words(void* p, const Words& v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]),
                 "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
                 "r"(v.w[7])
                 : "memory");
}

template <class T, int U>
__global__ void __launch_bounds__(32 * kEightWarps)
pack_wide_kernel(const __grid_constant__ EightArgs a) {
    constexpr int W = sizeof(T) / 2;                     // 32-byte words of 16 values
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kEightWarps + threadIdx.x / 32;
    const int64_t row = id / a.sections;
    if (row >= a.n_rows) return;
    const int first = static_cast<int>((id - row * a.sections) * a.section) + threadIdx.x % 32 * 16;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    Words v[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = first + 512 * u;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            v[u][w] = Words{};
            if (c < a.dim) v[u][w] = ld_words(x + c + 8 * w);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = first + 512 * u;
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if constexpr (W == 1)
                y[e] = __uint_as_float(e % 2 == 0 ? v[u][0].w[e / 2] << 16
                                                  : v[u][0].w[e / 2] & 0xFFFF0000u);
            else
                y[e] = __uint_as_float(v[u][e / 8].w[e % 8]);
        }
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(y[e]));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        uint32_t s = eight_exponent(m), q[4];
        if (__any_sync(0xFFFFFFFFu, s >= kEightTop)) {
            m = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) m = fmaxf(m, finite_magnitude(y[e]));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            s = eight_exponent(m);
            const float inverse = __uint_as_float((254 - s) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = eight_codes_rare(y[4 * i], y[4 * i + 1], inverse, s == kEightTop) |
                       eight_codes_rare(y[4 * i + 2], y[4 * i + 3], inverse, s == kEightTop) << 16;
        } else {
            const float inverse = __uint_as_float((254 - s) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = eight_codes(y[4 * i], y[4 * i + 1], inverse) |
                       eight_codes(y[4 * i + 2], y[4 * i + 3], inverse) << 16;
        }
        if (c < a.dim) {
            *reinterpret_cast<uint4*>(a.codes + row * a.codes_stride + c) =
                make_uint4(q[0], q[1], q[2], q[3]);
            if (c % kEightBlock == 0)
                a.scales[row * a.blocks + c / kEightBlock] = __uint_as_float(s << 23);
        }
    }
}

template <class T, int U>
__global__ void __launch_bounds__(32 * kEightWarps)
unpack_wide_kernel(const __grid_constant__ EightArgs a) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kEightWarps + threadIdx.x / 32;
    const int64_t row = id / a.sections;
    if (row >= a.n_rows) return;
    const int first = static_cast<int>((id - row * a.sections) * a.section) + threadIdx.x % 32 * 16;
    T* out = static_cast<T*>(a.out) + row * a.x_stride;
    uint4 q[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = first + 512 * u;
        q[u] = make_uint4(0, 0, 0, 0);
        scale[u] = 0.0f;
        if (c < a.dim) {
            q[u] = *reinterpret_cast<const uint4*>(a.codes + row * a.codes_stride + c);
            scale[u] = a.scales[row * a.blocks + c / kEightBlock];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = first + 512 * u;
        if (c >= a.dim) break;
        const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
        Words v[sizeof(T) / 2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = eight_values((w[i / 2] >> (16 * (i % 2))) & 0xFFFFu, scale[u]);
            if constexpr (sizeof(T) == 2) {
                v[0].w[i] = pack_bf16x2(f.x, f.y);
            } else {
                v[i / 4].w[2 * (i % 4)] = __float_as_uint(f.x);
                v[i / 4].w[2 * (i % 4) + 1] = __float_as_uint(f.y);
            }
        }
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) st_words(out + c + 8 * i, v[i]);
    }
}

// How rows are held where they go straight to registers: octets a thread, threads of a
// group, groups of a CTA.
struct RmsShape {
    int k, group, per_cta;
};

RmsShape rms_shape(int64_t dim, int k) {
    const int group = static_cast<int>((dim + 256 * k - 1) / (256 * k) * 32);
    int per_cta = 512 / group;
    if (per_cta > 8) per_cta = 8;               // 16 hardware barriers a CTA
    return {k, group, per_cta};
}

// The form through shared memory: groups and slots a ring that fit an SM.
constexpr int64_t kRowsSmem = 226 * 1024;

struct RowsShape {
    int k, group, per_cta, slots;
    int64_t slot_bytes, smem;
};

RowsShape rows_shape(int64_t dim, int elem, int64_t slot_bytes, bool weight_f32, bool back) {
    RowsShape s{};
    // octets a thread (8192 x 2048 bf16 forward by one 28 us, by two 32, backward 35 / 33; 16384 x
    // 4096 by one 105, by two 89, by four 105; 8192 x 8192 by two 92, by four 106)
    s.k = dim <= (back ? 1024 : 2048) ? 1 : dim <= 8192 ? 2 : 4;
    s.group = static_cast<int>((dim + 256 * s.k - 1) / (256 * s.k) * 32);
    s.slot_bytes = slot_bytes;
    const int64_t weight = weight_bytes(s.k, weight_f32) * ((dim + 7) / 8 * 8);
    const int64_t room = kRowsSmem - weight - 1024;
    s.per_cta = rows_threads(s.k, elem, back) / s.group;
    if (s.per_cta > 8) s.per_cta = 8;           // 16 hardware barriers a CTA
    const int least = back && s.k == 4 ? 3 : 2;
    while (s.per_cta > 1 && room / (s.per_cta * slot_bytes) < least) --s.per_cta;
    const int64_t one = s.per_cta * slot_bytes;
    // 64 KB on their way an SM: 16384 x 4096 bf16 forward 89 us so (two slots a group), with
    // three 101, with eight 106; backward 90, with one more 89 to 98; 8192 x 2048 forward 28,
    // with 32 KB 31
    int64_t ahead = (64 * 1024 + one - 1) / one;
    ahead = ahead < least ? least : ahead > 8 ? 8 : ahead;
    s.slots = static_cast<int>(room / one < ahead ? room / one : ahead);
    s.smem = s.slots * one + weight + 8 * s.per_cta * s.slots;
    if (s.smem < s.per_cta * dim * 4) s.smem = s.per_cta * dim * 4;
    return s;
}

int64_t rms_grid(const RmsShape& s, int64_t rows, int64_t per_sm) {
    const int64_t need = (rows + s.per_cta - 1) / s.per_cta;
    const int64_t most = static_cast<int64_t>(device_sms()) * per_sm;
    return need < 1 ? 1 : need < most ? need : most;
}

int64_t rms_forward_grid(const RmsShape& s, int64_t rows) {
    return rms_grid(s, rows, s.k == 1 ? 1024 / (s.group * s.per_cta) : 512 / (s.group * s.per_cta));
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

// A kernel's leave to use all of the shared memory, once a device.
template <class K>
cudaError_t allow_smem(K kernel, std::once_flag (&once)[64], cudaError_t (&set)[64]) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kRowsSmem));
    });
    return set[dev];
}

// What a call takes: rows through shared memory, or straight to registers.
struct RmsPlan {
    bool rows, wide;
    RowsShape through;
    RmsShape straight;
    int64_t grid;
};

RmsPlan forward_plan(const RmsArgs& a, int act_bytes) {
    RmsPlan p{};
    p.wide = wide_rows(a.x, a.x_stride, act_bytes) &&
             wide_rows(a.residual, a.residual_stride, act_bytes) &&
             wide_rows(a.total, a.total_stride, act_bytes) &&
             wide_rows(a.out, a.out_stride, act_bytes) && wide_codes(a.out8, a.out8_stride) &&
             wide_codes(a.total8, a.total8_stride);
    p.straight = rms_shape(a.dim, a.dim <= 4096 ? 1 : a.dim <= 8192 ? 2 : 4);
    p.through = rows_shape(a.dim, act_bytes,
                           (a.residual != nullptr ? 2 : 1) * row_room(a.dim, act_bytes, true),
                           a.weight != nullptr && a.param_f32, false);
    p.rows = p.wide && a.dim % 8 == 0 && p.through.slots >= 2;
    p.grid = p.rows ? rms_grid({0, 0, p.through.per_cta}, a.n_rows, 1)
                    : rms_forward_grid(p.straight, a.n_rows);
    return p;
}

RmsPlan backward_plan(const RmsArgs& a, int act_bytes) {
    RmsPlan p{};
    const bool eight = a.total8 != nullptr;
    p.wide = wide_rows(a.x, a.x_stride, act_bytes) &&
             wide_rows(a.grad_out, a.grad_out_stride, act_bytes) &&
             wide_rows(a.grad_total, a.grad_total_stride, act_bytes) &&
             wide_rows(a.grad_x, a.grad_x_stride, act_bytes) &&
             wide_rows(a.out, a.out_stride, act_bytes) && wide_codes(a.total8, a.total8_stride);
    p.straight = rms_shape(a.dim, kWideOctets);
    const bool grid = p.wide && a.dim % 8 == 0 &&
                      (!eight || (a.dim % 16 == 0 && wide_rows(a.total8, a.total8_stride, 1)));
    p.through = rows_shape(a.dim, act_bytes,
                           (a.grad_total != nullptr ? 2 : 1) * row_room(a.dim, act_bytes, grid) +
                               row_room(a.dim, eight ? 1 : act_bytes, grid),
                           a.weight != nullptr && a.param_f32, true);
    p.rows = p.through.slots >= 2;
    if (p.rows) p.wide = grid;
    p.grid = p.rows ? rms_grid({0, 0, p.through.per_cta}, a.n_rows, 1)
                    : rms_backward_grid(p.straight, a.n_rows);
    return p;
}

template <class T, int K, bool WIDE, bool BACK, bool EIGHT>
cudaError_t launch_rows(RmsArgs a, const RmsPlan& p, cudaStream_t stream) {
    if (cudaError_t e = device_status_word(&a.status); e != cudaSuccess) return e;
    static std::once_flag once[64];
    static cudaError_t set[64];
    const auto kernel = [] {
        if constexpr (BACK) return rms_rows_grad_kernel<T, K, WIDE, EIGHT>;
        else return rms_rows_kernel<T, K>;
    }();
    if (cudaError_t e = allow_smem(kernel, once, set); e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(p.grid), p.through.group * p.through.per_cta, p.through.smem,
             stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

int rms_grad_ctas(int64_t n_rows) {
    const int64_t sms = device_sms();
    return static_cast<int>(n_rows < 1 ? 1 : n_rows < sms ? n_rows : sms);
}

cudaError_t launch_rms_norm(RmsArgs a, int act_bytes, cudaStream_t stream) {
    const RmsPlan p = forward_plan(a, act_bytes);
    a.group_threads = p.rows ? p.through.group : p.straight.group;
    a.slots = p.through.slots;
    a.slot_bytes = static_cast<uint32_t>(p.through.slot_bytes);
    return by_type(act_bytes, [&](auto t) {
        using T = decltype(t);
        return by_k(p.rows ? p.through.k : p.straight.k, [&](auto k) {
            constexpr int K = k.value;
            if (p.rows) return launch_rows<T, K, true, false, false>(a, p, stream);
            const unsigned grid = static_cast<unsigned>(p.grid);
            const int threads = p.straight.group * p.straight.per_cta;
            if (p.wide) rms_norm_kernel<T, K, true><<<grid, threads, 0, stream>>>(a);
            else rms_norm_kernel<T, K, false><<<grid, threads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_rms_norm_grad(RmsArgs a, int act_bytes, cudaStream_t stream) {
    const RmsPlan p = backward_plan(a, act_bytes);
    a.group_threads = p.rows ? p.through.group : p.straight.group;
    a.slots = p.through.slots;
    a.slot_bytes = static_cast<uint32_t>(p.through.slot_bytes);
    return by_type(act_bytes, [&](auto t) {
        using T = decltype(t);
        if (p.rows)
            return by_k(p.through.k, [&](auto k) {
                constexpr int K = k.value;
                return a.total8 != nullptr
                           ? (p.wide ? launch_rows<T, K, true, true, true>(a, p, stream)
                                     : launch_rows<T, K, false, true, true>(a, p, stream))
                           : (p.wide ? launch_rows<T, K, true, true, false>(a, p, stream)
                                     : launch_rows<T, K, false, true, false>(a, p, stream));
            });
        auto kernel =
            p.wide ? rms_norm_grad_kernel<T, true, false> : rms_norm_grad_kernel<T, false, false>;
        if (a.total8 != nullptr) {
            // (shared memory holds two rows of bf16 beside 8 bits, however wide)
            if constexpr (sizeof(T) == 2) return cudaErrorInvalidConfiguration;
            else
                kernel = p.wide ? rms_norm_grad_kernel<T, true, true>
                                : rms_norm_grad_kernel<T, false, true>;
        }
        // one group of up to 16384 columns: 64 KB
        if (cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
            e != cudaSuccess)
            return e;
        kernel<<<static_cast<unsigned>(p.grid), p.straight.group * p.straight.per_cta,
                 sizeof(float) * p.straight.per_cta * a.dim, stream>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_rms_reduce(const RmsArgs& a, int act_bytes, cudaStream_t stream) {
    const int64_t parts = backward_plan(a, act_bytes).grid;
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
    const bool pack = a.out == nullptr;
    const void* act = pack ? a.x : a.out;
    const bool wide = wide_rows(act, a.x_stride, act_bytes) && wide_codes(a.codes, a.codes_stride);
    // 32-byte words of 16 columns (16384 x 4096 bf16: packed 34.8 us, by octets 36.3;
    // unpacked 35.6 / 39.3)
    const bool words = a.dim % 16 == 0 && aligned_to(act, 32) && a.x_stride * act_bytes % 32 == 0 &&
                       aligned_to(a.codes, 16) && a.codes_stride % 16 == 0;
    a.section = words ? 512 * kWideUnits : 256 * (pack ? kPackOctets : kUnpackOctets);
    a.sections = (a.dim + a.section - 1) / a.section;
    const int64_t ctas = (a.n_rows * a.sections + kEightWarps - 1) / kEightWarps;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(ctas);
    return by_type(act_bytes, [&](auto t) {
        using T = decltype(t);
        const auto kernel = words  ? (pack ? pack_wide_kernel<T, kWideUnits>
                                           : unpack_wide_kernel<T, kWideUnits>)
                            : pack ? (wide ? pack_kernel<T, true> : pack_kernel<T, false>)
                                   : (wide ? unpack_kernel<T, true> : unpack_kernel<T, false>);
        kernel<<<grid, 32 * kEightWarps, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace zf
