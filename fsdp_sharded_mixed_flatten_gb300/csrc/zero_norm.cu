// Layer norm over rows of `dim` values:
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r,
//   y = xh w + b,
// and its backward pass for g = dy w:
//   dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy.
//
// A row lives in the registers of a group of threads, E elements each, so that
// every byte of x, dy and the output crosses memory once.  A CTA holds several
// groups, which work through the rows independently; the next rows' loads are
// under way while a row is worked on (cp.async to shared memory, each thread its
// own words, so that no barrier separates copy and use).  The parameters stay in
// registers or, to leave room for more warps, in shared memory (each thread its
// own columns: no barrier), and the backward pass's columns of dw and db in
// registers over all rows; each CTA writes one pair of partial rows, which a
// second launch adds up in CTA order.
//
// Bound by memory where rows are many: forward of 16384 x 4096 bf16 50 us (5.4 TB/s),
// backward of 8192 x 8192 bf16 78 us (5.1 TB/s), of 8192 x 768 bf16 14.6 us (2.6 TB/s: the
// launch, the first rows and the second launch are most of it).  Few rows take as
// long as the host's call: 8 x 768 7.5 us forward, 9.1 us backward.
//
// The variance is taken about a mean at every step: a warp's squares about the
// warp's mean, then sum (M2_w + n_w (mean_w - mu)^2) over the warps of the
// row, so that a mean far from zero costs no digits and one exchange is enough.
#include "zero_ops.cuh"

#include <mutex>

namespace zf {

namespace {

constexpr int kNormThreads = 512;      // of a CTA, but for the backward pass at E = 8
constexpr int kNormWarps = 24;         // of a CTA, at most

// Of the backward pass at E = 8: one CTA of 768 threads an SM with bf16 (80
// registers), of 512 with fp32 (128), whose rows take twice as many.  8192 x 768:
// bf16 15.2 us, with two CTAs of 256 17.2; fp32 20.9 us, with two of 256 23.2.
__host__ __device__ constexpr int grad_threads(int elem) { return elem == 2 ? 768 : 512; }

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
    __device__ void sync_any() const {
        if (warps == 1) __syncwarp();
        else sync();
    }
};

// How a row's elements are reached: by 16-byte words; by words, shifted, where
// rows do not start on 16-byte boundaries; by single elements.  Shifting costs a
// row two barriers more, and pays where a row's elements keep a thread busy: 8192
// rows, in us, shifted / single:
//            1500 bf16  4001 bf16  8190 bf16  1501 fp32  4001 fp32  8190 fp32
//   forward   25 / 21    46 / 68    85 / 138   29 / 24    72 / 81   155 / 165
//   backward  33 / 49    65 / 133  140 / 272   44 / 39    91 / 119  179 / 242
// Beyond 8192 columns shared memory has no room for it.
enum Access { kWide, kShift, kSingle };
__host__ __device__ constexpr Access access_of(bool wide, int e, int elem, bool back) {
    if (wide) return kWide;
    return e == 16 || (e == 8 && elem == 2 && back) ? kShift : kSingle;
}

// Rows under way at a time in shared memory (0: one, in registers), for `arrays`
// matrices.  In us by rows under way (1, 2, 3, 4):
//   forward of 16384 rows: 768 bf16 20.7, 17.1, 17.1, 17.2; 2048 fp32 58.8, 45.8,
//     48.6, 50.8; 4096 bf16 65.0, 51.0, 80.0 (no room for a second CTA), 71.9;
//     8192 fp32 180.9, 179.2, 164.9, 165.8
//   backward of 8192 rows: 768 bf16 15.9, 14.8, 15.1, 15.2; 2048 fp32 53.1, 39.7,
//     40.2, 40.8; 4096 bf16 65.6, 44.2, 43.6, 53.2; 8192 fp32 158.6, 133.4, 137.2
// (Through shifts a row's slot serves its result too: one more for as many.)
__host__ __device__ constexpr int depth_of(Access access, int e, int elem, int arrays) {
    if (access == kSingle) return 0;
    if (e == 8) return access == kWide ? 2 : 3;
    if (e == 16) return (arrays == 1) == (elem == 4) ? 3 : 2;
    return elem == 2 ? 2 : arrays - 1;
}

__device__ __forceinline__ void cp_async16_fill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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
    // the same through shared memory: this thread's words of one row
    __device__ static __forceinline__ void copy(uint32_t to, const T* at, bool in,
                                                const Columns<VEC, E>& c) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int bytes = in ? c.left[n] * static_cast<int>(sizeof(T)) : 0;
            cp_async16_fill(to + 16u * n * blockDim.x, at + (bytes != 0 ? n * c.step : 0), bytes);
        }
    }
    __device__ __forceinline__ void read(const char* from) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            p[n] = *reinterpret_cast<const Pack<T, VEC>*>(from + 16u * n * blockDim.x);
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

// The first `left` of a pack's values.
template <class T, int VEC>
__device__ __forceinline__ void store_pack(T* at, const Pair* y, int left) {
    if (left == 0) return;
    Pack<T, VEC> v;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) reinterpret_cast<uint32_t*>(&v)[i] = narrow2(y[i]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float2 f = unpair(y[i]);
            v.x[2 * i] = narrow<T>(f.x);
            v.x[2 * i + 1] = narrow<T>(f.y);
        }
    }
    if (left == VEC) {
        st_pack<T, VEC>(at, v);
    } else {
#pragma unroll
        for (int e = 0; e < VEC - 1; ++e) {
            if (e < left) at[e] = v.x[e];
        }
    }
}

template <class T, int VEC, int E>
__device__ __forceinline__ void store_row(T* at, const Pair (&y)[E / 2], const Columns<VEC, E>& c) {
#pragma unroll
    for (int n = 0; n < E / VEC; ++n) {
        if constexpr (VEC == 1) {
            const float2 f = unpair(y[n / 2]);
            if (c.left[n] != 0) at[n * c.step] = narrow<T>(n % 2 == 0 ? f.x : f.y);
        } else {
            store_pack<T, VEC>(at + n * c.step, y + n * VEC / 2, c.left[n]);
        }
    }
}

// Rows through shifts: the group copies the aligned words that hold the row, each
// thread takes its 16 bytes from two of them, and the result goes through the
// row's slot to aligned words again, its ends by single elements.  Of the first
// word the bytes before the row are read, and not used.

__device__ __forceinline__ int off_grid(const void* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16);
}

template <class T, int E>
struct Shift {
    static constexpr int V = 16 / sizeof(T), N = E / V;
    // Words of a slot: those of the row and one more.
    __device__ static __forceinline__ int words(const Group& g) { return N * g.threads + 1; }
    __device__ static __forceinline__ void copy(uint32_t slot, const T* row, bool in, int dim,
                                                const Group& g) {
        const int mis = off_grid(row);
        const char* from = reinterpret_cast<const char*>(row) - mis;
        const int bytes = in ? mis + dim * static_cast<int>(sizeof(T)) : 0;
        auto word = [&](int w) {
            const int n = min(max(bytes - 16 * w, 0), 16);
            cp_async16_fill(slot + 16u * w, from + (n != 0 ? 16 * w : 0), n);
        };
#pragma unroll
        for (int n = 0; n < N; ++n) word(n * g.threads + g.t);
        if (g.t == 0) word(N * g.threads);
    }
    __device__ static __forceinline__ void read(Row<T, V, E>& r, const uint4* slot, const T* row,
                                                const Group& g) {
        const int mis = off_grid(row);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint4* at = slot + n * g.threads + g.t;
            *reinterpret_cast<uint4*>(&r.p[n]) = shifted<T>(at[0], at[1], mis);
        }
    }
    // The slot has been read by all of the group.
    __device__ static __forceinline__ void store(T* row, const Pair (&y)[E / 2], uint4* slot,
                                                 int dim, const Group& g) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint4 v;
            if constexpr (sizeof(T) == 2) {
                v = make_uint4(narrow2(y[4 * n]), narrow2(y[4 * n + 1]), narrow2(y[4 * n + 2]),
                               narrow2(y[4 * n + 3]));
            } else {
                const float2 lo = unpair(y[2 * n]), hi = unpair(y[2 * n + 1]);
                v = make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y),
                               __float_as_uint(hi.x), __float_as_uint(hi.y));
            }
            slot[n * g.threads + g.t] = v;
        }
        g.sync_any();
        const int mis = off_grid(row);
        const int head = min(dim, mis == 0 ? 0 : V - mis / static_cast<int>(sizeof(T)));
        const int full = (dim - head) / V, by = head * static_cast<int>(sizeof(T));
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int q = n * g.threads + g.t;
            if (q < full)
                *reinterpret_cast<uint4*>(row + head + q * V) =
                    shifted<T>(slot[q], slot[q + 1], by);
        }
        const T* at = reinterpret_cast<const T*>(slot);
        const int tail = head + full * V;
        if (g.t < head) row[g.t] = at[g.t];
        if (g.t < dim - tail) row[tail + g.t] = at[tail + g.t];
    }
};

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

// Sums of a pair of values over a group, in a fixed order: lanes, then warps.
// The first exchange leaves one value to each half of the warp, so that five
// steps add up both.  `red` has two halves that are used in turn: one barrier a
// call is enough.
__device__ __forceinline__ float2 group_sum2(const Group& g, float x, float y,
                                             float (*red)[2][kNormWarps], int& half) {
    const int lane = threadIdx.x % 32;
    const bool low = lane < 16;
    float v = low ? x : y;
    v += __shfl_xor_sync(0xFFFFFFFFu, low ? y : x, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (g.warps == 1)
        return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
    float(*slot)[kNormWarps] = red[half];
    half ^= 1;
    const int w0 = g.index * g.warps;
    if (lane % 16 == 0) slot[low ? 0 : 1][w0 + g.t / 32] = v;
    g.sync();
    if (g.warps <= 6) {
        x = y = 0.0f;
        for (int w = 0; w < g.warps; ++w) {
            x += slot[0][w0 + w];
            y += slot[1][w0 + w];
        }
        return make_float2(x, y);
    }
    v = lane % 16 < g.warps ? slot[low ? 0 : 1][w0 + lane % 16] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
}

template <class T, int VEC, int E, bool SHIFT>
__global__ void __launch_bounds__(kNormThreads, E == 32 ? 1 : 2)
norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kDepth = depth_of(SHIFT ? kShift : VEC > 1 ? kWide : kSingle, E, sizeof(T), 1);
    constexpr bool kAsync = kDepth > 0;
    extern __shared__ __align__(16) char params[];           // weight, bias, rows
    constexpr int P = E / 2;
    __shared__ float2 red[2][kNormWarps];
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
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + (SHIFT ? 0 : c.first);
    T* out = static_cast<T*>(a.out) + row * a.out_stride + (SHIFT ? 0 : c.first);
    const T* here = x;                                       // the row worked on
    Row<T, VEC, E> next;
    // this thread's words of row slot k, or with SHIFT its group's: at held + k * slot
    const uint32_t slot = SHIFT ? 16 * Shift<T, E>::words(g) : sizeof(T) * E * blockDim.x;
    char* held = params + 2 * sizeof(float) * E * blockDim.x +
                 (SHIFT ? kDepth * slot * g.index : 16 * threadIdx.x);
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(held));
    int64_t ahead = row;                                     // the next row to copy
    int put = 0, get = 0;
    // (a row beyond the last: nothing is read, from an address that is)
    auto copy_next = [&] {
        const bool in = ahead < a.n_rows;
        const T* from = in ? x : static_cast<const T*>(a.x);
        if constexpr (SHIFT) Shift<T, E>::copy(to + put * slot, from, in, a.dim, g);
        else Row<T, VEC, E>::copy(to + put * slot, from, in, c);
        cp_async_commit();
        x += step * a.x_stride;
        ahead += step;
        put = put + 1 == kDepth ? 0 : put + 1;
    };
    if constexpr (kAsync) {
        for (int k = 0; k < kDepth - 1; ++k) copy_next();
    } else {
        next.load(x, row < a.n_rows, c);
    }
    for (; row < a.n_rows; row += step, out += step * a.out_stride) {
        uint4* const words = reinterpret_cast<uint4*>(held + get * slot);
        if constexpr (SHIFT) {
            // the row has come, and all have done with the slot that the next copy takes
            cp_async_wait<kDepth - 2 < 0 ? 0 : kDepth - 2>();
            g.sync_any();
            copy_next();
            Shift<T, E>::read(next, words, here, g);
            here += step * a.x_stride;
            get = get + 1 == kDepth ? 0 : get + 1;
        } else if constexpr (kAsync) {
            copy_next();
            cp_async_wait<kDepth - 1 < 0 ? 0 : kDepth - 1>();
            next.read(held + get * slot);
            get = get + 1 == kDepth ? 0 : get + 1;
        }
        Pair v[P];
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = next[j];
        if constexpr (!kAsync) {
            x += step * a.x_stride;
            next.load(x, row + step < a.n_rows, c);
        }
        float2 s;                // a warp's sum, and its squares about its mean
        Pair t = v[0];
#pragma unroll
        for (int j = 1; j < P; ++j) t = add2(t, v[j]);
        s.x = warp_sum(both(t));
        const Pair m = splat(-s.x * inv_n);
        Pair q = 0;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            Pair d = add2(v[j], m);
            if (VEC == 1 || ragged) {
                const float2 f = unpair(d);
                d = pair(c.ok(2 * j / VEC, 2 * j % VEC) ? f.x : 0.0f,
                         c.ok((2 * j + 1) / VEC, (2 * j + 1) % VEC) ? f.y : 0.0f);
            } else {
                d = c.left[2 * j / VEC] != 0 ? d : 0;
            }
            q = fma2(d, d, q);
        }
        s.y = warp_sum(both(q));
        if (g.warps > 1) {
            const int w0 = g.index * g.warps;
            if (lane == 0) red[half][w0 + g.t / 32] = s;
            g.sync();
            const float2 o = lane < g.warps ? red[half][w0 + lane] : make_float2(0.0f, 0.0f);
            s.x = warp_sum(o.x);
            const float d = __fmaf_rn(o.x, lane_inv_n, -s.x * inv_d);
            s.y = warp_sum(lane < g.warps ? __fmaf_rn(lane_n * d, d, o.y) : 0.0f);
            half ^= 1;
        }
        const float mu = s.x * inv_d;
        const float r = inv_sqrt(__fmaf_rn(s.y, inv_d, a.eps));
        if (g.t == 0) {
            if (a.mean != nullptr) a.mean[row] = mu;
            if (a.rstd != nullptr) a.rstd[row] = r;
        }
        const Pair m2 = splat(-mu), r2 = splat(r);
#pragma unroll
        for (int j = 0; j < P / 2; ++j) {
            const ulonglong2 wj = w[j], bj = b[j];
            v[2 * j] = fma2(mul2(add2(v[2 * j], m2), r2), wj.x, bj.x);
            v[2 * j + 1] = fma2(mul2(add2(v[2 * j + 1], m2), r2), wj.y, bj.y);
        }
        if constexpr (SHIFT) {
            if (g.warps == 1) __syncwarp();              // the others: at the sums
            Shift<T, E>::store(out, v, words, a.dim, g);
        } else {
            store_row<T, VEC, E>(out, v, c);
        }
    }
}

template <class T, int VEC, int E, bool SHIFT>
__global__ void __launch_bounds__(E == 8 ? grad_threads(sizeof(T)) : kNormThreads, 1)
norm_grad_kernel(const __grid_constant__ NormArgs a) {
    constexpr int P = E / 2;
    constexpr bool kKeep = E > 8;            // the weight in shared memory
    constexpr int kDepth = depth_of(SHIFT ? kShift : VEC > 1 ? kWide : kSingle, E, sizeof(T), 2);
    constexpr bool kAsync = kDepth > 0;
    // 32 columns of dw and db leave no registers for the row: it is read from its
    // slot twice, before and after its sums (8192 x 16384: bf16 181 us, 4.5 TB/s, kept
    // in registers 308; fp32 334 us, 4.8 TB/s, in registers 771)
    constexpr bool kTwice = E == 32 && kAsync;
    extern __shared__ __align__(16) char dyn[];
    float* cols = reinterpret_cast<float*>(dyn);     // [groups][dim] at the end;
                                                     // before, the weight and the rows
    __shared__ float red[2][2][kNormWarps];
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
    const int64_t step = static_cast<int64_t>(gridDim.x) * g.per_cta;
    int64_t row = static_cast<int64_t>(blockIdx.x) * g.per_cta + g.index;
    const int first = SHIFT ? 0 : c.first;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + first;
    const T* dy = static_cast<const T*>(a.grad_out) + row * a.grad_out_stride + first;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + first;
    const T *x_here = x, *dy_here = dy;                      // the row worked on
    Row<T, VEC, E> next_x, next_y;
    float next_mu = 0.0f, next_r = 0.0f;
    // this thread's words of row slot k, or with SHIFT its group's: at held + k * slot,
    // x then dy
    const uint32_t one = SHIFT ? 16 * Shift<T, E>::words(g) : sizeof(T) * E * blockDim.x;
    const uint32_t slot = 2 * one;
    char* held = dyn + (kKeep ? sizeof(float) * E * blockDim.x : 0) +
                 (SHIFT ? kDepth * slot * g.index : 16 * threadIdx.x);
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(held));
    int64_t ahead = row;                                     // the next row to copy
    int put_at = 0, get = 0;
    // (a row beyond the last: nothing is read, from an address that is)
    auto copy_next = [&] {
        const bool in = ahead < a.n_rows;
        const T* from_x = in ? x : static_cast<const T*>(a.x);
        const T* from_y = in ? dy : static_cast<const T*>(a.grad_out);
        if constexpr (SHIFT) {
            Shift<T, E>::copy(to + put_at * slot, from_x, in, a.dim, g);
            Shift<T, E>::copy(to + put_at * slot + one, from_y, in, a.dim, g);
        } else {
            Row<T, VEC, E>::copy(to + put_at * slot, from_x, in, c);
            Row<T, VEC, E>::copy(to + put_at * slot + one, from_y, in, c);
        }
        cp_async_commit();
        x += step * a.x_stride;
        dy += step * a.grad_out_stride;
        ahead += step;
        put_at = put_at + 1 == kDepth ? 0 : put_at + 1;
    };
    auto load_stats = [&](int64_t at) {
        if (at < a.n_rows) {
            next_mu = a.mean[at];
            next_r = a.rstd[at];
        }
    };
    auto load = [&](int64_t at) {
        next_x.load(x, at < a.n_rows, c);
        next_y.load(dy, at < a.n_rows, c);
    };
    load_stats(row);
    if constexpr (kAsync) {
        for (int k = 0; k < (kDepth == 1 ? 1 : kDepth - 1); ++k) copy_next();
    } else {
        load(row);
    }
    for (; row < a.n_rows; row += step, out += step * a.out_stride) {
        uint4* const words = reinterpret_cast<uint4*>(held + get * slot);
        if constexpr (SHIFT) {
            cp_async_wait<kDepth - 2 < 0 ? 0 : kDepth - 2>();
            g.sync_any();
            copy_next();
            Shift<T, E>::read(next_x, words, x_here, g);
            Shift<T, E>::read(next_y, words + one / 16, dy_here, g);
            x_here += step * a.x_stride;
            dy_here += step * a.grad_out_stride;
            get = get + 1 == kDepth ? 0 : get + 1;
        } else if constexpr (kTwice) {
            // (one slot: the next row is copied when this one has been used up)
            if (kDepth > 1) copy_next();
            cp_async_wait<kDepth - 1 < 0 ? 0 : kDepth - 1>();
            const char* const at = held + get * slot;
            const float r = next_r;
            const Pair mu2 = splat(-next_mu), r2 = splat(r);
            // f(pair, pair of its pack, xh, dy, g), done(pack)
            auto each = [&](auto&& f, auto&& done) {
#pragma unroll
                for (int n = 0; n < E / VEC; ++n) {
                    Row<T, VEC, VEC> px, py;
                    px.read(at + 16u * n * blockDim.x);
                    py.read(at + one + 16u * n * blockDim.x);
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        const int j = n * VEC / 2 + i;
                        const Pair wj = j % 2 == 0 ? kept[j / 2].x : kept[j / 2].y;
                        f(j, i, mul2(add2(px[i], mu2), r2), py[i], mul2(py[i], wj));
                    }
                    done(n);
                }
            };
            Pair s1 = 0, s2 = 0;
            each([&](int, int, Pair xh, Pair, Pair gr) {
                s1 = add2(s1, gr);
                s2 = fma2(gr, xh, s2);
            }, [](int) {});
            load_stats(row + step);
            const float2 s = group_sum2(g, both(s1), both(s2), red, half);
            const Pair m1 = splat(-s.x * inv_d * r), m2 = splat(-s.y * inv_d * r);
            Pair y[VEC / 2];
            each([&](int j, int i, Pair xh, Pair d, Pair gr) {
                dw[j] = fma2(d, xh, dw[j]);
                db[j] = add2(db[j], d);
                y[i] = fma2(xh, m2, fma2(gr, r2, m1));
            }, [&](int n) { store_pack<T, VEC>(out + n * c.step, y, c.left[n]); });
            get = get + 1 == kDepth ? 0 : get + 1;
            if (kDepth == 1) copy_next();
            continue;
        } else if constexpr (kAsync) {
            copy_next();
            cp_async_wait<kDepth - 1 < 0 ? 0 : kDepth - 1>();
            next_x.read(held + get * slot);
            next_y.read(held + get * slot + one);
            get = get + 1 == kDepth ? 0 : get + 1;
        }
        Pair xh[P], gr[P];
        // dy is 0 where there is no column, and adds nothing there
        const float r = next_r;
        const Pair mu2 = splat(-next_mu), r2 = splat(r);
        Pair s1 = 0, s2 = 0;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const Pair d = next_y[j];
            Pair wj = w[j];
            if (kKeep) wj = j % 2 == 0 ? kept[j / 2].x : kept[j / 2].y;
            xh[j] = mul2(add2(next_x[j], mu2), r2);
            gr[j] = mul2(d, wj);
            dw[j] = fma2(d, xh[j], dw[j]);
            db[j] = add2(db[j], d);
            s1 = add2(s1, gr[j]);
            s2 = fma2(gr[j], xh[j], s2);
        }
        if constexpr (!kAsync) {
            x += step * a.x_stride;
            dy += step * a.grad_out_stride;
            load(row + step);
        }
        load_stats(row + step);
        const float2 s = group_sum2(g, both(s1), both(s2), red, half);
        const Pair m1 = splat(-s.x * inv_d * r), m2 = splat(-s.y * inv_d * r);
#pragma unroll
        for (int j = 0; j < P; ++j) gr[j] = fma2(xh[j], m2, fma2(gr[j], r2, m1));
        if constexpr (SHIFT) {
            if (g.warps == 1) __syncwarp();              // the others: at the sums
            Shift<T, E>::store(out, gr, words, a.dim, g);
        } else {
            store_row<T, VEC, E>(out, gr, c);
        }
    }
    if constexpr (kAsync) cp_async_wait<0>();        // nothing is to come in the columns' place
    float* part = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.dim;
    auto put = [&](const Pair (&acc)[P], float* to) {
        if constexpr (VEC >= 4) {
            if (a.dim % 4 == 0) {
                // 16 bytes at a time: single values 8 columns apart would meet
                // in the same banks
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    const int n = 2 * j / VEC, e = 2 * j % VEC;
                    const float2 f = unpair(acc[j]), h = unpair(acc[j + 1]);
                    if (c.ok(n, e))
                        *reinterpret_cast<float4*>(to + c.at(n) + e) =
                            make_float4(f.x, f.y, h.x, h.y);
                }
                return;
            }
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float2 f = unpair(acc[j]);
            const int n0 = 2 * j / VEC, n1 = (2 * j + 1) / VEC;
            if (c.ok(n0, 2 * j % VEC)) to[c.at(n0) + 2 * j % VEC] = f.x;
            if (c.ok(n1, (2 * j + 1) % VEC)) to[c.at(n1) + (2 * j + 1) % VEC] = f.y;
        }
    };
    // no other CTA's partial rows: the sums themselves (not where a thread holds 32
    // columns: one row of 16384 bf16 25.4 us, with the second launch 21.3 then)
    const bool alone = E < 32 && gridDim.x == 1;
    if (g.per_cta == 1 && !alone) {
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
            void* to = which == 0 ? a.grad_weight : a.grad_bias;
            if (!alone) part[which * a.dim + k] = t;
            else if (to != nullptr) st_param(to, a.param_f32, k, t);
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

Shape shape_for(int64_t dim, int elem, bool back) {
    const int e = dim <= 2048 ? 8 : dim <= 16 * kNormThreads ? 16 : 32;
    const int group = static_cast<int>((dim + e * 32 - 1) / (e * 32) * 32);
    int per_cta = (back && e == 8 ? grad_threads(elem) : kNormThreads) / group;
    if (per_cta > 8) per_cta = 8;               // 16 hardware barriers a CTA
    return {e, group, per_cta};
}

size_t smem_of(const Shape& s, int64_t dim, int elem, bool wide, bool back) {
    const size_t threads = s.group * s.per_cta;
    const Access access = access_of(wide, s.e, elem, back);
    const size_t slot = elem * s.e * threads + (access == kShift ? 16 * s.per_cta : 0);
    const size_t rows =
        static_cast<size_t>(depth_of(access, s.e, elem, back ? 2 : 1)) * (back ? 2 : 1) * slot;
    if (!back) return 2 * sizeof(float) * s.e * threads + rows;
    const size_t kept = s.e > 8 ? sizeof(float) * s.e * threads : 0;
    const size_t cols = sizeof(float) * s.per_cta * dim;
    return kept + rows > cols ? kept + rows : cols;
}

// Rows of the backward pass that one CTA takes by itself: what it adds up are
// the sums, and the second launch is saved.  Up to 2048 columns 8 rounds of its
// groups and 24576 elements (one launch / two, in us: 32 x 768 bf16, four rounds,
// 9.2 / 10.8, fp32, seven, 10.2 / 10.8, 64 x 768 bf16 13.0 / 11.8), beyond one round
// (8 x 4096 bf16 in four 12.8 / 11.6).  The host holds these up: replayed from a graph,
// 16 x 768 takes 4.9 / 5.2 in bf16 and 5.5 / 4.9 in fp32, 32 x 768 6.7 / 5.3 and 7.7 / 5.0.
int64_t rows_alone(const Shape& s, int64_t dim) {
    if (s.e > 8) return s.per_cta;
    const int64_t by_size = 24576 / dim;
    return by_size < 8 * s.per_cta ? by_size : 8 * s.per_cta;
}

// CTAs: what the registers (launch bounds) and the shared memory of an SM hold,
// or what the rows need.
int64_t ctas_for(const Shape& s, int64_t rows, int64_t dim, int elem, bool wide, bool back) {
    const int threads = s.group * s.per_cta;
    int per_sm = back ? (s.e == 8 ? grad_threads(elem) / threads : 1)
                      : (s.e == 32 ? 1 : 2 * kNormThreads / threads);
    const int by_smem =
        static_cast<int>(225 * 1024 / (smem_of(s, dim, elem, wide, back) + 2048));
    if (by_smem < per_sm) per_sm = by_smem > 0 ? by_smem : 1;
    const int64_t few = back ? rows_alone(s, dim) : 0;
    const int64_t need = rows > few ? (rows + s.per_cta - 1) / s.per_cta : 1;
    const int64_t most = static_cast<int64_t>(device_sms()) * per_sm;
    return need < most ? need : most;
}

// Whether every row of a matrix starts on a 16-byte boundary.
bool wide_rows(int elem, const void* p, int64_t stride) {
    return aligned_to(p, 16) && stride % (16 / elem) == 0;
}

template <class T, int E, Access ACCESS, bool BACK>
cudaError_t launch_e(const NormArgs& a, unsigned grid, int threads, size_t smem,
                     cudaStream_t stream) {
    constexpr int VEC = ACCESS == kSingle ? 1 : 16 / sizeof(T);
    const auto kernel = BACK ? norm_grad_kernel<T, VEC, E, ACCESS == kShift>
                             : norm_kernel<T, VEC, E, ACCESS == kShift>;
    // more than 48 KB of shared memory need asking for
    static std::once_flag once[64];
    static cudaError_t set[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        224 * 1024);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    kernel<<<grid, threads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <class T, bool WIDE, bool BACK>
cudaError_t launch_shape(NormArgs a, cudaStream_t stream) {
    constexpr int B = sizeof(T);
    const Shape s = shape_for(a.dim, B, BACK);
    a.group_threads = s.group;
    int sms = 0;
    if (cudaError_t e = device_sms(&sms); e != cudaSuccess) return e;
    const unsigned g = static_cast<unsigned>(ctas_for(s, a.n_rows, a.dim, B, WIDE, BACK));
    const int threads = s.group * s.per_cta;
    const size_t smem = smem_of(s, a.dim, B, WIDE, BACK);
    if (s.e == 8) return launch_e<T, 8, access_of(WIDE, 8, B, BACK), BACK>(a, g, threads, smem, stream);
    if (s.e == 16)
        return launch_e<T, 16, access_of(WIDE, 16, B, BACK), BACK>(a, g, threads, smem, stream);
    return launch_e<T, 32, access_of(WIDE, 32, B, BACK), BACK>(a, g, threads, smem, stream);
}

// Whether every row of every matrix starts on a 16-byte boundary.
template <bool BACK>
bool wide(const NormArgs& a, int act_bytes) {
    return wide_rows(act_bytes, a.x, a.x_stride) && wide_rows(act_bytes, a.out, a.out_stride) &&
           (!BACK || wide_rows(act_bytes, a.grad_out, a.grad_out_stride));
}

template <bool BACK>
cudaError_t dispatch(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    const bool w = wide<BACK>(a, act_bytes);
    if (act_bytes == 4)
        return w ? launch_shape<float, true, BACK>(a, stream)
                 : launch_shape<float, false, BACK>(a, stream);
    return w ? launch_shape<uint16_t, true, BACK>(a, stream)
             : launch_shape<uint16_t, false, BACK>(a, stream);
}

}  // namespace

// The most of any type and alignment.
int norm_grad_ctas(int64_t n_rows, int64_t dim) {
    int64_t most = 1;
    for (int elem = 2; elem <= 4; elem += 2) {
        const Shape s = shape_for(dim, elem, true);
        for (bool w : {false, true}) {
            const int64_t n = ctas_for(s, n_rows, dim, elem, w, true);
            if (n > most) most = n;
        }
    }
    return static_cast<int>(most);
}

cudaError_t launch_norm(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    return dispatch<false>(a, act_bytes, stream);
}

cudaError_t launch_norm_grad(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    return dispatch<true>(a, act_bytes, stream);
}

cudaError_t launch_norm_grad_reduce(const NormArgs& a, int act_bytes, cudaStream_t stream) {
    const int64_t width = 2 * static_cast<int64_t>(a.dim);
    const Shape s = shape_for(a.dim, act_bytes, true);
    const int64_t parts = ctas_for(s, a.n_rows, a.dim, act_bytes, wide<true>(a, act_bytes), true);
    if (parts == 1 && s.e < 32) return cudaSuccess;      // the sums themselves are there
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
    return cudaLaunchKernelEx(&cfg, norm_grad_reduce_kernel, a, static_cast<int>(parts));
}

}  // namespace zf
