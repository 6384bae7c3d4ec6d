// Distillation from a teacher's top logits.  For a row of student logits z
// over the vocabulary and the teacher's entries (id_k, l_k):
//   p = softmax(l / tau) over the entries,  q = softmax(z / tau) over the row,
//   loss = w tau^2 sum_k p_k (log p_k - log q_{id_k}),
//   dloss/dz_v = w tau (q_v - sum_{k: id_k = v} p_k).
//
// A cluster of CTAs holds a row in shared memory, each CTA a slice, and stays
// for many rows.  DRAM sees one read and one write of the logits:
//   - every thread copies its own 16-byte words with cp.async and is the only
//     one to read them, so no barrier separates copy and use;
//   - it adds up the exponentials as the words arrive; one cluster barrier
//     exchanges the warps' sums through distributed shared memory;
//   - it forms the gradient from the copy, and into each word it has used up
//     it copies the same word of the CTA's next row, so that reads and writes
//     of memory overlap all the time;
//   - one more warp reads the teacher's entries, a row ahead, and sets the
//     gradient's entries right once the plain values are written.
// Words beyond shared memory are read again from L2.
//
// Exponentials are 2^(z c - M), c = log2(e) / tau: one fused multiply-add and
// one ex2 each.  M is an integer, ceil(c max z) of what a thread has seen, so
// that moving from one M to another scales by an exact power of two.  Rows
// whose largest |c z| passes kFar (all logits at the type's lowest value, or
// infinities) take the difference first: 2^((z - max z) c).
#include "zero_ops.cuh"

#include <cooperative_groups.h>

#include <mutex>

namespace cg = cooperative_groups;

namespace zf {

namespace {

constexpr int kWorkers = 384;                    // threads that hold the slice
constexpr int kWorkerWarps = kWorkers / 32;
constexpr int kRowThreads = kWorkers + 32;       // and the teacher's warp
constexpr int kMaxCluster = 8;
constexpr int kSections = 3;                     // copy groups of a row
constexpr int kPatchAlone = 128;                 // entries the teacher's warp patches by itself
constexpr int kSliceBytes = 68 * 1024;           // a CTA's slice with 3 CTAs an SM
constexpr int kMostBytes = 176 * 1024;           // what one CTA an SM holds
constexpr float kInf = __builtin_huge_valf();
constexpr float kFar = 1e30f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^(x c + m), both halves
__device__ __forceinline__ Pair ex2_fma2(Pair x, Pair c, Pair m) {
    Pair p;
    asm("{\n\t.reg .b64 e;\n\t.reg .f32 a, b;\n\t"
        "fma.rn.f32x2 e, %1, %2, %3;\n\t"
        "mov.b64 {a, b}, e;\n\t"
        "ex2.approx.ftz.f32 a, a;\n\t"
        "ex2.approx.ftz.f32 b, b;\n\t"
        "mov.b64 %0, {a, b};\n\t}"
        : "=l"(p)
        : "l"(x), "l"(c), "l"(m));
    return p;
}

// A 16-byte word's values as pairs, and their maximum (NaN loses).
template <class T>
struct Word;

template <>
struct Word<uint16_t> {
    static constexpr int kPairs = 4;
    static __device__ __forceinline__ void split(uint4 w, Pair (&x)[4]) {
        x[0] = widen2(w.x);
        x[1] = widen2(w.y);
        x[2] = widen2(w.z);
        x[3] = widen2(w.w);
    }
    static __device__ __forceinline__ float top(uint4 w) {
        auto h = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(w.x), h(w.y)), __hmax2(h(w.z), h(w.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ uint4 join(const Pair (&y)[4]) {
        return make_uint4(narrow2(y[0]), narrow2(y[1]), narrow2(y[2]), narrow2(y[3]));
    }
};

template <>
struct Word<float> {
    static constexpr int kPairs = 2;
    static __device__ __forceinline__ void split(uint4 w, Pair (&x)[2]) {
        x[0] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
        x[1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ float top(uint4 w) {
        return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                     fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    static __device__ __forceinline__ uint4 join(const Pair (&y)[2]) {
        const float2 a = unpair(y[0]), b = unpair(y[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                          __float_as_uint(b.y));
    }
};

// A sum of 2^(z c - off) with an integer off.
struct Running {
    float off, s;
};

// Joined over a warp: the largest off, every sum scaled to it.
__device__ __forceinline__ Running warp_join(Running r) {
    const float off = warp_max(r.off);
    return {off, warp_sum(r.s * ex2(r.off - off))};
}

// The row's exponentials: near: 2^(z c - off), far: 2^((z - off) c).
struct Exponent {
    float c, off;
    bool far;
    __device__ __forceinline__ float log2q(float z) const {
        return far ? (z - off) * c : __fmaf_rn(z, c, -off);
    }
};

// This CTA's slice of a row: n 16-byte words from `words` on, of which the
// first `staged` are in shared memory, and the row's single elements before
// its first 16-byte boundary (rank 0) and after its last (the last rank).
template <class T>
struct Slice {
    static constexpr int kV = 16 / sizeof(T);
    const T* z;             // the row
    int first;              // the slice's first element (of its words)
    int n, staged;
    int single, single_n;   // this CTA's single elements: [single, single + single_n)
    int head;

    __device__ Slice(const DistillArgs& a, int64_t row, int rank) {
        z = static_cast<const T*>(a.logits) + row * a.logits_stride;
        const int vocab = static_cast<int>(a.vocab);
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(z) % 16) / sizeof(T);
        head = mis == 0 ? 0 : kV - mis;
        if (head > vocab) head = vocab;
        const int words = (vocab - head) / kV;
        const int per = (words + a.ranks - 1) / a.ranks;
        const int v0 = rank * per < words ? rank * per : words;
        n = words - v0 < per ? words - v0 : per;
        staged = n < a.stage_words ? n : a.stage_words;
        first = head + v0 * kV;
        // with one rank both ends are its own: then the head is handled with
        // the tail, as head_n() more elements
        single = rank == a.ranks - 1 ? head + words * kV : 0;
        single_n = rank == a.ranks - 1 ? vocab - single : 0;
        if (rank != 0) head = 0;
    }
    __device__ const T* word(int i) const { return z + first + static_cast<int64_t>(i) * kV; }
    // single element j of this CTA (j < head + single_n), as an index of the row
    __device__ int single_at(int j) const { return j < head ? j : single + (j - head); }
    __device__ int singles() const { return head + single_n; }
};

// Maximum or sum of a value over the cluster's workers, for the rows that take
// the difference first.
template <bool MAX>
__device__ float cluster_all(float x, float* red, float* slots, int rank, int ranks) {
    cg::cluster_group cluster = cg::this_cluster();
    x = MAX ? warp_max(x) : warp_sum(x);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = red[0];
    for (int i = 1; i < kWorkerWarps; ++i) x = MAX ? fmaxf(x, red[i]) : x + red[i];
    if (static_cast<int>(threadIdx.x) < ranks)
        cluster.map_shared_rank(slots, threadIdx.x)[rank] = x;
    cluster.sync();
    x = slots[0];
    for (int i = 1; i < ranks; ++i) x = MAX ? fmaxf(x, slots[i]) : x + slots[i];
    return x;
}

// One row's teacher entries in shared memory.
struct Teacher {
    float* p;        // probabilities
    float* z;        // the student's logits there
    int32_t* id;     // -1: absent
};

// The teacher's warp: entries of a row, p, sum p log p and whether there is any.
template <class T>
__device__ void read_teacher(const DistillArgs& a, int64_t row, const Teacher& t, float* terms) {
    const int lane = threadIdx.x % 32;
    const T* z = static_cast<const T*>(a.logits) + row * a.logits_stride;
    const int64_t t0 = row * a.top;
    float best = -kInf;
    for (int k = lane; k < a.top; k += 32) {
        const int32_t id = a.ids[t0 + k];
        const float raw = ld_param(a.teacher, a.teacher_f32, t0 + k);
        const bool in = id >= 0 && id < a.vocab;
        const float l = in ? raw * a.inv_tau : -kInf;
        t.id[k] = in ? id : -1;
        t.z[k] = in ? widen<T>(z[id]) : 0.0f;
        t.p[k] = l;
        best = fmaxf(best, l);
    }
    for (int k = a.top + lane; k < (a.top + 3) / 4 * 4; k += 32) t.id[k] = -1;
    best = warp_max(best);
    const float top = best == -kInf ? 0.0f : best;
    float sum = 0.0f;
    for (int k = lane; k < a.top; k += 32) sum += expf(t.p[k] - top);
    sum = warp_sum(sum);
    const float log_sum = logf(sum), inv = 1.0f / sum;
    float acc = 0.0f;
    for (int k = lane; k < a.top; k += 32) {
        const float l = t.p[k] - top;
        const float p = best == -kInf ? 0.0f : expf(l) * inv;
        if (p != 0.0f) acc += p * (l - log_sum);
        t.p[k] = p;
    }
    acc = warp_sum(acc);
    if (lane == 0) {
        terms[0] = acc;
        terms[1] = best == -kInf ? 0.0f : 1.0f;
    }
    __syncwarp();
}

// The gradient's entries k, k + step, ... that lie in [lo, hi): q - p, equal
// ids added up in the order of the entries and written by the first of them.
template <class T>
__device__ __forceinline__ void patch(const DistillArgs& a, const Teacher& t, T* dz, int lo, int hi,
                                      int k, int step, const Exponent& ex, float s, float w) {
    for (; k < a.top; k += step) {
        const int32_t id = t.id[k];
        if (id < lo || id >= hi) continue;
        float p = 0.0f;
        bool earlier = false;
        for (int j = 0; j < a.top; j += 4) {
            const int4 v = *reinterpret_cast<const int4*>(t.id + j);
            if (v.x != id && v.y != id && v.z != id && v.w != id) continue;
            if (v.x == id) p += t.p[j];
            if (v.y == id) p += t.p[j + 1];
            if (v.z == id) p += t.p[j + 2];
            if (v.w == id) p += t.p[j + 3];
            const int at = v.x == id ? j : v.y == id ? j + 1 : v.z == id ? j + 2 : j + 3;
            earlier |= at < k;
        }
        if (!earlier) dz[id] = narrow<T>(a.tau * w * (ex2(ex.log2q(t.z[k])) / s - p));
    }
}

template <class T, bool GRAD>
__global__ void __launch_bounds__(kRowThreads, 3)
distill_kernel(const __grid_constant__ DistillArgs a) {
    using W = Word<T>;
    constexpr int kV = 16 / sizeof(T);
    constexpr int kP = W::kPairs;
    extern __shared__ __align__(16) uint4 mem[];         // the slice, then two rows of entries
    __shared__ Running sums[2][kMaxCluster * kWorkerWarps];   // written by the cluster's CTAs
    __shared__ float far_red[kRowThreads / 32], far_max[kMaxCluster], far_sum[kMaxCluster];
    __shared__ float terms[2][2];

    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = a.ranks, rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool worker = warp < kWorkerWarps;
    const int64_t stride = gridDim.x / ranks;
    const int top4 = (a.top + 3) / 4 * 4;
    auto teacher_of = [&](int parity) {
        float* base = reinterpret_cast<float*>(mem + a.stage_words) + parity * 3 * top4;
        return Teacher{base, base + top4, reinterpret_cast<int32_t*>(base + 2 * top4)};
    };
    const uint32_t my_mem = static_cast<uint32_t>(__cvta_generic_to_shared(mem)) + 16u * tid;
    const int section = a.section * kWorkers;            // words of a copy group

    // the copies of one group of a row, as one commit group
    auto copy_section = [&](const Slice<T>& sl, int sec) {
        const int end = sec == kSections - 1 ? sl.staged
                                             : min(sl.staged, (sec + 1) * section);
        for (int i = sec * section + tid; i < end; i += kWorkers)
            cp_async16(my_mem + 16u * (i - tid), sl.word(i));
        cp_async_commit();
    };

    int64_t row = blockIdx.x / ranks;
    float w = a.weights != nullptr ? a.weights[row] : 1.0f;
    Slice<T> sl(a, row, rank);
    if (worker && w != 0.0f) {
#pragma unroll
        for (int sec = 0; sec < kSections; ++sec) copy_section(sl, sec);
    }
    if (!worker && w != 0.0f) read_teacher<T>(a, row, teacher_of(0), terms[0]);
    if (ranks > 1) cluster.sync();       // every CTA runs: their memory may be written to

    int parity = 0;           // of the row: the teacher's entries
    int flip = 0;             // of the rows read: the exchanged sums
    for (; row < a.n_rows; row += stride, parity ^= 1) {
        const int64_t next_row = row + stride;
        float next_w = 0.0f;
        if (next_row < a.n_rows) next_w = a.weights != nullptr ? a.weights[next_row] : 1.0f;
        const Teacher t = teacher_of(parity);
        T* dz = GRAD ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
        const bool read = w != 0.0f;
        bool live = false;
        Running r{-kFar, 0.0f};
        if (read) {
            if (worker) {
                const Pair c2 = pair(a.c, a.c);
                Pair s2 = 0;
                auto add_word = [&](uint4 v) {
                    const float t0 = ceilf(W::top(v) * a.c);
                    const float off = fmaxf(r.off, fminf(t0, kFar));
                    const float f = ex2(r.off - off);
                    r.off = off;
                    const Pair m2 = pair(-off, -off);
                    s2 = mul2(s2, pair(f, f));
                    Pair x[kP];
                    W::split(v, x);
#pragma unroll
                    for (int j = 0; j < kP; ++j) s2 = add2(s2, ex2_fma2(x[j], c2, m2));
                };
                int i = tid;
                cp_async_wait<2>();
                for (const int end = min(sl.staged, section); i < end; i += kWorkers)
                    add_word(mem[i]);
                cp_async_wait<1>();
                for (const int end = min(sl.staged, 2 * section); i < end; i += kWorkers)
                    add_word(mem[i]);
                cp_async_wait<0>();
                for (; i < sl.staged; i += kWorkers) add_word(mem[i]);
                for (; i < sl.n; i += kWorkers)
                    add_word(*reinterpret_cast<const uint4*>(sl.word(i)));
                const float2 s = unpair(s2);
                r.s = s.x + s.y;
                for (int j = tid; j < sl.singles(); j += kWorkers) {
                    const float x = widen<T>(sl.z[sl.single_at(j)]);
                    const float off = fmaxf(r.off, fminf(ceilf(x * a.c), kFar));
                    r.s = r.s * ex2(r.off - off) + ex2(__fmaf_rn(x, a.c, -off));
                    r.off = off;
                }
                r = warp_join(r);
                Running* slot = sums[flip] + rank * kWorkerWarps + warp;
                if (lane < ranks) *cluster.map_shared_rank(slot, lane) = r;
            }
            if (ranks > 1) cluster.sync();
            else __syncthreads();
            r = {-kFar, 0.0f};
            for (int i = lane; i < ranks * kWorkerWarps; i += 32) {
                const Running o = sums[flip][i];
                const float off = fmaxf(r.off, o.off);
                r.s = r.s * ex2(r.off - off) + o.s * ex2(o.off - off);
                r.off = off;
            }
            r = warp_join(r);
            flip ^= 1;
            live = terms[parity][1] != 0.0f;
        } else {
            __syncthreads();      // every row has one: entries are kept for two rows
        }
        Exponent ex{a.c, r.off, !(fabsf(r.off) < kFar)};
        if (live && ex.far) {
            float m = -kInf, s = 0.0f;
            auto word_of = [&](int i) {
                return i < sl.staged ? mem[i] : *reinterpret_cast<const uint4*>(sl.word(i));
            };
            if (worker) {
                for (int i = tid; i < sl.n; i += kWorkers) m = fmaxf(m, W::top(word_of(i)));
                for (int j = tid; j < sl.singles(); j += kWorkers)
                    m = fmaxf(m, widen<T>(sl.z[sl.single_at(j)]));
            }
            ex.off = cluster_all<true>(m, far_red, far_max, rank, ranks);
            if (worker) {
                for (int i = tid; i < sl.n; i += kWorkers) {
                    Pair x[kP];
                    W::split(word_of(i), x);
#pragma unroll
                    for (int j = 0; j < kP; ++j) {
                        const float2 v = unpair(x[j]);
                        s += ex2(ex.log2q(v.x)) + ex2(ex.log2q(v.y));
                    }
                }
                for (int j = tid; j < sl.singles(); j += kWorkers)
                    s += ex2(ex.log2q(widen<T>(sl.z[sl.single_at(j)])));
            }
            r.s = cluster_all<false>(s, far_red, far_sum, rank, ranks);
        }
        const Slice<T> next(a, next_row < a.n_rows ? next_row : row, rank);
        if (worker) {
            const float f = live ? a.tau * w / r.s : 0.0f;
            const bool copy = next_w != 0.0f;
            // the slice's gradient from its copy, word by word; then the next
            // row's copy into the word
            auto write_words = [&](auto&& grad_word) {
                T* out = dz + sl.first;
                int i = tid;
#pragma unroll
                for (int sec = 0; sec < kSections; ++sec) {
                    const int limit = sec == kSections - 1 ? a.stage_words : (sec + 1) * section;
                    if (GRAD) {
                        for (const int end = min(sl.staged, limit); i < end; i += kWorkers) {
                            *reinterpret_cast<uint4*>(out + static_cast<int64_t>(i) * kV) =
                                grad_word(mem[i]);
                            if (copy && i < next.staged)
                                cp_async16(my_mem + 16u * (i - tid), next.word(i));
                        }
                    }
                    if (copy) {
                        int j = GRAD ? i : sec * section + tid;
                        for (const int end = min(next.staged, limit); j < end; j += kWorkers)
                            cp_async16(my_mem + 16u * (j - tid), next.word(j));
                        cp_async_commit();
                    }
                }
                if (GRAD) {
                    for (; i < sl.n; i += kWorkers)
                        *reinterpret_cast<uint4*>(out + static_cast<int64_t>(i) * kV) =
                            grad_word(*reinterpret_cast<const uint4*>(sl.word(i)));
                }
            };
            const bool same_grid = !GRAD || ((reinterpret_cast<uintptr_t>(sl.z) ^
                                              reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
            if (same_grid) {
                if (!live) {
                    write_words([](uint4) { return make_uint4(0, 0, 0, 0); });
                } else if (!ex.far) {
                    const Pair c2 = pair(a.c, a.c), f2 = pair(f, f), m2 = pair(-ex.off, -ex.off);
                    write_words([&](uint4 v) {
                        Pair x[kP];
                        W::split(v, x);
#pragma unroll
                        for (int j = 0; j < kP; ++j) x[j] = mul2(ex2_fma2(x[j], c2, m2), f2);
                        return W::join(x);
                    });
                } else {
                    write_words([&](uint4 v) {
                        Pair x[kP];
                        W::split(v, x);
#pragma unroll
                        for (int j = 0; j < kP; ++j) {
                            const float2 y = unpair(x[j]);
                            x[j] = pair(ex2(ex.log2q(y.x)) * f, ex2(ex.log2q(y.y)) * f);
                        }
                        return W::join(x);
                    });
                }
            } else {
                // the gradient's rows lie otherwise on the 16-byte grid: single
                // elements, which other threads have copied
                asm volatile("bar.sync 2, %0;" ::"n"(kWorkers) : "memory");
                const T* held = reinterpret_cast<const T*>(mem);
                const int in_copy = sl.staged * kV;
                for (int i = tid; i < sl.n * kV; i += kWorkers) {
                    float y = 0.0f;
                    if (live)
                        y = ex2(ex.log2q(widen<T>(i < in_copy ? held[i] : sl.z[sl.first + i]))) * f;
                    dz[sl.first + i] = narrow<T>(y);
                }
                asm volatile("bar.sync 2, %0;" ::"n"(kWorkers) : "memory");
                if (copy) {
#pragma unroll
                    for (int sec = 0; sec < kSections; ++sec) copy_section(next, sec);
                }
            }
            if (GRAD) {
                for (int j = tid; j < sl.singles(); j += kWorkers) {
                    const int i = sl.single_at(j);
                    dz[i] = narrow<T>(live ? ex2(ex.log2q(widen<T>(sl.z[i]))) * f : 0.0f);
                }
            }
        } else {
            if (rank == 0) {
                float loss = 0.0f;
                if (live) {
                    // sum_k p_k (log p_k - ln 2 (log2 of the term k)) + log sum
                    float acc = 0.0f;
                    for (int k = lane; k < a.top; k += 32) {
                        if (t.p[k] != 0.0f) acc += t.p[k] * ex.log2q(t.z[k]);
                    }
                    acc = warp_sum(acc);
                    loss = w * a.tau2 * (terms[parity][0] - acc * 0.69314718f + logf(r.s));
                }
                if (lane == 0) a.loss[row] = loss;
            }
            if (next_w != 0.0f)
                read_teacher<T>(a, next_row, teacher_of(parity ^ 1), terms[parity ^ 1]);
        }
        if (GRAD && read) {
            // the CTA's plain values are written: now the teacher's entries
            const int lo = rank == 0 ? 0 : sl.first;
            const int hi = rank == ranks - 1 ? static_cast<int>(a.vocab) : sl.first + sl.n * kV;
            if (a.top <= kPatchAlone) {
                if (worker) {
                    __threadfence_block();
                    asm volatile("bar.arrive 1, %0;" ::"n"(kRowThreads) : "memory");
                } else {
                    asm volatile("bar.sync 1, %0;" ::"n"(kRowThreads) : "memory");
                    if (live) patch(a, t, dz, lo, hi, lane, 32, ex, r.s, w);
                }
            } else {
                __syncthreads();
                if (live) patch(a, t, dz, lo, hi, tid, kRowThreads, ex, r.s, w);
            }
        }
        w = next_w;
        sl = next;
    }
}

// CTAs of a row: enough for its slices to fit three to an SM, and more where
// rows are few, so that a row's read is spread over the GPU.
int ranks_for(int64_t rows, int64_t row_bytes) {
    int ranks = 1;
    while (ranks < kMaxCluster &&
           (row_bytes > static_cast<int64_t>(ranks) * kSliceBytes ||
            (rows * ranks * 2 <= device_sms() && row_bytes > ranks * 8192)))
        ranks *= 2;
    return ranks;
}

// Clusters of a launch's shape that the GPU holds at once; the last shapes
// asked for are kept, per kernel and device.
struct Resident {
    std::mutex lock;
    struct Entry {
        int dev, ranks;
        size_t smem;
        int clusters;
    } kept[16];
    int n = 0;

    cudaError_t get(const void* kernel, const cudaLaunchConfig_t& cfg, int dev, int ranks,
                    int* clusters) {
        std::lock_guard<std::mutex> hold(lock);
        for (const Entry& e : kept) {
            if (e.clusters > 0 && e.dev == dev && e.ranks == ranks &&
                e.smem == cfg.dynamicSmemBytes) {
                *clusters = e.clusters;
                return cudaSuccess;
            }
        }
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMostBytes + 24 * static_cast<int>(kMaxTeacher));
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (*clusters < 1) *clusters = 1;
        kept[n] = {dev, ranks, cfg.dynamicSmemBytes, *clusters};
        n = (n + 1) % 16;
        return cudaSuccess;
    }
};

template <class T, bool GRAD>
cudaError_t launch(DistillArgs a, cudaStream_t stream) {
    static Resident resident;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const auto kernel = distill_kernel<T, GRAD>;
    const int64_t row_bytes = a.vocab * static_cast<int64_t>(sizeof(T));
    a.ranks = ranks_for(a.n_rows, row_bytes);
    const int64_t slice = (row_bytes / 16 + a.ranks - 1) / a.ranks;
    a.stage_words = static_cast<int32_t>(slice < kMostBytes / 16 ? slice : kMostBytes / 16);
    const int per_thread = (a.stage_words + kWorkers - 1) / kWorkers;
    a.section = (per_thread + kSections - 1) / kSections;
    const size_t top4 = (static_cast<size_t>(a.top) + 3) / 4 * 4;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ranks));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.stage_words) * 16 + 24 * top4;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(a.ranks);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaError_t e = resident.get(reinterpret_cast<const void*>(kernel), cfg, dev, a.ranks,
                                     &clusters);
        e != cudaSuccess)
        return e;
    const int64_t n = a.n_rows < clusters ? a.n_rows : clusters;
    cfg.gridDim = dim3(static_cast<unsigned>(n * a.ranks));
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int logits_bytes, cudaStream_t stream) {
    if (logits_bytes == 4)
        return a.grad != nullptr ? launch<float, true>(a, stream) : launch<float, false>(a, stream);
    return a.grad != nullptr ? launch<uint16_t, true>(a, stream)
                             : launch<uint16_t, false>(a, stream);
}

}  // namespace zf
