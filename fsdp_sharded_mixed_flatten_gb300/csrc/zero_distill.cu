// Distillation from a teacher's top logits.  For a row of student logits z
// over the vocabulary and the teacher's entries (id_k, l_k):
//   p = softmax(l / tau) over the entries,  q = softmax(z / tau) over the row,
//   loss = w tau^2 sum_k p_k (log p_k - log q_{id_k}),
//   dloss/dz_v = w tau (q_v - sum_{k: id_k = v} p_k).
//
// A CTA holds a row in shared memory, two CTAs an SM, and works through many
// rows.  DRAM sees one read and one write of the logits:
//   - every worker copies its own 16-byte words with cp.async and is the only
//     one to read them, so no barrier separates copy and use;
//   - it adds up the exponentials as the words arrive; one barrier a row
//     exchanges the warps' sums, the teacher's with the student's;
//   - it forms the gradient from the copy, and into each word it has used up
//     goes the same word of the CTA's next row, so that reads and writes of
//     memory overlap;
//   - warps of their own hold the teacher's entries, one a thread, fetched a row
//     ahead.  The entries of the gradient are written, and the loss added up,
//     after the next row's barrier, when every plain value of the row is there.
// Words beyond shared memory are read again, from L2.  Where rows are fewer
// than SMs a cluster of CTAs takes a row, each a slice, and the sums go through
// distributed shared memory; with many rows that costs more than it gives (a
// cluster barrier waits for the gradient's stores to arrive: 4096 x 50257 took
// 221 us with clusters of one CTA and a split barrier).
//
// Measured, loss and gradient: 4096 x 50257 bf16 with 64 entries 140 us (5.5 TB/s of
// the rows that have a weight), 4096 x 25000 fp32 6.2 TB/s, 8192 x 131072 bf16 with 128
// entries 852 us (5.0 TB/s; its words beyond shared memory come from L2 a second time),
// 1021 x 32003 fp32 55.7 us (4.6 TB/s: 3.4 rounds of 304 CTAs take as long as 4), 16 x
// 50257 the loss alone 8.2 us, as long as the host takes for a call.
//
// Exponentials are 2^(z c - M), c = log2(e) / tau: one fused multiply-add and
// one ex2 each.  M is an integer, ceil(c max z) of what a thread has seen, so
// that moving from one M to another scales by an exact power of two.  The fused
// multiply-add takes the exact z c, M comes from the rounded one, and what lies
// between them is an exponent of two: below kFar a quarter at most, at 2^31 more
// than an fp32 holds.  So M stays within kFar, and rows whose largest c z lies
// beyond (every logit a mask's value, some very large, infinities) take the
// difference first: 2^((z - max z) c).  Logits far below the rest, of whatever
// size, add 0 to a sum at M >= -kFar.
#include "zero_ops.cuh"

#include <cooperative_groups.h>

#include <mutex>

namespace cg = cooperative_groups;

namespace zf {

namespace {

constexpr int kMaxCluster = 8;
constexpr int kSections = 3;                     // copy groups of a row
constexpr int kRing = 4;                         // rows whose entries are kept
constexpr int kRowWarps = 16;                    // of a CTA, two of them an SM
constexpr int kMostBytes = 110 * 1024;           // of a CTA of 16 warps: words and entries
constexpr int kShortRow = 48 * 1024;             // rows up to this take one CTA
constexpr float kInf = __builtin_huge_valf();
constexpr float kFar = 1 << 22;                  // of |c z|, whose ulp is a half there
constexpr float kNone = -2 * kFar;               // off of a sum without terms

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Where a row does not fit shared memory (!WHOLE), copies and stores carry an L2
// policy: what is not read again leaves L2 first, so that the words that are stay.
__device__ __forceinline__ uint64_t l2_policy() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
template <bool WHOLE>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint64_t policy) {
    if (WHOLE) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        return;
    }
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(src), "l"(policy)
                 : "memory");
}
template <bool WHOLE>
__device__ __forceinline__ void store16(void* dst, uint4 v, uint64_t policy) {
    if (WHOLE) {
        *static_cast<uint4*>(dst) = v;
        return;
    }
    asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(dst), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w), "l"(policy)
                 : "memory");
}
// Words beyond shared memory: kept in L2 from the first reading, let go at the
// second, which is the gradient's.  (The loss alone reads them once, and has them
// kept all the same.)
__device__ __forceinline__ uint64_t l2_keep() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint4 load16(const void* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.b32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy)
                 : "memory");
    return v;
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
    __device__ __forceinline__ void raise(float to) {
        if (to > off) {
            s *= ex2(off - to);
            off = to;
        }
    }
};

// Joined over a warp: the largest off, every sum scaled to it.
__device__ __forceinline__ Running warp_join(Running r) {
    float off;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(off) : "f"(r.off));
    return {off, warp_sum(r.s * ex2(r.off - off))};
}

// The exponents of the row's or its entries' exponentials: near: z c - off,
// rounded once, so that logits far from zero lose no digits of their
// differences; far: (z - off) c.
struct Exponent {
    float c, off;
    bool far;
    __device__ __forceinline__ float of(float z) const {
        return far ? (z - off) * c : __fmaf_rn(z, c, -off);
    }
};

// This CTA's slice of a row, elements [lo, hi): n 16-byte words from element
// `first` on, of which the first `staged` are in shared memory, and single
// elements before (rank 0: up to the row's first 128-byte boundary) and after
// them (the last rank): fewer than the workers.
template <class T>
struct Slice {
    static constexpr int kV = 16 / sizeof(T);
    const T* z;             // the row
    int first, n, staged, lo, hi;

    __device__ Slice(const DistillArgs& a, const T* at, int rank) {
        z = at;
        const int vocab = static_cast<int>(a.vocab);
        // words from a 128-byte boundary on: a warp's 512 bytes are whole lines
        // (rows that start 16 bytes off one took 10 % longer)
        const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(z) % 128) / sizeof(T);
        const int head = min(vocab, mis == 0 ? 0 : 8 * kV - mis);
        const int words = (vocab - head) / kV;
        const int per = (words + a.ranks - 1) >> a.rank_shift;
        const int v0 = min(rank * per, words);
        n = min(words - v0, per);
        staged = min(n, a.stage_words);
        first = head + v0 * kV;
        lo = rank == 0 ? 0 : first;
        hi = rank == a.ranks - 1 ? vocab : first + n * kV;
    }
    __device__ const T* word(int i) const { return z + first + static_cast<int64_t>(i) * kV; }
    __device__ int singles() const { return hi - lo - n * kV; }
    __device__ int single_at(int j) const { return lo + j < first ? lo + j : lo + j + n * kV; }
};

// Maximum or sum of a value over the cluster's threads, for the rows that take
// the difference first.
template <bool MAX>
__device__ float cluster_all(float x, float* red, float* slots, int rank, int ranks) {
    cg::cluster_group cluster = cg::this_cluster();
    x = MAX ? warp_max(x) : warp_sum(x);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = red[0];
    for (int i = 1; i < static_cast<int>(blockDim.x) / 32; ++i)
        x = MAX ? fmaxf(x, red[i]) : x + red[i];
    if (static_cast<int>(threadIdx.x) < ranks)
        cluster.map_shared_rank(slots, threadIdx.x)[rank] = x;
    cluster.sync();
    x = slots[0];
    for (int i = 1; i < ranks; ++i) x = MAX ? fmaxf(x, slots[i]) : x + slots[i];
    return x;
}

// The teacher's entries of a row in shared memory: those in this CTA's slice.
struct Entries {
    int32_t* id;     // -1: absent, or in another CTA's slice
    float* l;        // the teacher's logit; later w tau p
    float* z;        // the student's logit there; later w tau q
};

// An entry that a thread holds.
struct Entry {
    int32_t id;
    float l, z;
};

// WW warps of workers, which hold the slice, and EW of the teacher's entries.
// WHOLE: every word of a row fits the CTA's shared memory.  HASH: how equal ids
// are found.
template <class T, bool GRAD, int WW, int EW, bool WHOLE, bool HASH>
__global__ void __launch_bounds__(32 * (WW + EW), 32 / (WW + EW))
distill_kernel(const __grid_constant__ DistillArgs a) {
    using W = Word<T>;
    constexpr int kV = 16 / sizeof(T);
    constexpr int kP = W::kPairs;
    constexpr int kWorkers = 32 * WW, kEntryThreads = 32 * EW;
    extern __shared__ __align__(16) uint4 mem[];      // the slice, then kRing rows of entries
    // written by the cluster's CTAs
    __shared__ Running sums[2][kMaxCluster * WW], entry_sums[2][kMaxCluster * EW];
    __shared__ float losses[kRing][kMaxCluster * EW];                       // of rank 0
    __shared__ float far_red[WW + EW], far_slots[3][kMaxCluster];
    __shared__ int64_t row_of[kRing];
    __shared__ float weight_of[kRing];
    __shared__ int equal[kRing];        // the last row (its number) there with equal ids

    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = a.ranks, rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool worker = warp < WW;
    const int et = tid - kWorkers;                       // of the entries' threads
    const int64_t stride = gridDim.x / ranks;
    const int top4 = (a.top + 3) / 4 * 4;
    const int section = a.section * kWorkers;            // words of a copy group
    const uint64_t policy = WHOLE ? 0 : l2_policy();
    const uint32_t my_mem = static_cast<uint32_t>(__cvta_generic_to_shared(mem)) + 16u * tid;

    auto entries_of = [&](int number) {
        int32_t* base =
            reinterpret_cast<int32_t*>(mem + a.stage_words) + (number % kRing) * 3 * top4;
        return Entries{base, reinterpret_cast<float*>(base + top4),
                       reinterpret_cast<float*>(base + 2 * top4)};
    };
    auto slice_of = [&](int64_t row) {
        return Slice<T>(a, static_cast<const T*>(a.logits) + row * a.logits_stride, rank);
    };
    auto copy_row = [&](const Slice<T>& sl) {
#pragma unroll
        for (int sec = 0; sec < kSections; ++sec) {
            const int end = sec == kSections - 1 ? sl.staged
                                                 : min(sl.staged, (sec + 1) * section);
            for (int i = sec * section + tid; i < end; i += kWorkers)
                cp_async16<WHOLE>(my_mem + 16u * (i - tid), sl.word(i), policy);
            cp_async_commit();
        }
    };
    // Entry k of a row.
    auto fetch_entry = [&](int64_t row, int k) {
        const int64_t at = row * a.top + k;
        return Entry{a.ids[at], ld_param(a.teacher, a.teacher_f32, at), 0.0f};
    };
    // the student's logit of an entry in this CTA's slice; others are absent
    auto fetch_logit = [&](const Slice<T>& sl, Entry& e) {
        if (e.id >= sl.lo && e.id < sl.hi) e.z = widen<T>(sl.z[e.id]);
        else e.id = -1;
    };

    // The next row from `row` on that has a weight (n_rows or more: none); the
    // rows before it get their zeros.
    auto next_row = [&](int64_t row, float& w) {
        for (; row < a.n_rows; row += stride) {
            w = a.weights != nullptr ? a.weights[row] : 1.0f;
            if (w != 0.0f) break;
            if (rank == 0 && tid == 0) a.loss[row] = 0.0f;
            if (GRAD && worker) {
                T* dz = static_cast<T*>(a.grad) + row * a.grad_stride;
                const Slice<T> sl(a, dz, rank);
                const uint4 zero = make_uint4(0, 0, 0, 0);
                for (int i = tid; i < sl.n; i += kWorkers)
                    *reinterpret_cast<uint4*>(dz + sl.first + static_cast<int64_t>(i) * kV) = zero;
                if (tid < sl.singles()) dz[sl.single_at(tid)] = narrow<T>(0.0f);
            }
        }
        return row;
    };

    // The exponentials of the row held, this worker's part; `single`: its single
    // element, if it has one.
    float single = 0.0f;
    auto add_up = [&](const Slice<T>& sl) {
        const bool has_single = tid < sl.singles();
        single = widen<T>(sl.z[has_single ? sl.single_at(tid) : 0]);
        Running r{-kFar, 0.0f};
        const Pair c2 = pair(a.c, a.c);
        Pair s0 = 0, s1 = 0;
        auto raise = [&](float top) {
            const float t = top * a.c;
            if (t > r.off) {
                const float off = fminf(ceilf(t), kFar);
                const float f = ex2(r.off - off);
                r.off = off;
                s0 = mul2(s0, pair(f, f));
                s1 = mul2(s1, pair(f, f));
            }
        };
        auto add_word = [&](uint4 v) {
            raise(W::top(v));
            const Pair m2 = pair(-r.off, -r.off);
            Pair x[kP];
            W::split(v, x);
#pragma unroll
            for (int j = 0; j < kP; j += 2) {
                s0 = add2(s0, ex2_fma2(x[j], c2, m2));
                s1 = add2(s1, ex2_fma2(x[j + 1], c2, m2));
            }
        };
        auto add_words = [&](uint4 u, uint4 v) {
            raise(fmaxf(W::top(u), W::top(v)));
            const Pair m2 = pair(-r.off, -r.off);
            Pair x[kP], y[kP];
            W::split(u, x);
            W::split(v, y);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                s0 = add2(s0, ex2_fma2(x[j], c2, m2));
                s1 = add2(s1, ex2_fma2(y[j], c2, m2));
            }
        };
        int i = tid;
        const uint4* at = mem + tid;
        auto add_to = [&](int end) {
            for (; i + kWorkers < end; i += 2 * kWorkers, at += 2 * kWorkers)
                add_words(at[0], at[kWorkers]);
            if (i < end) {
                add_word(*at);
                i += kWorkers;
                at += kWorkers;
            }
        };
        cp_async_wait<2>();
        add_to(min(sl.staged, section));
        cp_async_wait<1>();
        add_to(min(sl.staged, 2 * section));
        cp_async_wait<0>();
        add_to(sl.staged);
        if (!WHOLE && i < sl.n) {
            // words beyond shared memory, four loads under way
            const uint64_t keep = l2_keep();
            const uint4* far = reinterpret_cast<const uint4*>(sl.word(i));
            for (; i + 3 * kWorkers < sl.n; i += 4 * kWorkers, far += 4 * kWorkers) {
                const uint4 v0 = load16(far, keep), v1 = load16(far + kWorkers, keep),
                            v2 = load16(far + 2 * kWorkers, keep),
                            v3 = load16(far + 3 * kWorkers, keep);
                add_words(v0, v1);
                add_words(v2, v3);
            }
            for (; i < sl.n; i += kWorkers, far += kWorkers) add_word(load16(far, keep));
        }
        const float2 both = unpair(add2(s0, s1));
        r.s = both.x + both.y;
        if (has_single) {
            r.raise(fminf(ceilf(single * a.c), kFar));
            r.s += ex2(__fmaf_rn(single, a.c, -r.off));
        }
        return warp_join(r);
    };

    // A row's entries to shared memory, and their sum of this warp.
    auto take_entries = [&](int64_t row, const Slice<T>& sl, const Entry& mine, int number) {
        const Entries t = entries_of(number);
        Running r{kNone, 0.0f};
        for (int k = et; k < top4; k += kEntryThreads) {
            Entry e = mine;
            if (k >= kEntryThreads) {
                e = k < a.top ? fetch_entry(row, k) : Entry{-1, 0.0f, 0.0f};
                fetch_logit(sl, e);
            }
            if (k >= a.top || e.l == -kInf) e.id = -1;
            if (e.id >= 0) {
                r.raise(fminf(fmaxf(ceilf(e.l * a.c), -kFar), kFar));
                r.s += ex2(__fmaf_rn(e.l, a.c, -r.off));
            }
            t.id[k] = e.id;
            t.l[k] = e.l;
            t.z[k] = e.z;
        }
        return warp_join(r);
    };

    // Whether an id of this thread's entries is another entry's too, by hashing:
    // every entry puts its number into a hashed place and reads who is there:
    // itself, an equal id, or another one; the last try again in a second table,
    // and what is left even then (1 of 100) compares with all.
    // The tables lie where row number + 2 will have its entries: those of row
    // number - 2 are done with, and a barrier of the row comes before either.
    auto any_equal_hashed = [&](const Entries& t, int number) {
        bool same = false;
        uint16_t* table = reinterpret_cast<uint16_t*>(entries_of(number + 2).id);
        const uint32_t size = 3 * static_cast<uint32_t>(top4);       // of one table
        uint32_t open = 0xFFFFFFFFu;                                 // a bit for each entry
#pragma unroll
        for (int stage = 0; stage < 2; ++stage) {
            auto place = [&](int32_t id) {
                const uint32_t h = static_cast<uint32_t>(id) * (stage == 0 ? 2654435761u : 2246822519u);
                return table + stage * size + __umulhi(h, size);
            };
            for (int k = et, r = 0; k < a.top; k += kEntryThreads, ++r) {
                const int32_t id = t.id[k];
                if (id < 0) open &= ~(1u << r);
                if ((open >> r) & 1u) *place(id) = static_cast<uint16_t>(k);
            }
            if (EW == 1) __syncwarp();
            else asm volatile("bar.sync 2, %0;" ::"n"(kEntryThreads) : "memory");
            for (int k = et, r = 0; k < a.top; k += kEntryThreads, ++r) {
                if (!((open >> r) & 1u)) continue;
                const int32_t id = t.id[k];
                const int there = *place(id);
                const bool equal_id = there != k && t.id[there] == id;
                same |= equal_id;
                if (there == k || equal_id) open &= ~(1u << r);
            }
        }
        for (int k = et, r = 0; k < a.top; k += kEntryThreads, ++r) {
            if (!((open >> r) & 1u)) continue;
            for (int j = 0; j < a.top; ++j) same |= j != k && t.id[j] == t.id[k];
        }
        return same;
    };

    // This warp's sum of row `number` to the CTAs of the cluster.
    auto publish = [&](const Running& r, int number) {
        if (lane < ranks) {
            if (worker) cluster.map_shared_rank(sums[number & 1], lane)[rank * WW + warp] = r;
            else cluster.map_shared_rank(entry_sums[number & 1], lane)[rank * EW + warp - WW] = r;
        }
    };
    auto join_all = [&](const Running* from, int n, float none) {
        Running r{none, 0.0f};
        for (int j = lane; j < n; j += 32) {
            const Running o = from[j];
            r.raise(o.off);
            r.s += o.s * ex2(o.off - r.off);
        }
        return warp_join(r);
    };

    // The entries' threads, after every plain value of row `number` is
    // written: its entries of the gradient, and its loss.
    auto finish = [&](int number) {
        if (number < 0) return;
        const int f = number % kRing;
        const int64_t row = row_of[f];
        if (GRAD) {
            T* dz = static_cast<T*>(a.grad) + row * a.grad_stride;
            const Entries t = entries_of(number);
            const bool equal_ids = equal[f] == number;
            for (int k = et; k < a.top; k += kEntryThreads) {
                const int32_t id = t.id[k];
                if (id < 0) continue;
                float p = t.l[k];
                if (equal_ids) {
                    // equal ids add up in the order of the entries; the first writes
                    p = 0.0f;
                    bool first = true;
                    for (int j = 0; j < a.top; ++j) {
                        if (t.id[j] != id) continue;
                        first &= j >= k;
                        p += t.l[j];
                    }
                    if (!first) continue;
                }
                dz[id] = narrow<T>(t.z[k] - p);
            }
        }
        if (rank == 0 && warp == WW) {
            float loss = 0.0f;
            for (int i = lane; i < ranks * EW; i += 32) loss += losses[f][i];
            loss = warp_sum(loss);
            // (one temperature after the other: their square may be below fp32)
            if (lane == 0) a.loss[row] = weight_of[f] * a.tau * (a.tau * (0.69314718f * loss));
        }
    };

    float w = 0.0f;
    int64_t row = next_row(blockIdx.x / ranks, w);
    if (row >= a.n_rows) return;                 // none with a weight: for all of the cluster
    Slice<T> sl = slice_of(row);
    Entry mine{-1, 0.0f, 0.0f};
    if (worker) {
        copy_row(sl);
    } else if (et < a.top) {
        mine = fetch_entry(row, et);
        fetch_logit(sl, mine);
    }
    if (tid < kRing) equal[tid] = -1;
    if (ranks > 1) cluster.sync();               // every CTA runs: their memory may be written to
    auto barrier = [&] {
        if (ranks > 1) cluster.sync();
        else __syncthreads();
    };

    int number = 0;                              // of this row among the cluster's
    for (;; ++number) {
        const int buf = number & 1;
        const Entries t = entries_of(number);
        publish(worker ? add_up(sl) : take_entries(row, sl, mine, number), number);
        barrier();
        Running r = join_all(sums[buf], ranks * WW, -kFar);
        Exponent ex{a.c, r.off, !(fabsf(r.off) < kFar)};
        Running rt{kNone, 0.0f};
        float entry_off = kNone;
        for (int j = lane; j < ranks * EW; j += 32) entry_off = fmaxf(entry_off, entry_sums[buf][j].off);
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(entry_off) : "f"(entry_off));
        const bool live = entry_off != kNone;         // the row has an entry
        const bool far_entries = live && !(fabsf(entry_off) < kFar);
        if (!worker) {
            rt = join_all(entry_sums[buf], ranks * EW, kNone);
            finish(number - 1);
        }
        if (live && ex.far) {
            float m = -kInf;
            auto word_of = [&](int j) {
                return j < sl.staged ? mem[j] : *reinterpret_cast<const uint4*>(sl.word(j));
            };
            if (worker) {
                for (int j = tid; j < sl.n; j += kWorkers) m = fmaxf(m, W::top(word_of(j)));
                if (tid < sl.singles()) m = fmaxf(m, single);
            }
            ex.off = cluster_all<true>(m, far_red, far_slots[0], rank, ranks);
            float sum = 0.0f;
            if (worker) {
                for (int j = tid; j < sl.n; j += kWorkers) {
                    Pair x[kP];
                    W::split(word_of(j), x);
#pragma unroll
                    for (int p = 0; p < kP; ++p) {
                        const float2 v = unpair(x[p]);
                        sum += ex2(ex.of(v.x)) + ex2(ex.of(v.y));
                    }
                }
                if (tid < sl.singles()) sum += ex2(ex.of(single));
            }
            r.s = cluster_all<false>(sum, far_red, far_slots[1], rank, ranks);
        }
        Exponent entry_ex{a.c, rt.off, far_entries};
        if (far_entries) {
            float m = -kInf;
            if (!worker) {
                for (int k = et; k < a.top; k += kEntryThreads) {
                    if (t.id[k] >= 0) m = fmaxf(m, t.l[k]);
                }
            }
            entry_ex.off = cluster_all<true>(m, far_red, far_slots[2], rank, ranks);
            float sum = 0.0f;
            if (!worker) {
                for (int k = et; k < a.top; k += kEntryThreads) {
                    if (t.id[k] >= 0) sum += ex2(entry_ex.of(t.l[k]));
                }
            }
            rt.s = cluster_all<false>(sum, far_red, far_slots[0], rank, ranks);
        }
        float next_w = 0.0f;
        const int64_t next = next_row(row + stride, next_w);
        const bool copy = next < a.n_rows;
        const Slice<T> next_sl = slice_of(copy ? next : row);
        const float f = live ? a.tau * w / r.s : 0.0f;
        if (!worker) {
            if (copy && et < a.top) mine = fetch_entry(next, et);
            // the entries: w tau q and w tau p, and their part of the loss
            if (et == 0) {
                row_of[number % kRing] = row;
                weight_of[number % kRing] = w;
            }
            float loss = 0.0f;
            const float log_s = log2f(r.s), log_t = log2f(rt.s);
            const float inv_t = 1.0f / rt.s, tau_w = a.tau * w;
            for (int k = et; k < a.top; k += kEntryThreads) {
                const int32_t id = t.id[k];
                if (id < 0) continue;
                const float lp = entry_ex.of(t.l[k]), p = ex2(lp) * inv_t, lq = ex.of(t.z[k]);
                if (p != 0.0f) loss += p * ((lp - log_t) - (lq - log_s));
                t.l[k] = tau_w * p;
                t.z[k] = ex2(lq) * f;
                if (!GRAD || HASH) continue;
                int same = 0;
                for (int j = 0; j < top4; j += 4) {
                    const int4 v = *reinterpret_cast<const int4*>(t.id + j);
                    same += (v.x == id) + (v.y == id) + (v.z == id) + (v.w == id);
                }
                if (same > 1) equal[number % kRing] = number;
            }
            if (GRAD && HASH && any_equal_hashed(t, number)) equal[number % kRing] = number;
            loss = warp_sum(loss);
            if (lane == 0)
                cluster.map_shared_rank(losses[number % kRing], 0)[rank * EW + warp - WW] = loss;
            if (copy && et < a.top) fetch_logit(next_sl, mine);
        } else {
            // the slice's gradient from its copy, word by word, and the copy of
            // the next row into the words used up
            T* dz = GRAD ? static_cast<T*>(a.grad) + row * a.grad_stride : nullptr;
            auto write_words = [&](auto&& grad_word) {
                uint4* out = reinterpret_cast<uint4*>(dz + sl.first) + tid;
                const uint4* from = reinterpret_cast<const uint4*>(next_sl.word(0)) + tid;
                const uint4* at = mem + tid;
                uint32_t to = my_mem;
                int i = tid;
                const int n_copy = copy ? next_sl.staged : 0;
#pragma unroll
                for (int sec = 0; sec < kSections; ++sec) {
                    const int limit = sec == kSections - 1 ? a.stage_words : (sec + 1) * section;
                    const int end = GRAD ? min(sl.staged, limit) : 0;
                    for (; i + kWorkers < min(end, n_copy); i += 2 * kWorkers) {
                        const uint4 v0 = at[0], v1 = at[kWorkers];
                        store16<WHOLE>(out, grad_word(v0), policy);
                        store16<WHOLE>(out + kWorkers, grad_word(v1), policy);
                        cp_async16<WHOLE>(to, from, policy);
                        cp_async16<WHOLE>(to + 16 * kWorkers, from + kWorkers, policy);
                        at += 2 * kWorkers;
                        out += 2 * kWorkers;
                        from += 2 * kWorkers;
                        to += 32 * kWorkers;
                    }
                    for (; i < max(end, min(n_copy, limit)); i += kWorkers) {
                        if (i < end) store16<WHOLE>(out, grad_word(*at), policy);
                        if (i < n_copy) cp_async16<WHOLE>(to, from, policy);
                        at += kWorkers;
                        out += kWorkers;
                        from += kWorkers;
                        to += 16 * kWorkers;
                    }
                    if (copy) cp_async_commit();
                }
                if (!WHOLE && GRAD && sl.staged < sl.n) {
                    // a shared word beyond the slice's own may have been passed
                    i = (sl.staged - tid + kWorkers - 1) / kWorkers * kWorkers + tid;
                    out = reinterpret_cast<uint4*>(dz + sl.first) + i;
                    const uint4* far = reinterpret_cast<const uint4*>(sl.word(i));
                    for (; i + 3 * kWorkers < sl.n; i += 4 * kWorkers) {
                        const uint4 v0 = load16(far, policy), v1 = load16(far + kWorkers, policy),
                                    v2 = load16(far + 2 * kWorkers, policy),
                                    v3 = load16(far + 3 * kWorkers, policy);
                        store16<WHOLE>(out, grad_word(v0), policy);
                        store16<WHOLE>(out + kWorkers, grad_word(v1), policy);
                        store16<WHOLE>(out + 2 * kWorkers, grad_word(v2), policy);
                        store16<WHOLE>(out + 3 * kWorkers, grad_word(v3), policy);
                        far += 4 * kWorkers;
                        out += 4 * kWorkers;
                    }
                    for (; i < sl.n; i += kWorkers, far += kWorkers, out += kWorkers)
                        store16<WHOLE>(out, grad_word(load16(far, policy)), policy);
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
                            x[j] = pair(ex2(ex.of(y.x)) * f, ex2(ex.of(y.y)) * f);
                        }
                        return W::join(x);
                    });
                }
            } else {
                // the gradient's rows lie otherwise on the 16-byte grid: single
                // elements, which other workers have copied
                asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory");
                const T* elements = reinterpret_cast<const T*>(mem);
                const int in_copy = sl.staged * kV;
                for (int i = tid; i < sl.n * kV; i += kWorkers) {
                    const float z = widen<T>(i < in_copy ? elements[i] : sl.z[sl.first + i]);
                    dz[sl.first + i] = narrow<T>(live ? ex2(ex.of(z)) * f : 0.0f);
                }
                asm volatile("bar.sync 1, %0;" ::"n"(kWorkers) : "memory");
                if (copy) copy_row(next_sl);
            }
            if (GRAD) {
                if (tid < sl.singles())
                    dz[sl.single_at(tid)] = narrow<T>(live ? ex2(ex.of(single)) * f : 0.0f);
            }
        }
        if (!copy) break;
        row = next;
        w = next_w;
        sl = next_sl;
    }
    barrier();
    if (!worker) finish(number);
}

// CTAs of a row: more than one only where the rows leave SMs idle even so, and a
// row is long enough to pay for the cluster's barriers.  In us by CTAs of a row (1,
// 2, 4, 8), bf16, 32 entries:
//     8 rows of  18000   8.4   9.2   9.2   9.0
//     8 rows of  50257  10.9  10.9  10.3   9.1
//    38 rows of  50257  11.0  11.0  10.9  14.8
//    76 rows of  50257  11.0  12.7  14.9  19.1
//     8 rows of 131072  17.2  15.0  10.9  10.3
//    76 rows of 131072  19.0  17.0  19.0  21.2
// (Several rows a cluster, to even out the last round of 1021 x 32003 in fp32,
// took 134 us instead of 56: its barrier waits for the gradient's stores.)
int ranks_for(int64_t rows, int64_t row_bytes, int sms) {
    if (row_bytes <= kShortRow) return 1;
    int ranks = 1;
    while (ranks < kMaxCluster && rows * ranks * 2 <= sms) ranks *= 2;
    return ranks == 2 && row_bytes <= kMostBytes ? 1 : ranks;
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
                                             kMostBytes);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (*clusters < 1) *clusters = 1;
        kept[n] = {dev, ranks, cfg.dynamicSmemBytes, *clusters};
        n = (n + 1) % 16;
        return cudaSuccess;
    }
};

// Bytes of a row's words in the shared memory of a CTA of `warps`, beside the entries.
int64_t room_for(int warps, int64_t top) {
    return (kMostBytes * warps / kRowWarps - (top + 3) / 4 * 4 * 12 * kRing) / 16 * 16;
}

// Whether a kernel finds equal ids by hashing: from 64 steps of comparing a
// thread on.  8192 rows of 4000 bf16 in us, comparing / hashing: 64 entries 58 / 60,
// 128 entries 86 / 77, 256 entries 168 / 119.  Not where words are read again, with
// time to compare meanwhile: 4096 x 131072 with 256 entries 461 / 495.  (Ids in one
// step; distinct ids at random take 143 us with 256 entries.)
bool hashes(int entry_warps, int64_t top, bool whole) {
    const int64_t rounds = (top + 32 * entry_warps - 1) / (32 * entry_warps);
    return whole && rounds * ((top + 3) / 4) >= 64;
}

template <class T, bool GRAD, int WW, int EW>
cudaError_t launch_shape(DistillArgs a, cudaStream_t stream) {
    static Resident resident[3];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const int64_t row_bytes = a.vocab * static_cast<int64_t>(sizeof(T));
    a.rank_shift = 0;
    while ((1 << a.rank_shift) < a.ranks) ++a.rank_shift;
    const int64_t slice = (row_bytes / 16 + a.ranks - 1) / a.ranks;
    const int64_t entries = (static_cast<int64_t>(a.top) + 3) / 4 * 4 * 12 * kRing;
    const int64_t room = room_for(WW + EW, a.top) / 16;
    a.stage_words = static_cast<int32_t>(slice < room ? slice : room);
    const bool whole = slice <= room;
    auto kernel = distill_kernel<T, GRAD, WW, EW, true, false>;
    int which = 0;
    if constexpr (WW + EW == kRowWarps) {        // smaller CTAs take whole rows alone
        if (!whole) {
            kernel = distill_kernel<T, GRAD, WW, EW, false, false>;
            which = 1;
        }
    }
    if constexpr (GRAD && WW != kRowWarps - 2) {     // that one has 64 entries at most
        if (hashes(EW, a.top, whole)) {
            kernel = distill_kernel<T, GRAD, WW, EW, true, true>;
            which = 2;
        }
    }
    const int per_thread = (a.stage_words + 32 * WW - 1) / (32 * WW);
    a.section = (per_thread + kSections - 1) / kSections;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.ranks));
    cfg.blockDim = dim3(32 * (WW + EW));
    cfg.dynamicSmemBytes = static_cast<size_t>(a.stage_words * 16 + entries);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(a.ranks);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaError_t e = resident[which].get(reinterpret_cast<const void*>(kernel), cfg, dev,
                                               a.ranks, &clusters);
        e != cudaSuccess)
        return e;
    const int64_t n = a.n_rows < clusters ? a.n_rows : clusters;
    cfg.gridDim = dim3(static_cast<unsigned>(n * a.ranks));
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Shorter rows take smaller CTAs, more to an SM, where there are enough of them:
// what a row costs besides its words then overlaps with more other rows'.  1500
// rows of 4000 bf16: 14.8 us with CTAs of 4 warps, 25.3 with 16 (8192 rows: 48, with
// 8 warps 73); 1500 rows of 18000: 29.8 us with 8 warps, 35.6 with 16.  64 rows of 9000
// with 256 entries: 14.2 us with 4 warps, 10.9 with 16.
template <class T, bool GRAD>
cudaError_t launch(DistillArgs a, cudaStream_t stream) {
    const int64_t row_bytes = a.vocab * static_cast<int64_t>(sizeof(T));
    int sms = 0;
    if (cudaError_t e = device_sms(&sms); e != cudaSuccess) return e;
    const bool many = a.n_rows > 2 * sms;
    a.ranks = 1;
    if (row_bytes <= room_for(4, a.top) && many)
        return launch_shape<T, GRAD, 3, 1>(a, stream);
    if (row_bytes <= room_for(8, a.top) && many)
        return launch_shape<T, GRAD, 6, 2>(a, stream);
    a.ranks = ranks_for(a.n_rows, row_bytes, sms);
    // more entries than two warps hold cost the row's critical path: 4096 x 50257
    // with 128 of them 148 us with four warps, 158 with two (with 64 of 131072
    // 427 and 415)
    if (a.top > 64) return launch_shape<T, GRAD, kRowWarps - 4, 4>(a, stream);
    return launch_shape<T, GRAD, kRowWarps - 2, 2>(a, stream);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int logits_bytes, cudaStream_t stream) {
    if (logits_bytes == 4)
        return a.grad != nullptr ? launch<float, true>(a, stream) : launch<float, false>(a, stream);
    return a.grad != nullptr ? launch<uint16_t, true>(a, stream)
                             : launch<uint16_t, false>(a, stream);
}

}  // namespace zf
