// Token table: y[t] = s W[id_t], and its gradient dW[v] = s sum_{t: id_t = v} dy[t],
// summed in fp32 in the order of the tokens and rounded once.  Ids outside
// [0, vocab) give a zero row and no gradient.
//
// The gradient sorts the tokens by id (stable, so the order within an id is
// the order of the tokens, whatever the machine does), then adds up runs of
// equal ids:
//   sort launch: one cluster of 8 CTAs runs a radix sort of (id, token), 2 to
//     4 passes of at most 9 bits; the other clusters write zeros to the rows
//     that no token has.
//   sum launch: a warp takes kChunk sorted places and 256 columns.  A run
//     inside the chunk is added up and written; a run over several chunks
//     leaves one partial row per chunk in the workspace, and the chunk that
//     finishes last adds the partials in chunk order.  No order depends on
//     timing, so neither does any result.
// Few tokens take one launch instead, of buckets (below).
//
// Where every row is written, most of the time goes into zeros: 65536 tokens of
// 4096 bf16 columns into 131072 rows take 322 us (1.6 GB, 5.0 TB/s), 174 to 182 us of
// them the sort launch with 0.90 GB of zeros (5.1 TB/s; a fill runs at 7.5), 137 to
// 140 the sums.  Writing the zeros from CTAs of the
// sum launch, beside its reads, was slower: 408 us instead of 325 then.
#include "zero_ops.cuh"
#include "zero_plan.cuh"

#include <cooperative_groups.h>

#include <mutex>

namespace cg = cooperative_groups;

namespace zf {

namespace {

// -------------------------------------------------------------- lookup ------

__device__ __forceinline__ int64_t ld_id(const void* ids, int id64, int64_t t) {
    return id64 ? static_cast<const int64_t*>(ids)[t]
                : static_cast<int64_t>(static_cast<const int32_t*>(ids)[t]);
}

// A warp takes R tokens and 32 N packs of columns: R N loads are under way at
// once, without conditions (an id outside the table reads row 0, a column beyond
// the row column 0).  One element a thread, its place found by division, took
// 58.7 us for 16384 x 1259 in fp32 from an odd element on, so it takes 29.2; 16384 x
// 768 bf16 8.7 us instead of 12.8 where L2 holds the rows, 10.7 from memory.
template <class W, class Y, int VEC, int R, int N>
__global__ void __launch_bounds__(256) embed_kernel(const __grid_constant__ EmbedArgs a) {
    const int lane = threadIdx.x;
    const int64_t per_cta = R * static_cast<int64_t>(blockDim.y);
    const int64_t width = 32 * N * VEC;
    for (int64_t col0 = blockIdx.y * width; col0 < a.dim; col0 += gridDim.y * width) {
        for (int64_t t0 = blockIdx.x * per_cta + R * threadIdx.y; t0 < a.n_tokens;
             t0 += gridDim.x * per_cta) {
            int64_t id[R];
#pragma unroll
            for (int r = 0; r < R; ++r)
                id[r] = ld_id(a.ids, a.id64, t0 + r < a.n_tokens ? t0 + r : a.n_tokens - 1);
            Pack<W, VEC> p[R][N];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool known = id[r] >= 0 && id[r] < a.vocab;
                const W* row = static_cast<const W*>(a.weight) + (known ? id[r] : 0) * a.dim;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int64_t c = col0 + (j * 32 + lane) * VEC;
                    p[r][j] = ld_pack<W, VEC>(row + (c < a.dim ? c : 0));
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (t0 + r >= a.n_tokens) break;
                const bool known = id[r] >= 0 && id[r] < a.vocab;
                Y* out = static_cast<Y*>(a.out) + (t0 + r) * a.out_stride;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int64_t c = col0 + (j * 32 + lane) * VEC;
                    if (c >= a.dim) continue;
                    float y[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        y[e] = known ? widen<W>(p[r][j].x[e]) * a.scale : 0.0f;
                    st_pack<Y, VEC>(out + c, pack<Y, VEC>(y));
                }
            }
        }
    }
}

// Zeros to n elements, by a warp: 16 bytes a lane from the first boundary on
// (by single elements, 20000 tokens into 50257 bf16 rows of 768
// from an odd element on took 79 us, so 70).
template <class G>
__device__ __forceinline__ void zero_span(G* to, int64_t n, int lane) {
    constexpr int kV = 16 / sizeof(G);
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(to) % 16) / sizeof(G);
    const int64_t head = mis == 0 ? 0 : n < kV - mis ? n : kV - mis;
    const int64_t words = (n - head) / kV;
    if (lane < head) to[lane] = narrow<G>(0.0f);
    for (int64_t i = lane; i < words; i += 32)
        reinterpret_cast<uint4*>(to + head)[i] = make_uint4(0, 0, 0, 0);
    const int64_t tail = head + words * kV;
    if (lane < n - tail) to[tail + lane] = narrow<G>(0.0f);
}

// ---------------------------------------------------------------- sort ------

constexpr int kSortThreads = 32 * kSortWarps;      // one token a thread and tile
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kFillRows = 32768;    // rows of one bitmap of used rows (4 KB)

constexpr int kChunk = 32;          // sorted places per warp of the sum launch
constexpr int kCols = 256;          // columns per warp

// Workspace: two buffers of keys and tokens, the run counters of the sum
// launch and its partial rows (two per chunk).
struct Workspace {
    int32_t* key[2];
    int32_t* tok[2];
    uint32_t* done;       // [chunks][column groups]
    float* partial;       // [chunks][2][dim]
    int64_t bytes;
};

__host__ __device__ inline int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }
__host__ __device__ inline int64_t chunks_of(int64_t n_tokens) {
    return (n_tokens + kChunk - 1) / kChunk;
}
__host__ __device__ inline int64_t groups_of(int64_t dim) { return (dim + kCols - 1) / kCols; }

__host__ __device__ inline Workspace workspace(void* base, int64_t n_tokens, int64_t dim) {
    Workspace w;
    char* p = static_cast<char*>(base);
    char* const start = p;
    const int64_t one = up16(n_tokens * 4);
    for (int i = 0; i < 2; ++i) {
        w.key[i] = reinterpret_cast<int32_t*>(p);
        p += one;
        w.tok[i] = reinterpret_cast<int32_t*>(p);
        p += one;
    }
    w.done = reinterpret_cast<uint32_t*>(p);
    p += up16(chunks_of(n_tokens) * groups_of(dim) * 4);
    w.partial = reinterpret_cast<float*>(p);
    p += chunks_of(n_tokens) * 2 * dim * 4;
    w.bytes = p - start;
    return w;
}

struct SortPlan {
    int passes;
    int bits;       // of one digit
};

__host__ __device__ inline SortPlan sort_plan(int64_t vocab) {
    int bits = 1;                                   // keys 0 .. vocab (vocab: no row)
    while (bits < 31 && (int64_t{1} << bits) <= vocab) ++bits;
    const int passes = (bits + kDigitBits - 1) / kDigitBits;
    return {passes, (bits + passes - 1) / passes};
}

struct SortSmem {
    uint32_t hist[2][kDigits];              // this CTA's digit counts, by pass parity
    uint32_t base[kDigits];                 // next place of each digit
    uint16_t warp[kSortWarps][kDigits];     // the tile's counts, then offsets, per warp
    uint32_t scan[32];
};

// The cluster's radix sort.  Pass 0 reads the ids, pass p > 0 buffer
// (p + 1) % 2; pass p writes buffer p % 2.
__device__ void sort_cluster(const EmbedGradArgs& a, const Workspace& ws, SortSmem& sm) {
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cluster.block_rank());
    const SortPlan plan = sort_plan(a.vocab);
    const int64_t share = (a.n_tokens + kSortCtas - 1) / kSortCtas;
    const int64_t lo = rank * share < a.n_tokens ? rank * share : a.n_tokens;
    const int64_t hi = lo + share < a.n_tokens ? lo + share : a.n_tokens;
    const uint32_t mask = (1u << plan.bits) - 1u;
    for (int pass = 0; pass < plan.passes; ++pass) {
        const int shift = pass * plan.bits;
        const bool odd = (pass & 1) != 0;
        const int32_t* src_key = odd ? ws.key[0] : ws.key[1];
        const int32_t* src_tok = odd ? ws.tok[0] : ws.tok[1];
        int32_t* dst_key = odd ? ws.key[1] : ws.key[0];
        int32_t* dst_tok = odd ? ws.tok[1] : ws.tok[0];
        uint32_t* hist = sm.hist[pass & 1];
        auto key_at = [&](int64_t i) -> uint32_t {
            if (pass > 0) return static_cast<uint32_t>(src_key[i]);
            const int64_t id = ld_id(a.ids, a.id64, i);
            return static_cast<uint32_t>(id >= 0 && id < a.vocab ? id : a.vocab);
        };
        if (tid < kDigits) hist[tid] = 0;
        __syncthreads();
        for (int64_t i = lo + tid; i < hi; i += 8 * kSortThreads) {
            uint32_t key[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t at = i + u * kSortThreads;
                key[u] = key_at(at < hi ? at : hi - 1);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (i + u * kSortThreads < hi) atomicAdd(&hist[(key[u] >> shift) & mask], 1u);
            }
        }
        cluster.sync();
        // first place of each digit for this CTA: all smaller digits, then
        // the same digit in the CTAs before it
        uint32_t before = 0, total = 0;
        if (tid < kDigits) {
            for (int r = 0; r < kSortCtas; ++r) {
                const uint32_t h = cluster.map_shared_rank(hist, r)[tid];
                if (r < rank) before += h;
                total += h;
            }
        }
        uint32_t incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sm.scan[warp] = incl;
        __syncthreads();
        if (tid < kDigits) {
            uint32_t s = incl - total + before;
            for (int w = 0; w < warp; ++w) s += sm.scan[w];
            sm.base[tid] = s;
        }
        auto load = [&](int64_t i, uint32_t& key, int32_t& tok) {
            const int64_t at = i < hi ? i : hi - 1;
            key = key_at(at);
            tok = pass > 0 ? src_tok[at] : static_cast<int32_t>(at);
        };
        uint32_t next_key = 0;
        int32_t next_tok = 0;
        if (lo < hi) load(lo + tid, next_key, next_tok);
        for (int64_t tile = lo; tile < hi; tile += kSortThreads) {
            const bool in = tile + tid < hi;
            const uint32_t key = next_key, digit = (key >> shift) & mask;
            const int32_t tok = next_tok;
            if (tile + kSortThreads < hi) load(tile + kSortThreads + tid, next_key, next_tok);
            for (int d = lane; d < kDigits / 2; d += 32)
                reinterpret_cast<uint32_t*>(sm.warp[warp])[d] = 0;
            __syncwarp();
            // the lanes with the same digit, and this lane's place among them
            uint32_t peers = __ballot_sync(0xFFFFFFFFu, in);
            if (!in) peers = ~peers;
            for (int b = 0; b < plan.bits; ++b) {
                const uint32_t set = __ballot_sync(0xFFFFFFFFu, (digit >> b) & 1u);
                peers &= (digit >> b) & 1u ? set : ~set;
            }
            const uint32_t below = __popc(peers & ((1u << lane) - 1u));
            if (in && below == 0) sm.warp[warp][digit] = static_cast<uint16_t>(__popc(peers));
            __syncthreads();
            if (tid < kDigits) {
                uint32_t c[kSortWarps];
#pragma unroll
                for (int w = 0; w < kSortWarps; ++w) c[w] = sm.warp[w][tid];
                uint32_t s = 0;
#pragma unroll
                for (int w = 0; w < kSortWarps; ++w) {
                    sm.warp[w][tid] = static_cast<uint16_t>(s);
                    s += c[w];
                }
                incl = s;      // the tile's count of this digit
            }
            __syncthreads();
            if (in) {
                const uint32_t at = sm.base[digit] + sm.warp[warp][digit] + below;
                dst_key[at] = static_cast<int32_t>(key);
                dst_tok[at] = tok;
            }
            __syncthreads();
            if (tid < kDigits) sm.base[tid] += incl;
        }
        __threadfence();
        cluster.sync();
    }
}

// Zeros to the rows of dW in [lo, hi) that no token has.
template <class G>
__device__ void fill_unused(const EmbedGradArgs& a, int64_t lo, int64_t hi, uint32_t* used) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int64_t r0 = lo; r0 < hi; r0 += kFillRows) {
        const int64_t n = hi - r0 < kFillRows ? hi - r0 : kFillRows;
        const int words = static_cast<int>((n + 31) / 32);
        __syncthreads();
        for (int i = tid; i < words; i += kSortThreads) used[i] = 0;
        __syncthreads();
        for (int64_t t = tid; t < a.n_tokens; t += 8 * kSortThreads) {
            // loads without conditions, so that all are under way
            int64_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t at = t + u * kSortThreads;
                v[u] = ld_id(a.ids, a.id64, at < a.n_tokens ? at : a.n_tokens - 1) - r0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (v[u] >= 0 && v[u] < n) atomicOr(&used[v[u] >> 5], 1u << (v[u] & 31));
            }
        }
        __syncthreads();
        for (int64_t r = warp; r < n; r += kSortWarps) {
            if ((used[r >> 5] >> (r & 31)) & 1u) continue;
            zero_span(static_cast<G*>(a.grad_weight) + (r0 + r) * a.dim, a.dim, lane);
        }
    }
}

template <class G>
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads)
embed_sort_kernel(const __grid_constant__ EmbedGradArgs a) {
    __shared__ SortSmem sm;
    const Workspace ws = workspace(a.workspace, a.n_tokens, a.dim);
    if (blockIdx.x < kSortCtas) {
        const int64_t n_done = chunks_of(a.n_tokens) * groups_of(a.dim);
        for (int64_t i = blockIdx.x * kSortThreads + threadIdx.x; i < n_done;
             i += kSortCtas * kSortThreads)
            ws.done[i] = 0;
        sort_cluster(a, ws, sm);
    } else {
        const int64_t ctas = gridDim.x - kSortCtas, i = blockIdx.x - kSortCtas;
        const int64_t per = (a.vocab + ctas - 1) / ctas;
        const int64_t lo = i * per, hi = lo + per < a.vocab ? lo + per : a.vocab;
        if (lo < hi) fill_unused<G>(a, lo, hi, reinterpret_cast<uint32_t*>(&sm));
    }
}

static_assert(sizeof(SortSmem) >= kFillRows / 8, "the bitmap shares the sort's memory");

// ----------------------------------------------------------------- sum ------

// Pairs of a pack's values in fp32.
template <class T, int VEC>
__device__ __forceinline__ Pair pair_of(const Pack<T, VEC>& p, int i) {
    if constexpr (sizeof(T) == 2) return widen2(reinterpret_cast<const uint32_t*>(&p)[i]);
    else return pair(p.x[2 * i], p.x[2 * i + 1]);
}

// acc += the N packs of a row.
template <class T, int VEC, int N, int PER>
__device__ __forceinline__ void add_row(Pair (&acc)[PER / 2], const Pack<T, VEC> (&v)[N]) {
    if constexpr (VEC == 1) {
#pragma unroll
        for (int i = 0; i < PER / 2; ++i)
            acc[i] = add2(acc[i], pair(widen<T>(v[2 * i].x[0]), widen<T>(v[2 * i + 1].x[0])));
    } else {
#pragma unroll
        for (int i = 0; i < PER / 2; ++i)
            acc[i] = add2(acc[i], pair_of(v[2 * i / VEC], i % (VEC / 2)));
    }
}

// What the sort leaves to the sum launch.
struct Sorted {
    const int32_t* key;
    const int32_t* tok;
    uint32_t* done;
    float* partial;
    int32_t groups;       // of columns
};

// A warp: a chunk (block z) and a group of columns (block y).  Lane columns: N
// groups of VEC, group n at (32 n + lane) VEC.
template <class Y, class G, int VEC, bool ACC>
__global__ void __launch_bounds__(256, VEC == 1 ? 2 : 3)
embed_sum_kernel(const __grid_constant__ EmbedGradArgs a, const __grid_constant__ Sorted s) {
    constexpr int kPer = kCols / 32;
    constexpr int N = kPer / VEC;
    constexpr int kAhead = ACC || sizeof(Y) == 4 || VEC == 1 ? 4 : 8;
    const int lane = threadIdx.x;
    const int chunk = blockIdx.x * blockDim.z + threadIdx.z;
    const int group = blockIdx.y * blockDim.y + threadIdx.y;
    const int T = static_cast<int>(a.n_tokens);
    const int64_t col0 = static_cast<int64_t>(group) * kCols;
    const int first = chunk * kChunk;
    if (first >= T || col0 >= a.dim) return;
    const int32_t none = static_cast<int32_t>(a.vocab);
    const int n = T - first < kChunk ? T - first : kChunk;
    // this lane's place of the chunk, and the neighbours' keys
    const int at = first + (lane < n ? lane : n - 1);
    const int32_t place_key = s.key[at], my_tok = s.tok[at];
    const int32_t key_before = first > 0 ? s.key[first - 1] : -1;
    const int32_t key_after = first + n < T ? s.key[first + n] : -1;
    const int32_t my_key = lane < n ? place_key : none;
    const int live = __popc(__ballot_sync(0xFFFFFFFFu, my_key != none));   // a prefix
    {
        auto column = [&](int j) -> int64_t {       // of a load: in the row
            const int64_t c = col0 + (j * 32 + lane) * VEC;
            return c < a.dim ? c : 0;
        };
        Pair acc[kPer / 2];
        auto clear = [&] {
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) acc[i] = 0;
        };
        auto load_row = [&](Pack<G, VEC> (&old)[N], int32_t k) {
            const G* row = static_cast<const G*>(a.grad_weight) + static_cast<int64_t>(k) * a.dim;
#pragma unroll
            for (int j = 0; j < N; ++j) old[j] = ld_pack<G, VEC>(row + column(j));
        };
        auto write_row = [&](int32_t k, const Pack<G, VEC> (&old)[N]) {
            G* row = static_cast<G*>(a.grad_weight) + static_cast<int64_t>(k) * a.dim;
            float sum[kPer];
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) {
                const float2 f = unpair(acc[i]);
                sum[2 * i] = f.x * a.scale;
                sum[2 * i + 1] = f.y * a.scale;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int64_t c = col0 + (j * 32 + lane) * VEC;
                if (c >= a.dim) continue;
                float y[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    y[e] = sum[j * VEC + e];
                    if (ACC) y[e] += widen<G>(old[j].x[e]);
                }
                st_pack<G, VEC>(row + c, pack<G, VEC>(y));
            }
        };
        auto put_partial = [&](int slot) {
            float* p = s.partial + (static_cast<int64_t>(chunk) * 2 + slot) * a.dim;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int64_t c = col0 + (e / VEC * 32 + lane) * VEC + e % VEC;
                const float2 f = unpair(acc[e / 2]);
                if (c < a.dim) __stcg(p + c, e % 2 == 0 ? f.x : f.y);
            }
        };
        // A run of key k over several chunks, `first_chunk` .. `last_chunk`, of
        // which this one has left its partial: the last to come adds them up.
        auto join = [&](int32_t k, int first_chunk, int last_chunk) {
            __threadfence();
            __syncwarp();
            uint32_t seen = 0;
            if (lane == 0) seen = atomicAdd(&s.done[static_cast<int64_t>(first_chunk) * s.groups + group], 1u);
            seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
            if (seen != static_cast<uint32_t>(last_chunk - first_chunk)) return;
            __threadfence();
            clear();
            for (int q = first_chunk; q <= last_chunk; q += 4) {
                float v[4][kPer];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    // the run starts in its first chunk's second slot; later chunks
                    // use the first
                    const int at = q + u <= last_chunk ? q + u : last_chunk;
                    const float* p =
                        s.partial + (static_cast<int64_t>(at) * 2 + (at == first_chunk ? 1 : 0)) * a.dim;
#pragma unroll
                    for (int e = 0; e < kPer; ++e) v[u][e] = __ldcg(p + column(e / VEC) + e % VEC);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (q + u > last_chunk) break;
#pragma unroll
                    for (int i = 0; i < kPer / 2; ++i)
                        acc[i] = add2(acc[i], pair(v[u][2 * i], v[u][2 * i + 1]));
                }
            }
            Pack<G, VEC> old[N];
            if (ACC) load_row(old, k);
            write_row(k, old);
        };
        // The chunk in which the run of k that enters this chunk starts.
        auto run_start = [&](int32_t k) -> int {
            for (int q = chunk - 1;; q -= 32) {
                // chunk q - lane: does the run enter it from the one before?
                const int c = q - lane;
                const bool goes_on = c > 0 && s.key[c * kChunk - 1] == k;
                const uint32_t stop = __ballot_sync(0xFFFFFFFFu, !goes_on);
                if (stop != 0) return q - (__ffs(stop) - 1);
            }
        };
        // The chunk in which the run of k that leaves this chunk ends.
        auto run_end = [&](int32_t k) -> int {
            for (int q = chunk + 1;; q += 32) {
                const int64_t next = (static_cast<int64_t>(q) + lane + 1) * kChunk;
                const bool goes_on = next < T && s.key[next] == k;
                const uint32_t stop = __ballot_sync(0xFFFFFFFFu, !goes_on);
                if (stop != 0) return q + (__ffs(stop) - 1);
            }
        };

        clear();
        int begin = 0;                                  // first place of the current run
        // places at which a run is over, or leaves the chunk
        const int32_t key_next = __shfl_down_sync(0xFFFFFFFFu, my_key, 1);
        const uint32_t over =
            __ballot_sync(0xFFFFFFFFu, lane < live && (lane + 1 == n || key_next != my_key));
        for (int i0 = 0; i0 < live; i0 += kAhead) {
            Pack<Y, VEC> v[kAhead][N];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                // without conditions, so that all are under way: past the end the
                // last place again, beyond the row its first column
                const int32_t t =
                    __shfl_sync(0xFFFFFFFFu, my_tok, i0 + u < live ? i0 + u : live - 1);
                const Y* row = static_cast<const Y*>(a.grad_out) + t * a.grad_stride;
#pragma unroll
                for (int j = 0; j < N; ++j) v[u][j] = ld_pack<Y, VEC>(row + column(j));
            }
            Pack<G, VEC> old[ACC ? kAhead : 1][N];
            if (ACC && ((over >> i0) & ((1u << kAhead) - 1u)) != 0) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    load_row(old[ACC ? u : 0],
                             __shfl_sync(0xFFFFFFFFu, my_key, i0 + u < live ? i0 + u : live - 1));
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u;
                if (i >= live) break;
                add_row<Y, VEC, N, kPer>(acc, v[u]);
                if (!((over >> i) & 1u)) continue;
                const int32_t k = __shfl_sync(0xFFFFFFFFu, my_key, i);
                // the run ends here, or goes on in the next chunk
                const bool enters = begin == 0 && key_before == k;
                const bool leaves = i + 1 == n && key_after == k;
                if (!enters && !leaves) {
                    write_row(k, old[ACC ? u : 0]);
                } else {
                    put_partial(enters ? 0 : 1);
                    const int from = enters ? run_start(k) : chunk;
                    const int to = leaves ? run_end(k) : chunk;
                    join(k, from, to);
                }
                clear();
                begin = i + 1;
            }
        }
    }
}

// ------------------------------------------------------------- buckets ------
//
// For up to kBucketTokens tokens one launch does it all.  A CTA owns the rows
// of a bucket (1 of B: the low bits of the id, mixed with a hash of the high
// ones) and 256 columns (128 with fp32).  It reads all ids, keeps its own tokens in order,
// counts them by row, groups them (a row's tokens stay in order), and its
// warps add up equal parts of the grouped tokens; runs over several parts are
// joined from shared memory in order.  Where every row is written, the rows
// without a token get their zeros on the way.

constexpr int kBucketThreads = 512;
constexpr int kBucketWarps = kBucketThreads / 32;
constexpr int kTokenBits = 14;
constexpr int64_t kBucketTokens = 1 << kTokenBits;
constexpr int64_t kFewTokens = 8192;                 // up to here whatever the width
constexpr int64_t kBucketElements = 10 << 20;        // and up to here beyond
constexpr int kBucketSmem = 160 * 1024;              // beside 33 KB of static memory

struct Bucket {
    int bits;            // B = 1 << bits
    int64_t rows;        // of a bucket, at most: ceil(vocab / B)
    int64_t smem;        // list, order, row starts (the partial rows are static)
};

// Tokens of a warp: whole groups of 32.
__host__ __device__ inline int bucket_share(int64_t n_tokens) {
    return static_cast<int>((n_tokens + kBucketWarps * 32 - 1) / (kBucketWarps * 32) * 32);
}

__host__ __device__ inline uint32_t bucket_mix(uint32_t high, int bits) {
    return bits == 0 ? 0u : (high * 2654435761u) >> (32 - bits);
}

// Columns of a CTA: 16 bytes a lane of the wider type.
__host__ __device__ constexpr int bucket_cols(int widest) { return 512 / widest; }

Bucket bucket_for(int64_t n_tokens, int64_t vocab, int64_t dim, int widest, int sms) {
    const int64_t most = 2 * sms / ((dim + bucket_cols(widest) - 1) / bucket_cols(widest));
    Bucket b{0, vocab, 0};
    while ((int64_t{2} << b.bits) <= most || b.rows > 8192) {
        if (b.bits == 16) break;
        ++b.bits;
        b.rows = ((vocab - 1) >> b.bits) + 1;
    }
    b.smem = kBucketWarps * bucket_share(n_tokens) * 6 + up16((b.rows + 1) * 4);
    return b;
}

// Whether a gradient takes the one launch.  Every CTA reads all ids, and above
// kFewTokens its lists leave an SM one CTA; what that costs grows with the
// elements.  In us, buckets / sort, added to a table of 50257 bf16 rows:
//   tokens    dim 128      768          2048         4096
//    4096     12.7 / 29.1  14.8 / 29.1  18.4 / 29.8   28.0 / 35.4
//    8192     16.9 / 29.8  23.0 / 30.0  34.1 / 37.9   55.1 / 52.4
//   12288     22.1 / 33.1  32.3 / 34.5  56.0 / 45.5  102.6 / 63.3
//   16384     28.1 / 35.3  39.9 / 37.3  80.5 / 55.5  137.5 / 74.4
// (4096 fp32 columns: 6144 tokens 60.2 / 69.9, 8192 92.8 / 86.5).  So at kFewTokens
// rows of 4096 columns lose 5 to 7 % by the one launch; wider ones are not measured.
bool takes_buckets(int64_t n_tokens, int64_t vocab, int64_t dim) {
    if (n_tokens > kBucketTokens || (n_tokens > kFewTokens && n_tokens * dim > kBucketElements))
        return false;
    const Bucket b = bucket_for(n_tokens, vocab, dim, 4, device_sms());
    return b.rows < (1 << (32 - kTokenBits)) && b.smem <= kBucketSmem &&
           dim <= 65535 * int64_t{bucket_cols(4)};
}

template <class Y, class G, int VEC, bool ACC>
__global__ void __launch_bounds__(kBucketThreads, 2)
embed_bucket_kernel(const __grid_constant__ EmbedGradArgs a, int bits, int n_rows) {
    constexpr int kPer = bucket_cols(sizeof(Y) > sizeof(G) ? sizeof(Y) : sizeof(G)) / 32;
    constexpr int kWidth = 32 * kPer;
    constexpr int N = kPer / VEC;
    constexpr int kAhead = VEC == 1 && kPer == 8 ? 2 : ACC ? 4 : 8;
    constexpr uint32_t kTokenMask = (1u << kTokenBits) - 1;
    extern __shared__ __align__(16) char smem[];
    __shared__ float partial[kBucketWarps][2][256];      // before: the rows with several tokens
    __shared__ int warp_n[kBucketWarps], through[kBucketWarps];
    __shared__ uint32_t warp_sums[kBucketWarps];
    __shared__ int n_several;
    const int T = static_cast<int>(a.n_tokens);
    const int share = bucket_share(T);                   // of a warp: its tokens and list
    uint32_t* list = reinterpret_cast<uint32_t*>(smem);  // row << 14 | token, by warp
    uint16_t* order = reinterpret_cast<uint16_t*>(list + kBucketWarps * share);
    uint32_t* start = reinterpret_cast<uint32_t*>(order + kBucketWarps * share);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bucket = blockIdx.x;
    const uint32_t low = (1u << bits) - 1u;
    const int64_t col0 = static_cast<int64_t>(blockIdx.y) * kWidth;

    for (int i = tid; i <= n_rows; i += kBucketThreads) start[i] = 0;
    if (tid == 0) n_several = 0;
    __syncthreads();

    // this bucket's tokens among the warp's, in order, and their rows' counts
    const int t0 = warp * share;
    int mine = 0;
    for (int it = 0; it * 32 < share; it += 8) {
        // loads without conditions (at a clamped place), so that all are under way
        int64_t id[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int t = t0 + (it + u) * 32 + lane;
            id[u] = ld_id(a.ids, a.id64, t < T ? t : T - 1);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int t = t0 + (it + u) * 32 + lane;
            const uint32_t high = static_cast<uint32_t>(id[u]) >> bits;
            const bool in = t < T && t < t0 + share && id[u] >= 0 && id[u] < a.vocab &&
                            ((static_cast<uint32_t>(id[u]) & low) ^ bucket_mix(high, bits)) == bucket;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, in);
            if (in) {
                list[t0 + mine + __popc(m & ((1u << lane) - 1u))] =
                    high << kTokenBits | static_cast<uint32_t>(t);
                atomicAdd(&start[high], 1u);
            }
            mine += __popc(m);
        }
    }
    if (lane == 0) warp_n[warp] = mine;
    __syncthreads();

    // rows' counts to first places; the rows with several tokens
    const int rows_per = (n_rows + kBucketThreads) / kBucketThreads;     // n_rows + 1 of them
    const int r0 = tid * rows_per < n_rows + 1 ? tid * rows_per : n_rows + 1;
    const int r1 = r0 + rows_per < n_rows + 1 ? r0 + rows_per : n_rows + 1;
    uint32_t sum = 0;
    for (int r = r0; r < r1; ++r) sum += start[r];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    uint32_t first = incl - sum;
    for (int w = 0; w < warp; ++w) first += warp_sums[w];
    uint32_t* several = reinterpret_cast<uint32_t*>(&partial[0][0][0]);
    for (int r = r0; r < r1; ++r) {
        const uint32_t c = start[r];
        start[r] = first;
        first += c;
        if (c > 1) several[atomicAdd(&n_several, 1)] = static_cast<uint32_t>(r);
    }
    __syncthreads();
    const int n = static_cast<int>(start[n_rows]);

    auto row_at = [&](uint32_t r) -> G* {       // row r of the bucket in the table
        const int64_t id = (static_cast<int64_t>(r) << bits) | (bucket ^ bucket_mix(r, bits));
        return static_cast<G*>(a.grad_weight) + id * a.dim;
    };
    // zeros to the rows of [lo, hi) without a token
    auto fill = [&](int lo, int hi) {
        float zero[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) zero[e] = 0.0f;
        const Pack<G, VEC> z = pack<G, VEC>(zero);
        for (int r = lo + warp; r < hi; r += kBucketWarps) {
            if (start[r] != start[r + 1]) continue;
            const int64_t id = (static_cast<int64_t>(r) << bits) |
                               (bucket ^ bucket_mix(static_cast<uint32_t>(r), bits));
            if (id >= a.vocab) continue;
            G* row = static_cast<G*>(a.grad_weight) + id * a.dim;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int64_t c = col0 + (j * 32 + lane) * VEC;
                if (c < a.dim) st_pack<G, VEC>(row + c, z);
            }
        }
    };
    // half of the zeros now, half while the first loads are under way
    if (!ACC) fill(0, n_rows / 2);

    // the tokens grouped by row: single ones by themselves, a row with several
    // by a warp that walks the lists
    for (int i = lane; i < mine; i += 32) {
        const uint32_t r = list[t0 + i] >> kTokenBits;
        if (start[r + 1] - start[r] == 1) order[start[r]] = static_cast<uint16_t>(t0 + i);
    }
    for (int k = warp; k < n_several; k += kBucketWarps) {
        const uint32_t r = several[k];
        uint32_t to = start[r];
        const uint32_t end = start[r + 1];
        for (int w = 0; w < kBucketWarps && to < end; ++w) {
            for (int i0 = 0; i0 < warp_n[w]; i0 += 32) {
                const int i = i0 + lane;
                const bool same = i < warp_n[w] && list[w * share + i] >> kTokenBits == r;
                const uint32_t m = __ballot_sync(0xFFFFFFFFu, same);
                if (same)
                    order[to + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(w * share + i);
                to += __popc(m);
            }
        }
    }
    __syncthreads();

    // equal parts of the grouped tokens, one a warp
    const int per = (n + kBucketWarps - 1) / kBucketWarps;
    const int p0 = warp * per < n ? warp * per : n;
    const int p1 = p0 + per < n ? p0 + per : n;
    auto entry = [&](int p) { return list[order[p]]; };
    float acc[kPer];
    auto clear = [&] {
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = 0.0f;
    };
    auto column = [&](int j) -> int64_t {       // of a load: in the row
        const int64_t c = col0 + (j * 32 + lane) * VEC;
        return c < a.dim ? c : 0;
    };
    auto load_row = [&](Pack<G, VEC> (&old)[N], const G* row) {
#pragma unroll
        for (int j = 0; j < N; ++j) old[j] = ld_pack<G, VEC>(row + column(j));
    };
    auto write_row = [&](G* row, const Pack<G, VEC> (&old)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t c = col0 + (j * 32 + lane) * VEC;
            if (c >= a.dim) continue;
            float y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                y[e] = acc[j * VEC + e] * a.scale;
                if (ACC) y[e] += widen<G>(old[j].x[e]);
            }
            st_pack<G, VEC>(row + c, pack<G, VEC>(y));
        }
    };
    int passes = 0, leaves = -1;                // the run goes through the part; leaves it
    bool filled = ACC;
    clear();
    if (p0 < p1) {
        const int before = p0 > 0 ? static_cast<int>(entry(p0 - 1) >> kTokenBits) : -1;
        int begin = p0;                          // of the current run in the part
        for (int q = p0; q < p1; q += 32) {
            const uint32_t my = entry(q + lane < p1 ? q + lane : p1 - 1);
            // places at which a run is over
            const uint32_t over = __ballot_sync(
                0xFFFFFFFFu, q + lane < p1 && start[(my >> kTokenBits) + 1] == q + lane + 1u);
            for (int u0 = 0; u0 < 32 && q + u0 < p1; u0 += kAhead) {
                Pack<Y, VEC> v[kAhead][N];
                Pack<G, VEC> old[ACC ? kAhead : 1][N];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    // without conditions: past the end the last place again,
                    // beyond the row its first column
                    const uint32_t e = __shfl_sync(0xFFFFFFFFu, my, u0 + u);
                    const Y* row = static_cast<const Y*>(a.grad_out) +
                                   static_cast<int64_t>(e & kTokenMask) * a.grad_stride;
#pragma unroll
                    for (int j = 0; j < N; ++j) v[u][j] = ld_pack<Y, VEC>(row + column(j));
                }
                if (ACC && ((over >> u0) & ((1u << kAhead) - 1u)) != 0) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const uint32_t e = __shfl_sync(0xFFFFFFFFu, my, u0 + u);
                        load_row(old[ACC ? u : 0], row_at(e >> kTokenBits));
                    }
                }
                if (!filled) {
                    fill(n_rows / 2, n_rows);
                    filled = true;
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int p = q + u0 + u;
                    if (p >= p1) break;
                    const uint32_t r = __shfl_sync(0xFFFFFFFFu, my, u0 + u) >> kTokenBits;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) acc[j * VEC + e] += widen<Y>(v[u][j].x[e]);
                    }
                    const bool ends = (over >> (u0 + u)) & 1u;
                    if (!ends && p + 1 < p1) continue;
                    const bool enters = begin == p0 && before == static_cast<int>(r);
                    if (ends && !enters) {
                        write_row(row_at(r), old[ACC ? u : 0]);
                    } else {
                        float* to = partial[warp][enters ? 0 : 1];
#pragma unroll
                        for (int e = 0; e < kPer; ++e) to[(e / VEC * 32 + lane) * VEC + e % VEC] = acc[e];
                        if (!ends) {
                            if (enters) passes = 1;
                            else leaves = static_cast<int>(r);
                        }
                    }
                    clear();
                    begin = p + 1;
                }
            }
        }
    }
    if (!filled) fill(n_rows / 2, n_rows);
    if (lane == 0) through[warp] = passes;
    __syncthreads();
    // the run that leaves this part for the next ones: joined in order
    if (leaves >= 0) {
        G* row = row_at(static_cast<uint32_t>(leaves));
        Pack<G, VEC> old[N];
        if (ACC) load_row(old, row);
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            acc[e] = partial[warp][1][(e / VEC * 32 + lane) * VEC + e % VEC];
        for (int w = warp + 1; w < kBucketWarps; ++w) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                acc[e] += partial[w][0][(e / VEC * 32 + lane) * VEC + e % VEC];
            if (!through[w]) break;
        }
        write_row(row, old);
    }
}

template <class Y, class G, int VEC, bool ACC>
cudaError_t embed_buckets_as(const EmbedGradArgs& a, cudaStream_t stream) {
    constexpr int kWidth = bucket_cols(sizeof(Y) > sizeof(G) ? sizeof(Y) : sizeof(G));
    int sms = 0;
    if (cudaError_t e = device_sms(&sms); e != cudaSuccess) return e;
    const Bucket b = bucket_for(a.n_tokens, a.vocab, a.dim, 512 / kWidth, sms);
    const dim3 grid(1u << b.bits, static_cast<unsigned>((a.dim + kWidth - 1) / kWidth));
    const auto kernel = embed_bucket_kernel<Y, G, VEC, ACC>;
    // more than 48 KB of shared memory need asking for
    static std::once_flag once[64];
    static cudaError_t set[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kBucketSmem);
    });
    if (set[dev] != cudaSuccess) return set[dev];
    kernel<<<grid, kBucketThreads, static_cast<size_t>(b.smem), stream>>>(
        a, b.bits, static_cast<int>(b.rows));
    return cudaGetLastError();
}

template <class Y, class G>
cudaError_t embed_buckets(const EmbedGradArgs& a, cudaStream_t stream) {
    constexpr int kV = sizeof(Y) == 2 && sizeof(G) == 2 ? 8 : 4;
    const bool vec = aligned_to(a.grad_out, kV * static_cast<int64_t>(sizeof(Y))) &&
                     aligned_to(a.grad_weight, kV * static_cast<int64_t>(sizeof(G))) &&
                     a.dim % kV == 0 && a.grad_stride % kV == 0;
    if (a.accumulate)
        return vec ? embed_buckets_as<Y, G, kV, true>(a, stream)
                   : embed_buckets_as<Y, G, 1, true>(a, stream);
    return vec ? embed_buckets_as<Y, G, kV, false>(a, stream)
               : embed_buckets_as<Y, G, 1, false>(a, stream);
}

template <class W, class Y>
cudaError_t embed(const EmbedArgs& a, cudaStream_t stream) {
    constexpr int kV = sizeof(W) == 2 && sizeof(Y) == 2 ? 8 : 4;
    const bool vec = aligned_to(a.weight, kV * static_cast<int64_t>(sizeof(W))) &&
                     aligned_to(a.out, kV * static_cast<int64_t>(sizeof(Y))) &&
                     a.dim % kV == 0 && a.out_stride % kV == 0;
    const int tokens = 8 * (vec ? 4 : 2), width = 32 * (vec ? kV : 4);
    int sms = 0;
    if (cudaError_t e = device_sms(&sms); e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(sms) * 64;
    const int64_t x = (a.n_tokens + tokens - 1) / tokens, y = (a.dim + width - 1) / width;
    const dim3 grid(static_cast<unsigned>(x < most ? x : most),
                    static_cast<unsigned>(y < 65535 ? y : 65535));
    if (vec) {
        embed_kernel<W, Y, kV, 4, 1><<<grid, dim3(32, 8), 0, stream>>>(a);
    } else {
        embed_kernel<W, Y, 1, 2, 4><<<grid, dim3(32, 8), 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <class Y, class G>
cudaError_t embed_sum(const EmbedGradArgs& a, cudaStream_t stream) {
    constexpr int kV = sizeof(Y) == 2 && sizeof(G) == 2 ? 8 : 4;
    const bool vec = aligned_to(a.grad_out, kV * static_cast<int64_t>(sizeof(Y))) &&
                     aligned_to(a.grad_weight, kV * static_cast<int64_t>(sizeof(G))) &&
                     a.dim % kV == 0 && a.grad_stride % kV == 0;
    const Workspace ws = workspace(a.workspace, a.n_tokens, a.dim);
    const int last = (sort_plan(a.vocab).passes - 1) % 2;
    const int groups = static_cast<int>(groups_of(a.dim));
    const Sorted sorted{ws.key[last], ws.tok[last], ws.done, ws.partial, groups};
    // 8 warps: the groups of a chunk side by side, then chunks
    const int gy = groups < 8 ? groups : 8, cz = 8 / gy;
    const dim3 block(32, gy, cz);
    const dim3 grid(static_cast<unsigned>((chunks_of(a.n_tokens) + cz - 1) / cz),
                    static_cast<unsigned>((groups + gy - 1) / gy));
    if (a.accumulate) {
        if (vec) embed_sum_kernel<Y, G, kV, true><<<grid, block, 0, stream>>>(a, sorted);
        else embed_sum_kernel<Y, G, 1, true><<<grid, block, 0, stream>>>(a, sorted);
    } else {
        if (vec) embed_sum_kernel<Y, G, kV, false><<<grid, block, 0, stream>>>(a, sorted);
        else embed_sum_kernel<Y, G, 1, false><<<grid, block, 0, stream>>>(a, sorted);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs& a, int weight_bytes, int out_bytes,
                         cudaStream_t stream) {
    if (weight_bytes == 2)
        return out_bytes == 2 ? embed<uint16_t, uint16_t>(a, stream)
                              : embed<uint16_t, float>(a, stream);
    return out_bytes == 2 ? embed<float, uint16_t>(a, stream) : embed<float, float>(a, stream);
}

int64_t embed_grad_workspace(int64_t n_tokens, int64_t vocab, int64_t dim) {
    return embed_grad_in_one(n_tokens, vocab, dim) ? 0 : workspace(nullptr, n_tokens, dim).bytes;
}

bool embed_grad_in_one(int64_t n_tokens, int64_t vocab, int64_t dim) {
    return takes_buckets(n_tokens, vocab, dim);
}

cudaError_t launch_embed_buckets(const EmbedGradArgs& a, int grad_bytes, int grad_weight_bytes,
                                 cudaStream_t stream) {
    if (grad_bytes == 2)
        return grad_weight_bytes == 2 ? embed_buckets<uint16_t, uint16_t>(a, stream)
                                      : embed_buckets<uint16_t, float>(a, stream);
    return grad_weight_bytes == 2 ? embed_buckets<float, uint16_t>(a, stream)
                                  : embed_buckets<float, float>(a, stream);
}

cudaError_t launch_embed_sort(const EmbedGradArgs& a, int grad_weight_bytes, cudaStream_t stream) {
    int sms = 0;
    if (cudaError_t e = device_sms(&sms); e != cudaSuccess) return e;
    const unsigned g =
        static_cast<unsigned>(sort_clusters(a.vocab, a.accumulate != 0, sms) * kSortCtas);
    if (grad_weight_bytes == 4) embed_sort_kernel<float><<<g, kSortThreads, 0, stream>>>(a);
    else embed_sort_kernel<uint16_t><<<g, kSortThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_embed_sum(const EmbedGradArgs& a, int grad_bytes, int grad_weight_bytes,
                             cudaStream_t stream) {
    if (grad_bytes == 2)
        return grad_weight_bytes == 2 ? embed_sum<uint16_t, uint16_t>(a, stream)
                                      : embed_sum<uint16_t, float>(a, stream);
    return grad_weight_bytes == 2 ? embed_sum<float, uint16_t>(a, stream)
                                  : embed_sum<float, float>(a, stream);
}

}  // namespace zf
