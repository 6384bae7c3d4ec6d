// Softmax cross entropy of the head, without keeping the logits: for hidden states h and
// the table W
//   z = h W^T,  lse = log sum_v exp z_v,  loss = lse - z[label],
//   dz = g (exp(z - lse) - 1[v = label]),  dh = dz W,  dW = dz^T h.
//
// The products run on the tensor cores (bf16 operands, fp32 sums) by pairs of CTAs on 256 x
// 256 tiles: one thread streams operands by TMA into a ring in shared memory, one thread of
// the pair issues the products, eight warps turn finished tiles of tensor memory into
// results while the next tile's products run.  The forward pass leaves a maximum of the logits
// and a sum of exponentials for each row and tile, joined by a second launch.  The backward pass
// works through the vocabulary in pieces: the piece's z again, its dz in bf16 to the
// workspace, then dz W, added up in fp32 over the pieces, and dz^T h.
//
// dz is rounded to bf16 because the tensor cores multiply bf16: 2^-8 of each term at most; its
// sums are held in fp32.  Where many tokens are live these roundings are as large as the
// result's own, and a second part of dz would cost as much again as the products of the first.
// Up to 128 live tokens leave half of a tile's rows free, and these hold what the rounding
// left, in bf16 too: 2^-16 of each term at most.
//
// Only live tokens take part: their hidden rows are copied side by side, so that a prompt's
// tokens without a label cost nothing and their values reach nothing.
//
// Bound by the tensor cores under the power cap where products are long: gradients of 8192
// tokens of a table of 131072 x 4096 15.5 to 16.2 ms (1.70 to 1.63 PFLOP/s), the loss of 5500
// live ones 3.1 to 3.7 ms (1.9 to 1.6).  Shorter sums are bound by shared memory, which operands
// on their way in and out fill at the tensor cores' rate, and results cross too: 8192 tokens,
// 50257 x 768, 1.18 to 1.34 ms (1.61 to 1.42 PFLOP/s).  Few tokens, whose loss has a kernel of
// its own: by reading the table, and a launch's start and end (8 tokens, 131072 x 4096 158 to
// 165 us, 6.8 to 6.5 TB/s; 32, 50257 x 768 19.5 to 21.7 us).
#include "zero_head.cuh"

#include <cfloat>
#include <mutex>

#include "zero_kernels.cuh"
#include "zero_ops.cuh"
#include "zero_status.cuh"
#include "zero_tile.cuh"

namespace zf {

namespace {

using namespace tile;

constexpr int kPairTile = 256;                  // rows, and most columns, of a pair's tile
constexpr int kTileK = 64;
constexpr int kHalf = 128;                  // of the tile, a CTA's share of each operand
constexpr int kStages = 6;
constexpr uint32_t kOperandBytes = kHalf * kTileK * 2;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr uint32_t kChunkBytes = kTileK * 128;        // 64 values along M or N, MN-major
constexpr uint32_t kStagingBytes = 4096;      // an epilogue warp's
constexpr int kEpilogueWarps = 8;
constexpr size_t kHeadSmem = kStages * kStageBytes + kEpilogueWarps * kStagingBytes + 1024;
constexpr int kHeadThreads = 64 + 32 * kEpilogueWarps;
constexpr uint32_t kTmemColumns = 512;      // two tiles' results
// Steps of a logit's sum that are summed in tensor memory at a time.  Sums there are cut off,
// not rounded: a loss of 4096 columns summed in one go was 2.0e-6 of itself off, four times as
// far as by plain fp32 products; in parts of 1536 columns that are added up in registers
// 6.6e-7 (1024: 4.6e-7, 2048: 9.8e-7; the parts cost 4 to 6 % of the time).  The gradient's
// logits are summed in the same parts: its probabilities are next to 1 where the loss's are.
constexpr int kLogitSteps = 24;
// The same of the gradients' sums, over the vocabulary or over the tokens: a step of 16
// products cuts off up to two units of the sum so far, so that 65536 values of one sign end
// 2^-11 low at most, beside bf16's own rounding of up to 2^-8.  2M tokens summed in one go were
// 1.2e-2 low, 1.6 units a step.  (131072 tokens, 8000 x 768 4.78 ms, in one go 4.66.)
constexpr int kSumSteps = 1024;
constexpr uint64_t kHeadWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

// What a launch computes: rows' statistics, the logits' gradient, or both gradients that are
// products of it: tiles of the hidden states' first, then of the table's.
// (kLossLong, kDzLong: from logits that are summed in several parts; kProductsLong: so are the
// gradients.)
enum Mode { kLoss, kLossLong, kDz, kDzLong, kProducts, kProductsLong };
__host__ __device__ constexpr bool is_loss(int mode) { return mode == kLoss || mode == kLossLong; }
__host__ __device__ constexpr bool is_dz(int mode) { return mode == kDz || mode == kDzLong; }
__host__ __device__ constexpr bool is_products(int mode) {
    return mode == kProducts || mode == kProductsLong;
}
__host__ __device__ constexpr bool is_long(int mode) {
    return mode == kLossLong || mode == kDzLong || mode == kProductsLong;
}
__host__ __device__ constexpr int steps_at_a_time(int mode) {
    return is_products(mode) ? kSumSteps : kLogitSteps;
}
// What a tile of the last is.
enum Kind { kDh, kDw };

struct HeadArgs {
    // live tokens, and (backward) the scale taken out of dz; null: tokens are rows as they are,
    // n_rows of them
    const int32_t* counts;
    const int32_t* label;         // of the live tokens, as the rest; or null, and
    const void* labels;           // of all, int32 or int64
    const float* lse;
    const float* grad;
    float2* parts;                // [rows][parts_pitch]: maximum and sum of a tile
    float* picked;                // z[label]
    // Row by row 128 bytes, whose 16-byte words are in the order that 128-byte swizzling
    // gives them in shared memory: word j of row r is at j ^ (r % 8).
    uint16_t* dz;                 // [blocks of 64 columns][rows][64]
    float* sums;                  // [splits][blocks of 32 columns][rows][32]
    uint16_t* grad_table;         // the piece's first row
    int64_t parts_pitch, rows;
    int32_t first;                // the piece's first row of the table, and its rows
    int32_t vocab;
    int32_t dim;
    int32_t splits;               // of the sum in the hidden states' gradient
    int32_t blocks;               // of 64 columns of the piece
    int32_t want_h, want_w;       // the hidden states' gradient, the table's
    int32_t add_h, add_w;         // to the sums, to the table's gradient, that are there
    int32_t wide;                 // rows of the table's gradient on 16-byte boundaries
    int32_t width;                // columns of a tile, a multiple of 32 (dz: of 64)
    int32_t width_h, width_w;     // of the two products' tiles
    int32_t part;                 // of a row's maxima and sums, the piece's first
    int32_t n_rows;
    int32_t label64;
    int32_t group;                // tiles along M that are worked on together
    int* status;                  // the device status word (set by the launch)
};

struct Shared {
    uint64_t full[kStages], empty[kStages], done[2], taken[2];
    int* status;
    uint32_t tmem;
    int stop;
};

// Waits for a phase; false when the CTA is to stop.
__device__ __noinline__ bool wait_long(volatile int* stop, int* status, uint32_t bar,
                                       uint32_t parity) {
    return bar_wait(bar, parity, stop, status, kHeadWaitNs);
}
template <class S>
__device__ __forceinline__ bool wait(S& sh, uint64_t& bar, uint32_t parity) {
    const uint32_t b = smem_address(&bar);
    return bar_try(b, parity) || wait_long(&sh.stop, sh.status, b, parity);
}

__device__ __forceinline__ int live_rows(const HeadArgs& a) {
    return a.counts != nullptr ? *a.counts : a.n_rows;
}
// What is taken out of dz before it is rounded to bf16, and put back to the products' sums:
// the mantissa, 1 <= m < 2, of the largest finite gradient of a loss.  Where all are alike
// (one over the tokens), their rounding would be the same error in every term, which no sum
// averages away; so it is none (817 live tokens, 32003 x 770: both gradients
// 0.0023 off, 0.0019 so, of which 0.0017 is their own rounding).
__device__ __forceinline__ float scale_of(const int32_t* counts) {
    return __int_as_float(counts[1]);
}
__device__ __forceinline__ int32_t scale_from(float largest) {
    return (__float_as_int(largest) & 0x7FFFFF) | 0x3F800000;
}
// Whether dz is in two parts: so few live tokens that the rows of the tile's second half take
// what rounding to bf16 left of the first half's.  (One live token, 20000 x 4096: gradients
// off by up to 0.0041, 0.0017 so.  32 tokens, 50257 x 768 91 us, in one part 89; 128 tokens,
// 128000 x 4096 774 us and 745.)
__device__ __forceinline__ bool dz_in_two(int live) { return live <= kHalf; }
// A row's label in the piece, or another number.
__device__ __forceinline__ int label_in_piece(const HeadArgs& a, int row) {
    if (a.label != nullptr) return a.label[row] - a.first;
    const int64_t y = a.label64 ? static_cast<const int64_t*>(a.labels)[row]
                                : static_cast<const int32_t*>(a.labels)[row];
    return y >= a.first && y < a.first + a.vocab ? static_cast<int>(y - a.first) : -1;
}

// The operands of a launch; the last two of kProducts' second kind of tiles.
struct HeadMaps {
    CUtensorMap a, b, aw, bw;
};

// A grid of tiles.
struct Grid {
    int m_tiles, n_tiles, steps, splits, group, total;
    struct At {
        int m, n, split, begin, end;          // rows / 256, columns / width, steps along K
    };
    __device__ Grid(int m, int n, int k, int width, int parts, int together)
        : m_tiles((m + kPairTile - 1) / kPairTile),
          n_tiles((n + width - 1) / width),
          steps((k + kTileK - 1) / kTileK),
          splits(parts),
          group(together),
          total(m_tiles * n_tiles * parts) {}
    __device__ __forceinline__ At operator()(int i) const {
        At t;
        const int per = m_tiles * n_tiles;
        t.split = splits == 1 ? 0 : i / per;
        i -= t.split * per;
        const int g = i / (group * n_tiles);
        i -= g * group * n_tiles;
        const int height = min(group, m_tiles - g * group);
        t.n = i / height;
        t.m = g * group + i - t.n * height;
        t.begin = splits == 1 ? 0 : static_cast<int>(static_cast<int64_t>(steps) * t.split / splits);
        t.end = splits == 1 ? steps
                            : static_cast<int>(static_cast<int64_t>(steps) * (t.split + 1) / splits);
        return t;
    }
};

// The tiles of a launch, in the order in which the pairs take them: call(kind, tile).
template <int MODE>
struct Tiles {
    Grid first, second;
    int total;
    __device__ Tiles(const HeadArgs& a, int live)
        : first(!is_products(MODE) ? Grid(live, a.vocab, a.dim, a.width, 1, a.group)
                                  : Grid(a.want_h ? live : 0, a.dim, a.vocab, a.width_h, a.splits,
                                         a.group)),
          // (nothing to add: the table's gradient stays untouched; dz in two parts: the steps
          // along the tokens twice)
          second(!is_products(MODE) || !a.want_w || (a.add_w && live == 0) ? 0 : a.vocab, a.dim,
                 dz_in_two(live) ? 2 * ((live + kTileK - 1) / kTileK) * kTileK : live,
                 !is_products(MODE) ? kPairTile : a.width_w, 1, a.group),
          total(first.total + second.total) {}
    template <class F>
    __device__ __forceinline__ void operator()(int i, F&& call) const {
        if constexpr (!is_products(MODE)) {
            call(std::integral_constant<int, -1>{}, first(i));
        } else if (i < first.total) {
            call(std::integral_constant<int, kDh>{}, first(i));
        } else {
            call(std::integral_constant<int, kDw>{}, second(i - first.total));
        }
    }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A warp's piece of a tile on its way to memory: 32 rows of 128 bytes in shared memory, the
// 16-byte words of row r in the order j ^ (r % 8), so that lanes may write a row each and
// read rows side by side without meeting in a bank.  (The tensor cores and the copies of
// operands keep shared memory busy, and what a result costs there it costs the products: a
// piece goes to memory by one bulk copy where memory is laid out like it.)
struct Stage {
    char* at;                     // 4 KB of this warp's
    int lane;
    __device__ __forceinline__ uint4& word(int r, int j) const {
        return *reinterpret_cast<uint4*>(at + 128 * r + 16 * (j ^ (r & 7)));
    }
    __device__ __forceinline__ float& value(int r, int c) const {       // of 32 fp32 values
        return *reinterpret_cast<float*>(at + 128 * r + 16 * ((c / 4) ^ (r & 7)) + 4 * (c % 4));
    }
    __device__ __forceinline__ uint16_t& value16(int r, int c) const {  // of 64 bf16 values
        return *reinterpret_cast<uint16_t*>(at + 128 * r + 16 * ((c / 8) ^ (r & 7)) + 2 * (c % 8));
    }
    // half of this lane's row: 32 of 64 bf16 values
    __device__ __forceinline__ void put_half(const Pair (&v)[16], int half) const {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            word(lane, 4 * half + j) = make_uint4(narrow2(v[4 * j]), narrow2(v[4 * j + 1]),
                                                  narrow2(v[4 * j + 2]), narrow2(v[4 * j + 3]));
    }
    // All of the warp's rows are there: on their way, and the place to be written again.
    __device__ __forceinline__ void send(void* to, bool add) const {
        share_writes();
        __syncwarp();
        if (lane == 0) {
            if (add) bulk_add(static_cast<float*>(to), smem_address(at), 4096);
            else bulk_store(to, smem_address(at), 4096);
        }
    }
    __device__ __forceinline__ void sent() const {
        if (lane == 0) bulk_wait_read();
        __syncwarp();
    }
    // this lane's row: 32 fp32 values
    __device__ __forceinline__ void put(const float (&v)[32]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            word(lane, j) = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                       __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
    }
};

// The result of a tile, by warps: each has 32 rows (its lanes') and half of the columns, in
// up to four parts of 32.
template <int MODE, int KIND>
struct Epilogue {
    const HeadArgs& a;
    Stage stage;
    float2 (*both)[kHalf];        // what the second half of the columns found, by row
    int live, place, half, lane;  // place: this warp's first row of the CTA's 128
    int width, begin, parts;             // this warp's columns: 32 begin ..., of the tile's
    float scale;                         // taken out of dz
    __device__ Epilogue(const HeadArgs& args, int n_live, char* staging, float2 (*found)[kHalf],
                        int warp, int l)
        : a(args),
          stage{staging, l},
          both(found),
          live(n_live),
          place(warp % 4 * 32),
          half((warp - 2) / 4),
          lane(l),
          width(!is_products(MODE) ? args.width : KIND == kDh ? args.width_h : args.width_w),
          scale(is_dz(MODE) || (is_products(MODE) && KIND == kDw) ? scale_of(args.counts) : 1.0f) {
        // the first half has the odd part
        constexpr int kUnit = is_dz(MODE) ? 2 : 1;
        const int all = width / 32, first = (all / kUnit + 1) / 2 * kUnit;
        begin = half == 0 ? 0 : first;
        parts = half == 0 ? first : all - first;
    }

    // `row0` of the launch's M: this warp's first; n: columns / width; `slot`: 0 and 1 in turn;
    // `each(f)` calls f(c, v) with columns 32 c ... of this warp's, c < parts
    template <class Each>
    __device__ __forceinline__ void operator()(int row0, int n, int split, int slot,
                                               Each&& each) const {
        const int column = n * width + 32 * begin;
        const int row = row0 + lane;
        if constexpr (is_loss(MODE)) {
            const int left = a.vocab - column;           // columns that exist
            const int mine = row < live ? label_in_piece(a, row) - column : -1;
            float top = -INFINITY, sum = 0.0f, z = 0.0f;
            each([&](int c, float (&v)[32]) {
                if (32 * c + 32 > left) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * c + i >= left) v[i] = -INFINITY;
                }
                if (mine >= 32 * c && mine < 32 * c + 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (mine == 32 * c + i) z = v[i];
                }
                float m = v[0];
#pragma unroll
                for (int i = 1; i < 32; ++i) m = fmaxf(m, v[i]);
                m = fmaxf(top, m);
                // Differences before anything is multiplied: they are as exact as logits of
                // any size hold them.  (-inf alone: no term)
                const float from = m == -INFINITY ? 0.0f : m;
                const Pair by = pair(kLog2e, kLog2e), minus = pair(-from, -from);
                sum *= exp2_fast((top - from) * kLog2e);
                Pair t = 0;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 x = unpair(mul2(add2(pair(v[i], v[i + 1]), minus), by));
                    t = add2(t, pair(exp2_fast(x.x), exp2_fast(x.y)));
                }
                const float2 s = unpair(t);
                sum += s.x + s.y;
                top = m;
            });
            if (mine >= 0 && mine < min(32 * parts, left)) a.picked[row] = z;
            // the two halves of the columns
            if (half == 1) both[slot][place + lane] = make_float2(top, sum);
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpilogueWarps) : "memory");
            if (half == 0 && row < live) {
                const float2 o = both[slot][place + lane];
                const float m = fmaxf(top, o.x), from = m == -INFINITY ? 0.0f : m;
                a.parts[row * a.parts_pitch + a.part + n] = make_float2(
                    m, sum * exp2_fast((top - from) * kLog2e) +
                           o.y * exp2_fast((o.x - from) * kLog2e));
            }
        } else if constexpr (is_dz(MODE)) {
            const bool two = dz_in_two(live), rest = two && row0 >= kHalf;   // of the warp
            const int token = two ? row % kHalf : row;
            const bool in = token < live;
            const int mine = in ? a.label[token] - a.first - column : -1;
            const float off = in ? -a.lse[token] : 0.0f;
            const float g = in ? a.grad[token] / scale : 0.0f;
            const Pair by = pair(kLog2e, kLog2e), minus = pair(off, off), times = pair(g, g);
            each([&](int c, float (&v)[32]) {
                // z - lse before anything is multiplied: of large logits only their
                // difference counts, and where it is small it is exact.
                Pair y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 x =
                        unpair(mul2(add2(pair(v[2 * i], v[2 * i + 1]), minus), by));
                    y[i] = mul2(pair(exp2_fast(x.x), exp2_fast(x.y)), times);
                }
                // Rows beyond the live ones are zeros in the hidden states' copy, but a table's
                // infinity makes NaN of them.
                if (!in) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = 0;
                }
                if (mine >= 32 * c && mine < 32 * c + 32) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (mine / 2 == 16 * c + i)
                            y[i] = add2(y[i], mine % 2 == 0 ? pair(-g, 0.0f) : pair(0.0f, -g));
                    }
                }
                const int first = column + 32 * c;
                if (first >= a.blocks * 64) return;
                if (first + 32 > a.vocab) {              // the sum over the vocabulary reads on
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 x = unpair(y[i]);
                        y[i] = pair(first + 2 * i < a.vocab ? x.x : 0.0f,
                                    first + 2 * i + 1 < a.vocab ? x.y : 0.0f);
                    }
                }
                if (rest) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        y[i] = fma2(widen2(narrow2(y[i])), pair(-1.0f, -1.0f), y[i]);
                }
                if (c % 2 == 0) stage.sent();
                stage.put_half(y, c % 2);
                if (c % 2 == 1)
                    stage.send(a.dz + (first / 64 * a.rows + row0) * 64, false);
            });
        } else if constexpr (KIND == kDh) {
            const int blocks = (a.dim + 31) / 32;
            each([&](int c, float (&v)[32]) {
                const int block = column / 32 + c;
                if (block >= blocks) return;
                stage.sent();
                stage.put(v);
                stage.send(a.sums + ((static_cast<int64_t>(split) * blocks + block) * a.rows + row0) * 32,
                           a.add_h != 0);
            });
        } else if (a.add_w == 0) {
            stage.sent();                                // (an earlier tile's)
            each([&](int c, float (&v)[32]) {
                Pair y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[i] = mul2(pair(v[2 * i], v[2 * i + 1]), pair(scale, scale));
                stage.put_half(y, c % 2);
                if (c % 2 == 0 && c + 1 < parts) return;
                __syncwarp();
                const int first = column + 32 * (c - c % 2);          // 64 columns, or 32
                const int end = min(a.dim, column + 32 * (c + 1));
                if (a.wide) {
                    const int col = first + lane % 8 * 8;
                    if (col < end) {
                        uint16_t* to =
                            a.grad_table + static_cast<int64_t>(row0 + lane / 8) * a.dim + col;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = lane / 8 + 4 * i;
                            if (row0 + r < a.vocab)
                                *reinterpret_cast<uint4*>(to + static_cast<int64_t>(4 * i) * a.dim) =
                                    stage.word(r, lane % 8);
                        }
                    }
                } else {
                    // Rows off the 16-byte grid: a row's whole aligned words, shifted into
                    // place, by 8 lanes, and the values before and after them one by one.
                    const int wide = end - first, rows = min(32, a.vocab - row0);
                    uint16_t* const to = a.grad_table + static_cast<int64_t>(row0) * a.dim + first;
                    auto head_of = [&](const uint16_t* p) {
                        return min(static_cast<int>(-(reinterpret_cast<uintptr_t>(p) / 2) & 7), wide);
                    };
#pragma unroll 4
                    for (int i = 0; i < 8; ++i) {
                        const int r = lane / 8 + 4 * i, w = lane % 8;
                        if (r >= rows) continue;
                        uint16_t* const p = to + static_cast<int64_t>(r) * a.dim;
                        const int head = head_of(p), tail = head + (wide - head) / 8 * 8;
                        if (head + 8 * w < tail)
                            *reinterpret_cast<uint4*>(p + head + 8 * w) =
                                shifted<uint16_t>(stage.word(r, w), stage.word(r, (w + 1) & 7), 2 * head);
#pragma unroll
                        for (int e = w; e < 16; e += 8) {
                            const int at = e < head ? e : tail + e - head;
                            if (at < wide) p[at] = stage.value16(r, at);
                        }
                    }
                }
                __syncwarp();
            });
        } else {
            stage.sent();
            each([&](int c, float (&v)[32]) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= scale;
                stage.put(v);
                __syncwarp();
                const int first = column + 32 * c;
                if (a.wide) {                            // 8 columns a lane, 8 rows at a time
                    const int col = first + lane % 4 * 8;
                    if (col < a.dim) {
                        uint16_t* to =
                            a.grad_table + static_cast<int64_t>(row0 + lane / 4) * a.dim + col;
                        const int64_t step = static_cast<int64_t>(8) * a.dim;
                        uint4 old[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            old[i] = make_uint4(0, 0, 0, 0);
                            if (row0 + lane / 4 + 8 * i < a.vocab)
                                old[i] = *reinterpret_cast<const uint4*>(to + i * step);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = lane / 4 + 8 * i;
                            const uint4 lo = stage.word(r, lane % 4 * 2);
                            const uint4 hi = stage.word(r, lane % 4 * 2 + 1);
                            Pair x[4] = {pair(__uint_as_float(lo.x), __uint_as_float(lo.y)),
                                         pair(__uint_as_float(lo.z), __uint_as_float(lo.w)),
                                         pair(__uint_as_float(hi.x), __uint_as_float(hi.y)),
                                         pair(__uint_as_float(hi.z), __uint_as_float(hi.w))};
                            x[0] = add2(x[0], widen2(old[i].x));
                            x[1] = add2(x[1], widen2(old[i].y));
                            x[2] = add2(x[2], widen2(old[i].z));
                            x[3] = add2(x[3], widen2(old[i].w));
                            if (row0 + r < a.vocab)
                                *reinterpret_cast<uint4*>(to + i * step) = make_uint4(
                                    narrow2(x[0]), narrow2(x[1]), narrow2(x[2]), narrow2(x[3]));
                        }
                    }
                } else {                                 // a column a lane, 8 rows at a time
                    // (7 tokens, 100000 x 4000 1.61 ms; row by row 4.30, by 16 1.56 and
                    // registers spilled, 3 % of the other forms)
                    const int col = first + lane;
                    if (col < a.dim) {
                        uint16_t* to = a.grad_table + static_cast<int64_t>(row0) * a.dim + col;
                        const int rows = min(32, a.vocab - row0);
#pragma unroll 1
                        for (int r0 = 0; r0 < rows; r0 += 8) {
                            uint16_t old[8];
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                old[r] = 0;
                                if (r0 + r < rows) old[r] = to[static_cast<int64_t>(r0 + r) * a.dim];
                            }
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                if (r0 + r < rows)
                                    to[static_cast<int64_t>(r0 + r) * a.dim] = float_to_bf16_rn(
                                        stage.value(r0 + r, lane) + bf16_to_float(old[r]));
                        }
                    }
                }
                __syncwarp();
            });
        }
    }
};

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kHeadThreads, 1)
head_kernel(const __grid_constant__ HeadMaps maps, const __grid_constant__ HeadArgs a) {
    constexpr bool kBmn = is_products(MODE);             // B is MN-major; A for kDw
    extern __shared__ char dyn[];
    __shared__ Shared sh;
    const uint32_t ring = (smem_address(dyn) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            bar_init(smem_address(&sh.full[s]), 1);
            bar_init(smem_address(&sh.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_address(&sh.done[i]), 1);
            bar_init(smem_address(&sh.taken[i]), 2 * kEpilogueWarps);
        }
        sh.stop = 0;
        sh.status = a.status;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane < (is_products(MODE) ? 4 : 2)) prefetch_map(&maps.a + lane);
    if (warp == 1) tmem_alloc(smem_address(&sh.tmem), kTmemColumns);
    fence_before_sync();
    __syncthreads();
    cluster_sync();
    fence_after_sync();
    const uint32_t tmem = sh.tmem;
    let_next_launch_begin();
    wait_for_launch_before();
    const int live = live_rows(a);
    const bool two = !is_loss(MODE) && dz_in_two(live);
    const Tiles<MODE> tiles(a, live);

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 1;
            bool run = true;
            for (int i = pair; run && i < tiles.total; i += pairs) {
                tiles(i, [&](auto kind, const Grid::At& t) {
                    constexpr int KIND = decltype(kind)::value;
                    const int width = KIND == kDh   ? a.width_h
                                      : KIND == kDw ? a.width_w
                                                    : a.width;
                    const bool two_chunks = width > 128; // of B, where it is MN-major
                    const uint32_t bytes =
                        2 * (kOperandBytes +
                             (kBmn ? (two_chunks ? 2 : 1) * kChunkBytes : width / 2 * 128));
                    // (dz in two parts: both CTAs have the same tokens' logits)
                    const int m0 = t.m * kPairTile +
                                   (is_dz(MODE) && two ? 0 : static_cast<int>(rank) * kHalf);
                    const int steps = t.end / 2;         // of a part of dz, for kDw
                    const int n0 = t.n * width + static_cast<int>(rank) * (width / 2);
                    const CUtensorMap* map_a = KIND == kDw ? &maps.aw : &maps.a;
                    const CUtensorMap* map_b = KIND == kDw ? &maps.bw : &maps.b;
                    for (int k = t.begin; k < t.end; ++k) {
                        if (!wait(sh, sh.empty[s], phase)) {
                            run = false;
                            return;
                        }
                        const uint32_t bar = smem_address(&sh.full[s]);
                        const uint32_t to_a = ring + s * kStageBytes, to_b = to_a + kOperandBytes;
                        if (rank == 0) bar_expect(bar, bytes);
                        const bool rest = KIND == kDw && two && k >= steps;
                        const int k0 = (rest ? k - steps : k) * kTileK;
                        if constexpr (KIND == kDw) {
                            const int row = k0 + (rest ? kHalf : 0);
                            tma_load(to_a, map_a, 0, row, m0 / 64, bar);
                            tma_load(to_a + kChunkBytes, map_a, 0, row, m0 / 64 + 1, bar);
                        } else if constexpr (KIND == kDh) {
                            tma_load(to_a, map_a, 0, m0, k, bar);
                        } else {
                            tma_load(to_a, map_a, k * kTileK, m0, bar);
                        }
                        if constexpr (kBmn) {
                            tma_load(to_b, map_b, n0, k0, bar);
                            if (two_chunks) tma_load(to_b + kChunkBytes, map_b, n0 + 64, k0, bar);
                        } else {
                            tma_load(to_b, map_b, k * kTileK, n0, bar);
                        }
                        if (++s == kStages) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                });
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            int s = 0, n = 0;
            uint32_t phase = 0;
            bool run = true;
            for (int i = pair; run && i < tiles.total; i += pairs) {
                tiles(i, [&](auto kind, const Grid::At& t) {
                    constexpr int KIND = decltype(kind)::value;
                    constexpr bool kAmn = KIND == kDw;
                    if (t.begin == t.end) return;
                    const uint32_t form = product_form(kAmn, kBmn,
                                                       KIND == kDh   ? a.width_h
                                                       : KIND == kDw ? a.width_w
                                                                     : a.width);
                    // a result in tensor memory: of all steps, or of some (is_long)
                    for (int begin = t.begin; begin < t.end;) {
                        const int end = is_long(MODE) ? min(begin + steps_at_a_time(MODE), t.end) : t.end;
                        const int slot = n % 2;
                        run = wait(sh, sh.taken[slot], (n / 2 + 1) % 2);
                        if (!run) return;
                        ++n;
                        fence_after_sync();
                        const uint32_t d = tmem + slot * kPairTile;
                        for (int k = begin; k < end; ++k) {
                            run = wait(sh, sh.full[s], phase);
                            if (!run) return;
                            fence_after_sync();
                            const uint32_t at = ring + s * kStageBytes;
                            const uint64_t da = operand(at, kAmn ? kChunkBytes : 16);
                            const uint64_t db = operand(at + kOperandBytes, kBmn ? kChunkBytes : 16);
#pragma unroll
                            for (int j = 0; j < kTileK / 16; ++j) {
                                // 16 values along K: 32 bytes of a row, or 16 rows
                                product(d, da + (kAmn ? 16 * 128 : 32) / 16 * j,
                                        db + (kBmn ? 16 * 128 : 32) / 16 * j, form,
                                        k != begin || j != 0);
                            }
                            products_arrive(smem_address(&sh.empty[s]));
                            if (++s == kStages) {
                                s = 0;
                                phase ^= 1;
                            }
                        }
                        products_arrive(smem_address(&sh.done[slot]));
                        begin = end;
                    }
                });
            }
        }
    } else {
        // (the forward pass stages nothing: its halves meet there)
        char* const staging = dyn + (ring - smem_address(dyn)) + kStages * kStageBytes;
        char* const mine = staging + (warp - 2) * kStagingBytes;
        float2(*const both)[kHalf] = reinterpret_cast<float2(*)[kHalf]>(staging);
        const Epilogue<MODE, kDh> epilogue_h(a, live, mine, both, warp, lane);
        const Epilogue<MODE, kDw> epilogue_w(a, live, mine, both, warp, lane);
        int n = 0, turn = 0;
        for (int i = pair; i < tiles.total; i += pairs, turn ^= 1) {
            tiles(i, [&](auto kind, const Grid::At& t) {
                constexpr int KIND = decltype(kind)::value;
                const auto& epilogue = [&]() -> const auto& {
                    if constexpr (KIND == kDw) return epilogue_w;
                    else return epilogue_h;
                }();
                const int parts = epilogue.parts;
                const int row0 = t.m * kPairTile + static_cast<int>(rank) * kHalf + epilogue.place;
                if (t.begin == t.end) {                  // a sum of nothing
                    epilogue(row0, t.n, t.split, 0, [&](auto&& f) {
#pragma unroll 1
                        for (int c = 0; c < parts; ++c) {
                            float v[32] = {};
                            f(c, v);
                        }
                    });
                    return;
                }
                // the next result in tensor memory (a wait that runs out: on with what is
                // there, so that no warp waits for another)
                auto come = [&] {
                    const int at = n % 2;
                    wait(sh, sh.done[at], (n / 2) % 2);
                    __syncwarp();
                    ++n;
                    fence_after_sync();
                    return at;
                };
                auto place = [&](int at) {
                    return tmem + at * kPairTile + 32 * epilogue.begin +
                           (static_cast<uint32_t>(epilogue.place) << 16);
                };
                auto free_place = [&](int at) {          // ... may be taken again
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) bar_arrive_in_cluster(in_cta(smem_address(&sh.taken[at]), 0));
                };
                const int slot = come();
                const uint32_t from = place(slot);
                auto release = [&] { free_place(slot); };
                epilogue(row0, t.n, t.split, turn, [&](auto&& f) {
                    constexpr int kPart = steps_at_a_time(MODE);
                    if constexpr (MODE == kProductsLong) {
                        // (sums in local memory: what they cost there is small beside the
                        // many steps of a part, and the results' code stays as short as below)
                        float sum[4][32];
                        for (int k = t.begin; k < t.end; k += kPart) {
                            const int at = k == t.begin ? slot : come();
#pragma unroll 1
                            for (int c = 0; c < parts; ++c) {
                                float v[32];
                                tmem_load(v, place(at) + 32 * c);
                                tmem_load_wait(v);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    sum[c][e] = k == t.begin ? v[e] : sum[c][e] + v[e];
                            }
                            free_place(at);
                        }
#pragma unroll 1
                        for (int c = 0; c < parts; ++c) {
                            f(c, sum[c]);
                            __syncwarp();
                        }
                        return;
                    }
                    if constexpr (is_long(MODE)) {
                        float sum[4][32];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c < parts) tmem_load(sum[c], from + 32 * c);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_load_wait(sum[c]);
                        release();
                        for (int k = t.begin + kPart; k < t.end; k += kPart) {
                            const int next = come();
                            const uint32_t more = place(next);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                if (c >= 2 * parts) break;
                                float v[16];
                                tmem_load(v, more + 16 * c);
                                tmem_load_wait(v);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    sum[c / 2][16 * (c % 2) + e] += v[e];
                            }
                            free_place(next);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c < parts) f(c, sum[c]);
                        }
                        return;
                    }
                    if constexpr (KIND == kDw) {         // (registers are short)
                        if (parts == 0) release();
#pragma unroll 1
                        for (int c = 0; c < parts; ++c) {
                            float v[32];
                            tmem_load(v, from + 32 * c);
                            tmem_load_wait(v);
                            if (c + 1 == parts) release();
                            f(c, v);
                            __syncwarp();
                        }
                        return;
                    }
                    // the next part is on its way while one is worked on
                    float v[2][32];
                    if (parts > 0) {
                        tmem_load(v[0], from);
                        tmem_load_wait(v[0]);
                    }
                    if (parts <= 1) release();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c >= parts) break;
                        if (c < 3 && c + 1 < parts) tmem_load(v[(c + 1) % 2], from + 32 * (c + 1));
                        f(c, v[c % 2]);
                        __syncwarp();
                        if (c < 3 && c + 1 < parts) {
                            tmem_load_wait(v[(c + 1) % 2]);
                            if (c + 2 == parts) release();
                        }
                    }
                });
            });
        }
        if (!is_loss(MODE) && lane == 0) bulk_wait();
    }
    __syncwarp();
    __syncthreads();
    if (sh.stop) {
        // what is still on its way to shared or tensor memory gets time to come
        const uint64_t t0 = now_ns();
        while (now_ns() - t0 < 20000000ull) {}
    }
    fence_before_sync();
    cluster_sync();
    fence_after_sync();
    if (warp == 1) tmem_free(tmem, kTmemColumns);
}

// ---------------------------------------------------------- few tokens ------

// The forward pass of up to 64 tokens, bound by reading the table: the vocabulary on the
// products' rows, 128 at a time, so that the tokens' side is small and a CTA by itself streams
// its share of the table, even to 16 rows, by a deep ring.  A thread keeps a running maximum
// and sum of each token over its rows of all tiles; they are joined at the end, one part of a
// row's statistics a CTA.  32 tokens x 50257 x 768 19.5 us (head_kernel 26.4), of which 5.6
// are two launches and an end of any size and the rest reads the table at 5.5 TB/s; 131072 x
// 4096 158 to 162 us, 6.8 to 6.6 TB/s (1 to 8 tokens with head_kernel 216 to 233).  The
// maximum and sum kept by one exponential a logit, labels looked for once in a warp's 32 rows:
// 2 us less a call.
constexpr int kFewMost = 64;
constexpr int kFewUnit = 16;                         // rows of the table
// (two warps that load and issue, and four that read 32 tokens' sums)
__host__ __device__ constexpr int few_threads(int tokens) { return 64 + 4 * tokens; }
constexpr int kFewMostStages = 10;
__host__ __device__ constexpr uint32_t few_stage(int tokens) {
    return kOperandBytes + tokens * 128u;
}
__host__ __device__ constexpr int few_stages(int tokens) { return tokens == 32 ? 10 : 8; }
__host__ __device__ constexpr size_t few_smem(int tokens) {
    return few_stages(tokens) * few_stage(tokens) + 1024;
}

struct FewArgs {
    const void* labels;
    float2* parts;                // [n_rows][CTAs]
    float* picked;
    int32_t n_rows;
    int32_t vocab;
    int32_t dim;
    int32_t label64;
    int* status;                  // the device status word
};
struct FewMaps {
    // 128 rows of the table, what the smaller and the larger shares have beyond whole tiles, and
    // the tokens.  (A copy for each 16 rows instead:
    // 32 tokens, 131072 x 4096 176 us, 163 with these.)
    CUtensorMap tile, rest[2], tokens;
};
struct FewShared {
    uint64_t full[kFewMostStages], empty[kFewMostStages], done[2], taken[2];
    int* status;
    uint32_t tmem;
    int stop;
};

// A maximum of logits, -FLT_MAX before any, and a sum of exponentials, joined with another.
__device__ __forceinline__ void join(float& top, float& sum, float t, float s) {
    const float m = fmaxf(top, t);
    sum = sum * exp2_fast((top - m) * kLog2e) + s * exp2_fast((t - m) * kLog2e);
    top = m;
}

template <int TOKENS>
__global__ void __launch_bounds__(few_threads(TOKENS), 1)
head_few_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a) {
    constexpr int kRing = few_stages(TOKENS);
    extern __shared__ char dyn[];
    __shared__ FewShared sh;
    const uint32_t ring = (smem_address(dyn) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; ++s) {
            bar_init(smem_address(&sh.full[s]), 1);
            bar_init(smem_address(&sh.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_address(&sh.done[i]), 1);
            bar_init(smem_address(&sh.taken[i]), TOKENS / 8);
        }
        sh.stop = 0;
        sh.status = a.status;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane < 4) prefetch_map(&maps.tile + lane);
    if (warp == 1) single::tmem_alloc(smem_address(&sh.tmem), 2 * kFewMost);
    let_next_launch_begin();
    wait_for_launch_before();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const int64_t units = (a.vocab + kFewUnit - 1) / kFewUnit;
    const int begin = static_cast<int>(units * blockIdx.x / gridDim.x);
    const int end = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    const int steps = (a.dim + kTileK - 1) / kTileK;
    constexpr int kUnits = kHalf / kFewUnit;             // of a tile

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 1;
            bool run = true;
            const bool more = end - begin > units / gridDim.x;
            for (int u = begin; run && u < end; u += kUnits) {
                const int n = min(kUnits, end - u);
                const CUtensorMap* const rows = n == kUnits ? &maps.tile : &maps.rest[more];
                for (int k = 0; k < steps; ++k) {
                    run = wait(sh, sh.empty[s], phase);
                    if (!run) break;
                    const uint32_t bar = smem_address(&sh.full[s]);
                    const uint32_t to = ring + s * few_stage(TOKENS);
                    bar_expect(bar, n * kFewUnit * 128 + TOKENS * 128);
                    single::tma_load(to, rows, k * kTileK, u * kFewUnit, bar);
                    single::tma_load(to + kOperandBytes, &maps.tokens, k * kTileK, 0, bar);
                    if (++s == kRing) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int s = 0, n = 0;
            uint32_t phase = 0;
            bool run = true;
            for (int u = begin; run && u < end; u += kUnits) {
                // (rows of a tile beyond the CTA's share: what an earlier tile left there)
                for (int from = 0; run && from < steps; from += kLogitSteps) {
                    const int slot = n % 2;
                    run = wait(sh, sh.taken[slot], (n / 2 + 1) % 2);
                    if (!run) break;
                    ++n;
                    fence_after_sync();
                    const uint32_t d = tmem + slot * kFewMost;
                    for (int k = from; k < min(from + kLogitSteps, steps); ++k) {
                        run = wait(sh, sh.full[s], phase);
                        if (!run) break;
                        fence_after_sync();
                        const uint32_t at = ring + s * few_stage(TOKENS);
                        const uint64_t da = operand(at, 16), db = operand(at + kOperandBytes, 16);
#pragma unroll
                        for (int j = 0; j < kTileK / 16; ++j)
                            single::product(d, da + 2 * j, db + 2 * j, single::product_form(TOKENS),
                                            k != from || j != 0);
                        single::products_arrive(smem_address(&sh.empty[s]));
                        if (++s == kRing) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                    if (run) single::products_arrive(smem_address(&sh.done[slot]));
                }
            }
        }
    } else {
        const int part = warp % 4;                       // of tensor memory's lanes
        const int first = (warp - 2) / 4 * 32;           // of the warp's tokens
        int label = -1;                                  // of the lane's token
        if (first + lane < a.n_rows) {
            const int64_t y = a.label64 ? static_cast<const int64_t*>(a.labels)[first + lane]
                                        : static_cast<const int32_t*>(a.labels)[first + lane];
            if (y >= 0 && y < a.vocab) label = static_cast<int>(y);
        }
        float top[32], sum[32];
#pragma unroll
        for (int t = 0; t < 32; ++t) {
            top[t] = -FLT_MAX;
            sum[t] = 0.0f;
        }
        int n = 0;
        for (int u = begin; u < end; u += kUnits) {
            const int place = part * 32 + lane, row = u * kFewUnit + place;
            const bool in = place < (end - u) * kFewUnit && row < a.vocab;
            float z[32];
            for (int from = 0; from < steps; from += kLogitSteps) {
                const int slot = n % 2;
                wait(sh, sh.done[slot], (n / 2) % 2);
                __syncwarp();
                ++n;
                fence_after_sync();
                float v[32];
                tmem_load(v, tmem + slot * kFewMost + first +
                                 (static_cast<uint32_t>(part * 32) << 16));
                tmem_load_wait(v);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) single::bar_arrive(smem_address(&sh.taken[slot]));
#pragma unroll
                for (int t = 0; t < 32; ++t) z[t] = from == 0 ? v[t] : z[t] + v[t];
            }
            // Few labels are in a warp's 32 rows.
            if (__any_sync(0xFFFFFFFFu, static_cast<uint32_t>(label - (row - lane)) < 32u)) {
#pragma unroll
                for (int t = 0; t < 32; ++t) {
                    const int of_t = __shfl_sync(0xFFFFFFFFu, label, t);
                    if (in && of_t == row) a.picked[first + t] = z[t];
                }
            }
            // One exponential a logit: the larger of it and the maximum counts 1.
#pragma unroll
            for (int t = 0; t < 32; ++t) {
                const float x = in ? z[t] : -INFINITY, d = x - top[t];
                const bool up = x > top[t];
                const float e = exp2_fast((up ? -d : d) * kLog2e);
                sum[t] = up ? __fmaf_rn(sum[t], e, 1.0f) : sum[t] + e;
                top[t] = up ? x : top[t];
            }
        }
        // Over the CTA's rows, through the ring: every copy into it and product from it has
        // come before the last tile's sums.  A warp joins its own 32 rows of its tokens, a
        // lane a token, and one of four those of all.
        constexpr int kPitch = 33;
        float2* const all = reinterpret_cast<float2*>(dyn + (ring - smem_address(dyn)));
        float2* const own = all + (first * 4 + part * 32) * kPitch;
#pragma unroll
        for (int t = 0; t < 32; ++t) own[lane * kPitch + t] = make_float2(top[t], sum[t]);
        __syncwarp();
        float m = -FLT_MAX, l = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float2 o = own[i * kPitch + lane];
            top[i] = o.x;
            sum[i] = o.y;
            m = fmaxf(m, o.x);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) l += sum[i] * exp2_fast((top[i] - m) * kLog2e);
        __syncwarp();
        own[lane] = make_float2(m, l);
        asm volatile("bar.sync 1, %0;" ::"n"(4 * TOKENS) : "memory");
        if (part == 0 && first + lane < a.n_rows) {
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                const float2 o = own[i * 32 * kPitch + lane];
                join(m, l, o.x, o.y);
            }
            a.parts[(first + lane) * static_cast<int64_t>(gridDim.x) + blockIdx.x] =
                make_float2(m, l);
        }
    }
    __syncwarp();
    __syncthreads();
    if (sh.stop) {
        // what is still on its way to shared or tensor memory gets time to come
        const uint64_t t0 = now_ns();
        while (now_ns() - t0 < 20000000ull) {}
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 1) single::tmem_free(tmem, 2 * kFewMost);
}

// One CTA waiting for a phase that nothing completes.
__global__ void wait_selftest_kernel(int* status, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    __shared__ int stop;
    if (threadIdx.x == 0) {
        bar_init(smem_address(&bar), 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    bar_wait(smem_address(&bar), 0, &stop, status, limit_ns);
}

// ---------------------------------------------------------------- rows ------

// The places in the workspace that the first launches fill.
struct HeadRows {
    int32_t* counts;              // live tokens, and (backward) the scale taken out of dz
    int32_t* index;               // token of a live row
    int32_t* slot;                // live row of a token, or -1
    int32_t* label;
    float* lse;
    float* grad;
    uint16_t* hidden;
    int64_t pitch;
};

// A token's label if it is live, else -1.
__device__ __forceinline__ int32_t live_label(const HeadCall& c, int64_t t, bool back) {
    const int64_t y = c.label64 ? static_cast<const int64_t*>(c.labels)[t]
                                : static_cast<const int32_t*>(c.labels)[t];
    const bool in = (!back || c.grad_loss[t] != 0.0f) & (y >= 0) & (y < c.vocab);
    return in ? static_cast<int32_t>(y) : -1;
}

// The size of a token's gradient of the loss, if it is finite.
__device__ __forceinline__ float finite_grad(const HeadCall& c, int64_t t) {
    const float g = fabsf(c.grad_loss[t]);
    return g <= FLT_MAX ? g : 0.0f;
}

__device__ __forceinline__ void put_token(const HeadCall& c, const HeadRows& r, int64_t t,
                                          int32_t y, int32_t to, bool back) {
    r.slot[t] = y >= 0 ? to : -1;
    if (y >= 0) {
        r.index[to] = static_cast<int32_t>(t);
        r.label[to] = y;
        if (back) {
            r.lse[to] = c.lse[t];
            r.grad[to] = c.grad_loss[t];
        }
    } else if (!back) {
        c.loss[t] = 0.0f;
        if (c.lse != nullptr) c.lse[t] = 0.0f;
    }
}

// The live tokens, in order, and what the other launches read of them: by one CTA.
constexpr int kRowThreads = 1024;

__global__ void __launch_bounds__(kRowThreads)
head_rows_kernel(const HeadCall c, const HeadRows r, bool back) {
    __shared__ int32_t warps[32];
    __shared__ float grads[32];
    // a warp's tokens: whole runs of 32
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t runs = (c.n_tokens + kRowThreads - 1) / kRowThreads;
    const int64_t begin = warp * runs * 32;
    auto label_of = [&](int64_t t) { return t < c.n_tokens ? live_label(c, t, back) : -1; };
    let_next_launch_begin();
    int32_t n = 0;
    float g = 0.0f;
#pragma unroll 8
    for (int64_t i = 0; i < runs; ++i) {
        const int64_t t = begin + 32 * i + lane;
        const bool live = label_of(t) >= 0;
        n += __popc(__ballot_sync(0xFFFFFFFFu, live));
        if (back && live) g = fmaxf(g, finite_grad(c, t));
    }
    g = warp_max(g);
    if (lane == 0) {
        warps[warp] = n;
        grads[warp] = g;
    }
    __syncthreads();
    g = warp_max(grads[lane]);
    int32_t at = lane < warp ? warps[lane] : 0, all = warps[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        at += __shfl_xor_sync(0xFFFFFFFFu, at, o);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    }
    if (threadIdx.x == 0) {
        r.counts[0] = all;
        r.counts[1] = scale_from(g);
    }
#pragma unroll 4
    for (int64_t i = 0; i < runs; ++i) {
        const int64_t t = begin + 32 * i + lane;
        const int32_t y = label_of(t);
        const uint32_t live = __ballot_sync(0xFFFFFFFFu, y >= 0);
        const int32_t to = at + __popc(live & ((1u << lane) - 1));
        at += __popc(live);
        if (t < c.n_tokens) put_token(c, r, t, y, to, back);
    }
}

constexpr int kCopyWarps = 8;
constexpr int kCopyColumns = 512;

// 16 bytes of a row that starts anywhere, from the aligned words that hold them (of the
// row's first and last word bytes beside it are read, and not used).  All 16 are the row's.
__device__ __forceinline__ uint4 row_word(const uint16_t* row, int column) {
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16);
    const char* p = reinterpret_cast<const char*>(row) - mis + 2 * column;
    const uint4 lo = *reinterpret_cast<const uint4*>(p);
    if (mis == 0) return lo;
    return shifted<uint16_t>(lo, *reinterpret_cast<const uint4*>(p + 16), mis);
}

// A lane's columns of a row: 8 from `first` on, and each 256 further.
__device__ __forceinline__ void copy_columns(const uint16_t* in, uint16_t* out, int first, int dim) {
    uint4 v[kCopyColumns / 256];
#pragma unroll
    for (int i = 0; i < kCopyColumns / 256; ++i) {
        if (first + 256 * i + 8 <= dim) v[i] = row_word(in, first + 256 * i);
    }
#pragma unroll
    for (int i = 0; i < kCopyColumns / 256; ++i) {
        const int c = first + 256 * i;
        if (c + 8 <= dim) {
            *reinterpret_cast<uint4*>(out + c) = v[i];
        } else {
            for (int e = c; e < dim; ++e) out[e] = in[e];
        }
    }
}

// Rows to copy beside other work: `count` rows of dim, side by side.
struct HeadCopy {
    const uint16_t* from;
    uint16_t* to;
    int64_t count;
    int64_t pitch;
    int32_t dim;
    int32_t sections;
};

// The same and the copy of the live tokens' rows in one launch, where tokens are few: a CTA
// has 8 of them, a warp each, and counts all by itself.
constexpr int64_t kFewTokens = 8192;
constexpr int kPrepareThreads = 256;
constexpr int kPrepareTokens = kPrepareThreads / 32;

__global__ void __launch_bounds__(kPrepareThreads)
head_prepare_kernel(const HeadCall c, const HeadRows r, const HeadCopy copy, unsigned own_ctas,
                    bool back) {
    if (blockIdx.x >= own_ctas) {                        // the first piece of the table
        let_next_launch_begin();
        const int64_t id =
            static_cast<int64_t>(blockIdx.x - own_ctas) * kPrepareTokens + threadIdx.x / 32;
        const int64_t row = id / copy.sections;
        if (row < copy.count)
            copy_columns(copy.from + row * copy.dim, copy.to + row * copy.pitch,
                         static_cast<int>(id - row * copy.sections) * kCopyColumns +
                             8 * (threadIdx.x % 32),
                         copy.dim);
        return;
    }
    __shared__ int32_t before[kPrepareTokens], total[kPrepareTokens];
    __shared__ float grads[kPrepareTokens];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int n = static_cast<int>(c.n_tokens), base = blockIdx.x * kPrepareTokens;
    let_next_launch_begin();
    // the CTA's own tokens, for every warp
    const int32_t mine = lane < kPrepareTokens && base + lane < n ? live_label(c, base + lane, back) : -1;
    const uint32_t own = __ballot_sync(0xFFFFFFFFu, mine >= 0);
    int32_t b = 0, all = 0;
    float g = 0.0f;
#pragma unroll 8
    for (int t = threadIdx.x; t < n; t += kPrepareThreads) {
        const int live = live_label(c, t, back) >= 0;
        all += live;
        b += t < base ? live : 0;
        if (back && live) g = fmaxf(g, finite_grad(c, t));
    }
    g = warp_max(g);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    }
    if (lane == 0) {
        before[warp] = b;
        total[warp] = all;
        grads[warp] = g;
    }
    __syncthreads();
    b = all = 0;
#pragma unroll
    for (int w = 0; w < kPrepareTokens; ++w) {
        b += before[w];
        all += total[w];
        g = fmaxf(g, grads[w]);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        r.counts[0] = all;
        r.counts[1] = scale_from(g);
    }
    const int32_t y = __shfl_sync(0xFFFFFFFFu, mine, warp);
    const int32_t j = b + __popc(own & ((1u << warp) - 1));
    const int t = base + warp;
    if (lane == 0 && t < n) put_token(c, r, t, y, j, back);
    const int dim = static_cast<int>(c.dim);
    if (y >= 0) {
        const uint16_t* in = c.hidden + t * c.hidden_stride;
        uint16_t* out = r.hidden + j * r.pitch;
#pragma unroll 4
        for (int col = 8 * lane; col + 8 <= dim; col += 256)
            *reinterpret_cast<uint4*>(out + col) = row_word(in, col);
        const int rest = dim / 8 * 8 + lane;
        if (rest < dim) out[rest] = in[rest];
    }
    if (!back) return;
    // zeros up to whole tiles: the sums over tokens go that far
    const int rows = (all + kPairTile - 1) / kPairTile * kPairTile;
    for (int z = all + t; z < rows; z += own_ctas * kPrepareTokens) {
        for (int col = 8 * lane; col < r.pitch; col += 256)
            *reinterpret_cast<uint4*>(r.hidden + z * r.pitch + col) = make_uint4(0, 0, 0, 0);
    }
}

// Rows of bf16 to rows on 16-byte boundaries, `pitch` apart; a warp takes up to 512 columns
// of a row.  With an index: the live tokens' rows, and zeros up to whole tiles.
__global__ void __launch_bounds__(32 * kCopyWarps)
head_copy_kernel(const uint16_t* from, int64_t stride, const int32_t* index, const int32_t* counts,
                 int64_t rows, int32_t dim, int32_t sections, uint16_t* to, int64_t pitch) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kCopyWarps + threadIdx.x / 32;
    const int64_t row = id / sections;
    if (row >= rows) return;
    const int lane = threadIdx.x % 32;
    const int first = static_cast<int>(id - row * sections) * kCopyColumns + 8 * lane;
    let_next_launch_begin();
    wait_for_launch_before();
    const int64_t live = index == nullptr ? rows : *counts;
    uint16_t* out = to + row * pitch;
    if (row >= live) {
        if (row < (live + kPairTile - 1) / kPairTile * kPairTile) {
#pragma unroll
            for (int i = 0; i < kCopyColumns / 256; ++i)
                if (first + 256 * i < pitch)
                    *reinterpret_cast<uint4*>(out + first + 256 * i) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const uint16_t* in = from + (index == nullptr ? row : index[row]) * stride;
    copy_columns(in, out, first, dim);
}

// The tiles' maxima and sums of a row joined: a warp a row, in a fixed order.
__global__ void __launch_bounds__(256)
head_join_kernel(const HeadCall c, const int32_t* counts, const int32_t* index,
                 const float2* parts, int32_t n_parts, const float* picked) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    wait_for_launch_before();
    const bool as_they_are = counts == nullptr;
    if (row >= (as_they_are ? c.n_tokens : *counts)) return;
    // (read beside the parts; of a token that does not count nothing has been written)
    const bool live = !as_they_are || live_label(c, row, false) >= 0;
    const float of_label = picked[row];
    const float2* p = parts + row * n_parts;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
    for (int i = lane; i < n_parts; i += 32) {
        const float2 v = p[i];
        const float m = fmaxf(top, v.x), from = m == -INFINITY ? 0.0f : m;
        sum = sum * exp2f((top - from) * kLog2e) + v.y * exp2f((v.x - from) * kLog2e);
        top = m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float t = __shfl_xor_sync(0xFFFFFFFFu, top, o), s = __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float m = fmaxf(top, t), from = m == -INFINITY ? 0.0f : m;
        // (both lanes of a pair add the same two terms)
        const float x = sum * exp2f((top - from) * kLog2e), y = s * exp2f((t - from) * kLog2e);
        sum = x + y;
        top = m;
    }
    if (lane == 0) {
        // The loss is what the largest logit lies above the label's, and the logarithm of a
        // sum that holds the largest one's 1: two numbers that are not negative.
        const float l = logf(sum);
        const int64_t t = as_they_are ? row : index[row];
        c.loss[t] = live ? (top - of_label) + l : 0.0f;
        if (c.lse != nullptr) c.lse[t] = live ? top + l : 0.0f;
    }
}

// The hidden states' gradient: the splits' sums of live tokens, zeros of the others.  512
// columns of a row by a warp, or, where there are many splits, by the warps of a CTA, which
// share them (MANY).
constexpr int kFinishWarps = 8;

template <bool WIDE, bool MANY>
__global__ void __launch_bounds__(32 * kFinishWarps)
head_finish_kernel(const int32_t* counts, const int32_t* slot, const float* sums, int64_t rows,
                   int32_t splits,
                   int64_t n_tokens, int32_t dim, int32_t sections, uint16_t* out,
                   int64_t stride) {
    constexpr int N = kCopyColumns / 128;
    __shared__ float4 shared[MANY ? kFinishWarps : 1][N][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t id = MANY ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kFinishWarps + warp;
    const int64_t t = id / sections;
    if (t >= n_tokens) return;
    const int first = static_cast<int>(id - t * sections) * kCopyColumns + 4 * lane;
    wait_for_launch_before();
    const int32_t j = slot[t];
    const float by = scale_of(counts);
    const bool two = dz_in_two(*counts);
    uint16_t* to = out + t * stride;
    float4 v[N];
    auto add = [](float4& x, const float4& y) {
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    };
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (j >= 0) {
        // (see HeadArgs)
        const int blocks = (dim + 31) / 32;
        const float* from =
            sums + (first / 32 * rows + j) * 32 + 4 * (first % 32 / 4 ^ (j & 7));
#pragma unroll 4
        for (int s = MANY ? warp : 0; s < splits; s += MANY ? kFinishWarps : 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (first + 128 * i < dim) {
                    const float* p = from + (static_cast<int64_t>(s) * blocks + 4 * i) * rows * 32;
                    add(v[i], *reinterpret_cast<const float4*>(p));
                    if (two) add(v[i], *reinterpret_cast<const float4*>(p + kHalf * 32));
                }
            }
        }
    }
    if constexpr (MANY) {
#pragma unroll
        for (int i = 0; i < N; ++i) shared[warp][i][lane] = v[i];
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int w = 1; w < kFinishWarps; ++w) add(v[i], shared[w][i][lane]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = first + 128 * i;
        v[i] = make_float4(v[i].x * by, v[i].y * by, v[i].z * by, v[i].w * by);
        if (WIDE && c + 4 <= dim) {
            *reinterpret_cast<uint2*>(to + c) =
                make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
        } else {
            const float f[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < dim) to[c + e] = float_to_bf16_rn(f[e]);
        }
    }
}

// ---------------------------------------------------------------- host ------

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

cudaError_t find_encode(Encode* f) {
    static std::once_flag once;
    static Encode found = nullptr;
    static cudaError_t status;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult how;
        status = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                  cudaEnableDefault, &how);
        if (status == cudaSuccess && how != cudaDriverEntryPointSuccess)
            status = cudaErrorSymbolNotFound;
        found = reinterpret_cast<Encode>(p);
    });
    *f = found;
    return status;
}

// Rows of `inner` bf16 values, `pitch` apart, in boxes of 64 values by `box_rows`; what a
// box has beyond the matrix is read as zeros.
cudaError_t make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t rows,
                     int64_t pitch, int box_rows) {
    Encode encode = nullptr;
    if (cudaError_t e = find_encode(&encode); e != cudaSuccess) return e;
    const cuuint64_t sizes[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, ones[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
                              sizes, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A launch that may be set up while the one before it in the stream ends; the kernel waits
// for that one's results itself.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int threads, size_t smem,
                         cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <class T>
T* at(const HeadCall& c, int64_t offset) {
    return reinterpret_cast<T*>(static_cast<char*>(c.workspace) + offset);
}

// Forward, one tile of tokens that TMA reaches: nothing is saved by leaving tokens out, and
// what they hold stays in their rows (32 x 50257 x 768: 41 us with a launch for the rows).
bool rows_as_they_are(const HeadCall& c) {
    return c.loss != nullptr && c.n_tokens <= kPairTile && aligned_to(c.hidden, 16) &&
           c.hidden_stride % 8 == 0 && c.hidden_stride < int64_t{1} << 32;
}
bool rows_in_one_launch(const HeadCall& c) {
    return c.n_tokens > 0 && c.n_tokens <= kFewTokens && !rows_as_they_are(c);
}

bool table_in_place(const HeadCall& c) { return head_table_in_place(c); }

int64_t piece_rows(const HeadCall& c, const HeadPlan& p, int64_t first) {
    return p.piece < c.vocab - first ? p.piece : c.vocab - first;
}

// The piece's rows of the table: in place, or copied to where TMA reaches them.
cudaError_t piece_map(CUtensorMap* map, const HeadCall& c, const HeadPlan& p, int64_t first,
                      int box_rows) {
    const int64_t rows = piece_rows(c, p, first);
    return table_in_place(c)
               ? make_map(map, c.table + first * c.dim, c.dim, rows, c.dim, box_rows)
               : make_map(map, at<uint16_t>(c, p.table), c.dim, rows, p.pitch, box_rows);
}

cudaError_t copy_rows(const uint16_t* from, int64_t stride, const int32_t* index,
                      const int32_t* counts, int64_t rows, int64_t dim, uint16_t* to,
                      int64_t pitch, cudaStream_t stream) {
    const int64_t sections = (pitch + kCopyColumns - 1) / kCopyColumns;
    const unsigned grid = static_cast<unsigned>((rows * sections + kCopyWarps - 1) / kCopyWarps);
    return launch_after(head_copy_kernel, grid, 32 * kCopyWarps, 0, stream, from, stride, index,
                        counts, rows, dim, sections, to, pitch);
}

// (The first piece's copy goes with the tokens' rows where those take one launch.)
cudaError_t copy_piece(const HeadCall& c, const HeadPlan& p, int64_t first, cudaStream_t stream) {
    if (table_in_place(c) || (first == 0 && rows_in_one_launch(c))) return cudaSuccess;
    const int64_t rows = piece_rows(c, p, first);
    const uint16_t* from = c.table + first * c.dim;
    return copy_rows(from, c.dim, nullptr, nullptr, rows, c.dim, at<uint16_t>(c, p.table), p.pitch,
                     stream);
}

// The piece's gradient of the logits, in boxes of 64 columns by `box_rows` (it is stored as
// swizzled as it has to be in shared memory).
cudaError_t dz_map(CUtensorMap* map, const HeadArgs& a, int box_rows) {
    Encode encode = nullptr;
    if (cudaError_t e = find_encode(&encode); e != cudaSuccess) return e;
    const cuuint64_t sizes[3] = {64, static_cast<cuuint64_t>(a.rows),
                                 static_cast<cuuint64_t>(a.blocks)};
    const cuuint64_t strides[2] = {128, static_cast<cuuint64_t>(a.rows) * 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, ones[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.dz, sizes, strides, box,
                              ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE>
cudaError_t launch_product(const HeadMaps& maps, HeadArgs a, int64_t tiles, cudaStream_t stream) {
    if (cudaError_t e = device_status_word(&a.status); e != cudaSuccess) return e;
    static std::once_flag once[64];
    static cudaError_t set[64];
    static int fit[64];                                  // pairs at a time
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        const auto kernel = head_kernel<MODE>;
        set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kHeadSmem));
        if (set[dev] != cudaSuccess) return;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kHeadThreads);
        cfg.dynamicSmemBytes = kHeadSmem;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        set[dev] = cudaOccupancyMaxActiveClusters(&fit[dev], kernel, &cfg);
        if (set[dev] == cudaSuccess && fit[dev] < 1) set[dev] = cudaErrorInvalidConfiguration;
    });
    if (set[dev] != cudaSuccess) return set[dev];
    const int64_t pairs = tiles < fit[dev] ? tiles : fit[dev];
    return launch_after(head_kernel<MODE>, static_cast<unsigned>(2 * pairs), kHeadThreads, kHeadSmem,
                        stream, maps, a);
}

HeadArgs product_args(const HeadCall& c, const HeadPlan& p, int64_t first) {
    HeadArgs a{};
    a.counts = at<int32_t>(c, p.counts);
    a.label = at<int32_t>(c, p.label);
    a.lse = at<float>(c, p.lse);
    a.grad = at<float>(c, p.grad);
    a.parts = at<float2>(c, p.parts);
    a.picked = at<float>(c, p.picked);
    a.dz = at<uint16_t>(c, p.dz);
    a.sums = at<float>(c, p.sums);
    a.grad_table = c.grad_table == nullptr ? nullptr : c.grad_table + first * c.dim;
    a.parts_pitch = p.parts_a_row;
    a.rows = p.rows;
    a.first = static_cast<int32_t>(first);
    a.vocab = static_cast<int32_t>(piece_rows(c, p, first));
    a.dim = static_cast<int32_t>(c.dim);
    a.splits = p.splits;
    a.blocks = (a.vocab + 63) / 64;
    a.group = 8;
    return a;
}

int64_t whole(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
int64_t tiles_of(int64_t x, int64_t width) { return (x + width - 1) / width; }

// Clock cycles of a tile of `steps` steps and `width` columns: the steps (256 + width, what
// the operands take on their way), the result's way out and what comes before; and of a
// launch of m rows of tiles, n columns, in rounds over the GPU's pairs.  Measured: 12 steps of
// width 256 7500 to 8400 cycles, 64 steps 36000 to 40000.
double tile_cost(double steps, int width) { return (256.0 + width) * steps + 12.0 * width + 800.0; }
int64_t pairs_of(int sms) { return sms / 2 > 0 ? sms / 2 : 1; }
double launch_cost(int64_t m, int64_t n, int64_t steps, int width, int64_t pairs) {
    const int64_t rounds = (m * tiles_of(n, width) + pairs - 1) / pairs;
    return static_cast<double>(rounds) * tile_cost(static_cast<double>(steps), width);
}

int best_width(int64_t m, int64_t n, int64_t steps, int unit, int64_t pairs) {
    int best = kPairTile;
    double least = launch_cost(m, n, steps, best, pairs);
    for (int w = kPairTile - unit; w >= unit; w -= unit) {
        const double cost = launch_cost(m, n, steps, w, pairs);
        if (cost < 0.98 * least) {
            best = w;
            least = cost;
        }
    }
    return best;
}

}  // namespace

// Pieces of the vocabulary whose gradient, and whose copy of the table where that is off the
// 16-byte grid, take at most 512 MB each (but 256 rows at least, whose gradient takes more
// beyond 1M tokens); as even as whole tiles allow.  Forward, a table that is read in place is
// one piece.
static HeadPlan plan_on(int sms, int64_t n_tokens, int64_t vocab, int64_t dim, bool back, bool in_place) {
    constexpr int64_t kMost = int64_t{512} << 20;
    const int64_t pairs = pairs_of(sms);
    HeadPlan p{};
    p.rows = whole(n_tokens < 1 ? 1 : n_tokens, kPairTile);
    p.pitch = whole(dim, 64);                // rows on 128-byte boundaries: fewer lines a box
    const int64_t copied = in_place ? 0 : p.pitch;
    const int64_t per_row = 2 * (back && p.rows > copied ? p.rows : p.pitch);
    const int64_t m = p.rows / kPairTile;
    int64_t most = kMost / per_row / kPairTile * kPairTile;
    if (most < kPairTile) most = kPairTile;
    if (!back && in_place) most = whole(vocab, kPairTile);
    const int64_t pieces = (vocab + most - 1) / most;
    p.piece = whole((vocab + pieces - 1) / pieces, kPairTile);
    p.splits = 1;
    const int64_t steps_dim = tiles_of(dim, kTileK);
    if (back) {
        p.width_z = best_width(m, p.piece < vocab ? p.piece : vocab, steps_dim, 64, pairs);
        const int64_t steps = tiles_of(p.piece, kTileK), steps_w = tiles_of(n_tokens, kTileK);
        p.width_w = best_width(tiles_of(p.piece, kPairTile), dim, steps_w, 32, pairs);
        // The sum over a piece in as many parts as keep the GPU's pairs busy: the launch takes
        // the tiles' average on a pair, half a tile more at its end, and every part is written,
        // and read again in the end, at 6 TB/s and 1.9 GHz.
        const double tile_w = tile_cost(steps_w, p.width_w);
        const double all_w =
            tile_w * tiles_of(p.piece, kPairTile) * tiles_of(dim, p.width_w) / pairs;
        const double way = 8.0 * p.rows * whole(dim, 32) / 6e12 * 1.9e9;
        double wide[kPairTile / 32 + 1];             // tiles of width 32 i
        for (int i = 1; i <= kPairTile / 32; ++i)
            wide[i] = static_cast<double>(m * tiles_of(dim, 32 * i));
        double best = 0.0;
        for (int64_t s : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 40, 48, 64}) {
            if (s > 1 && (s * 4 > steps || s * p.rows * p.pitch * 4 > kMost)) break;
            for (int w = kPairTile; w >= 32; w -= 32) {
                const double tile = tile_cost(steps / static_cast<double>(s), w);
                const double cost =
                    tile * wide[w / 32] * s / pairs + all_w +
                    0.5 * (tile > tile_w ? tile : tile_w) + way * s;
                if ((s == 1 && w == kPairTile) || cost < 0.98 * best) {
                    best = cost;
                    p.splits = static_cast<int32_t>(s);
                    p.width_h = w;
                }
            }
        }
    } else {
        p.width_z = best_width(m, p.piece < vocab ? p.piece : vocab, steps_dim, 32, pairs);
        p.parts_a_piece = static_cast<int32_t>(tiles_of(p.piece, p.width_z));
        p.parts_a_row = static_cast<int32_t>((pieces - 1) * p.parts_a_piece +
                                             tiles_of(vocab - (pieces - 1) * p.piece, p.width_z));
    }
    int64_t end = 0;
    auto place = [&](int64_t bytes) {
        const int64_t here = end;
        end += whole(bytes, 1024);
        return here;
    };
    const int64_t n = n_tokens < 1 ? 1 : n_tokens;
    p.counts = place(8);
    p.index = place(4 * n);
    p.slot = place(4 * n);
    p.label = place(4 * n);
    p.hidden = place(2 * p.rows * p.pitch);
    p.table = place(2 * p.piece * copied);
    if (back) {
        p.lse = place(4 * n);
        p.grad = place(4 * n);
        p.dz = place(2 * p.rows * whole(p.piece < vocab ? p.piece : vocab, 64));
        p.sums = place(4 * p.splits * p.rows * whole(dim, 32));
    } else {
        // (of few tokens one part a CTA, perhaps)
        const int64_t few = n <= kFewMost ? sms : 0;
        p.parts = place(8 * n * (p.parts_a_row > few ? p.parts_a_row : few));
        p.picked = place(4 * n);
    }
    p.bytes = end;
    return p;
}

HeadPlan head_plan(int64_t n_tokens, int64_t vocab, int64_t dim, bool back, bool in_place) {
    return plan_on(device_sms(), n_tokens, vocab, dim, back, in_place);
}

// A smaller call's pieces may be larger and its splits more, and with them its needs.  A plan
// goes by whole tiles and, for the table's gradient, steps of tokens, and grows within them.
int64_t head_bytes(int64_t n_tokens, int64_t vocab, int64_t dim, bool back, bool in_place) {
    const int sms = device_sms();
    int64_t most = plan_on(sms, n_tokens, vocab, dim, back, in_place).bytes;
    for (int64_t n = kTileK; n < n_tokens; n += kTileK) {
        const int64_t bytes = plan_on(sms, n, vocab, dim, back, in_place).bytes;
        if (bytes > most) most = bytes;
    }
    return most;
}

bool head_table_in_place(const HeadCall& c) { return aligned_to(c.table, 16) && c.dim % 8 == 0; }

bool head_rows_as_they_are(const HeadCall& c) { return rows_as_they_are(c); }

cudaError_t launch_head_rows(const HeadCall& c, const HeadPlan& p, bool back, cudaStream_t stream) {
    const HeadRows r{at<int32_t>(c, p.counts), at<int32_t>(c, p.index),  at<int32_t>(c, p.slot),
                     at<int32_t>(c, p.label),  at<float>(c, p.lse),      at<float>(c, p.grad),
                     at<uint16_t>(c, p.hidden), p.pitch};
    if (rows_in_one_launch(c)) {
        const unsigned own =
            static_cast<unsigned>((c.n_tokens + kPrepareTokens - 1) / kPrepareTokens);
        HeadCopy copy{};
        if (!table_in_place(c)) {
            copy.from = c.table;
            copy.to = at<uint16_t>(c, p.table);
            copy.count = piece_rows(c, p, 0);
            copy.pitch = p.pitch;
            copy.dim = static_cast<int32_t>(c.dim);
            copy.sections = static_cast<int32_t>((c.dim + kCopyColumns - 1) / kCopyColumns);
        }
        const unsigned grid =
            own + static_cast<unsigned>((copy.count * copy.sections + kPrepareTokens - 1) / kPrepareTokens);
        head_prepare_kernel<<<grid, kPrepareThreads, 0, stream>>>(c, r, copy, own, back);
        return cudaGetLastError();
    }
    head_rows_kernel<<<1, kRowThreads, 0, stream>>>(c, r, back);
    return cudaGetLastError();
}

cudaError_t launch_head_gather(const HeadCall& c, const HeadPlan& p, cudaStream_t stream) {
    if (c.n_tokens <= kFewTokens) return cudaSuccess;     // done with the rows
    return copy_rows(c.hidden, c.hidden_stride, at<int32_t>(c, p.index), at<int32_t>(c, p.counts),
                     p.rows, c.dim, at<uint16_t>(c, p.hidden), p.pitch, stream);
}

// Few tokens that TMA reaches, as it does the table; more than 32 from 80 rows of the table an
// SM on (64 tokens, us with head_few_kernel and with head_kernel: 5000 x 256 8.4 and 7.5,
// 9728 x 256 8.4 and 8.0, 14000 x 256 8.8 and 9.0, 14000 x 2048 18.6 and 19.7; 32 tokens 6.4
// and 7.4, 6.5 and 7.9, 6.7 and 8.8, 16.5 and 19.4).
int64_t few_units(const HeadCall& c) { return (c.vocab + kFewUnit - 1) / kFewUnit; }
int few_ctas(const HeadCall& c) {
    const int64_t units = few_units(c), sms = device_sms();
    return static_cast<int>(units < sms ? units : sms);
}
bool few_tokens(const HeadCall& c) {
    return rows_as_they_are(c) && table_in_place(c) &&
           (c.n_tokens <= 32 || (c.n_tokens <= kFewMost && few_units(c) >= 5 * device_sms()));
}

template <int TOKENS>
cudaError_t launch_few(const HeadCall& c, const HeadPlan& p, cudaStream_t stream) {
    static std::once_flag once[64];
    static cudaError_t set[64];
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        set[dev] = cudaFuncSetAttribute(head_few_kernel<TOKENS>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(few_smem(TOKENS)));
    });
    if (set[dev] != cudaSuccess) return set[dev];
    FewMaps maps;
    if (cudaError_t e = make_map(&maps.tile, c.table, c.dim, c.vocab, c.dim, kHalf);
        e != cudaSuccess)
        return e;
    const int64_t share = few_units(c) / few_ctas(c);
    for (int more = 0; more < 2; ++more) {
        const int rest = static_cast<int>((share + more) % (kHalf / kFewUnit));
        if (cudaError_t e = make_map(&maps.rest[more], c.table, c.dim, c.vocab, c.dim,
                                     (rest ? rest : 1) * kFewUnit);
            e != cudaSuccess)
            return e;
    }
    if (cudaError_t e = make_map(&maps.tokens, c.hidden, c.dim, c.n_tokens, c.hidden_stride, TOKENS);
        e != cudaSuccess)
        return e;
    FewArgs a{};
    if (cudaError_t e = device_status_word(&a.status); e != cudaSuccess) return e;
    a.labels = c.labels;
    a.parts = at<float2>(c, p.parts);
    a.picked = at<float>(c, p.picked);
    a.n_rows = static_cast<int32_t>(c.n_tokens);
    a.vocab = static_cast<int32_t>(c.vocab);
    a.dim = static_cast<int32_t>(c.dim);
    a.label64 = c.label64;
    return launch_after(head_few_kernel<TOKENS>, static_cast<unsigned>(few_ctas(c)),
                        few_threads(TOKENS),
                        few_smem(TOKENS), stream, maps, a);
}

cudaError_t launch_head_loss(const HeadCall& c, const HeadPlan& p, int64_t first,
                             cudaStream_t stream) {
    if (few_tokens(c))
        return c.n_tokens <= 32 ? launch_few<32>(c, p, stream) : launch_few<kFewMost>(c, p, stream);
    if (cudaError_t e = copy_piece(c, p, first, stream); e != cudaSuccess) return e;
    const bool as_they_are = head_rows_as_they_are(c);
    HeadMaps maps{};
    if (cudaError_t e = as_they_are ? make_map(&maps.a, c.hidden, c.dim, c.n_tokens, c.hidden_stride, kHalf)
                                    : make_map(&maps.a, at<uint16_t>(c, p.hidden), c.dim, p.rows, p.pitch,
                                               kHalf);
        e != cudaSuccess)
        return e;
    if (cudaError_t e = piece_map(&maps.b, c, p, first, p.width_z / 2); e != cudaSuccess) return e;
    HeadArgs a = product_args(c, p, first);
    a.width = p.width_z;
    a.part = static_cast<int32_t>(first / p.piece * p.parts_a_piece);
    if (as_they_are) {
        a.counts = a.label = nullptr;
        a.labels = c.labels;
        a.label64 = c.label64;
        a.n_rows = static_cast<int32_t>(c.n_tokens);
    }
    const int64_t tiles = p.rows / kPairTile * tiles_of(a.vocab, a.width);
    return c.dim <= kLogitSteps * kTileK ? launch_product<kLoss>(maps, a, tiles, stream)
                                         : launch_product<kLossLong>(maps, a, tiles, stream);
}

cudaError_t launch_head_join(const HeadCall& c, const HeadPlan& p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((c.n_tokens + 7) / 8);
    const bool as_they_are = head_rows_as_they_are(c);
    return launch_after(head_join_kernel, grid, 256, 0, stream, c,
                        as_they_are ? nullptr : at<int32_t>(c, p.counts), at<int32_t>(c, p.index),
                        at<float2>(c, p.parts), few_tokens(c) ? few_ctas(c) : p.parts_a_row,
                        at<float>(c, p.picked));
}

cudaError_t launch_head_dz(const HeadCall& c, const HeadPlan& p, int64_t first,
                           cudaStream_t stream) {
    if (cudaError_t e = copy_piece(c, p, first, stream); e != cudaSuccess) return e;
    HeadMaps maps{};
    if (cudaError_t e = make_map(&maps.a, at<uint16_t>(c, p.hidden), c.dim, p.rows, p.pitch, kHalf);
        e != cudaSuccess)
        return e;
    if (cudaError_t e = piece_map(&maps.b, c, p, first, p.width_z / 2); e != cudaSuccess) return e;
    HeadArgs a = product_args(c, p, first);
    a.width = p.width_z;
    const int64_t tiles = p.rows / kPairTile * tiles_of(a.vocab, a.width);
    return c.dim <= kLogitSteps * kTileK ? launch_product<kDz>(maps, a, tiles, stream)
                                         : launch_product<kDzLong>(maps, a, tiles, stream);
}

cudaError_t launch_head_products(const HeadCall& c, const HeadPlan& p, int64_t first,
                                 cudaStream_t stream) {
    HeadArgs a = product_args(c, p, first);
    a.want_h = c.grad_hidden != nullptr && c.n_tokens > 0;
    a.want_w = c.grad_table != nullptr;
    a.add_h = first > 0;
    a.add_w = c.accumulate;
    a.width_h = p.width_h;
    a.width_w = p.width_w;
    a.wide = aligned_to(c.grad_table, 16) && c.dim % 8 == 0;
    HeadMaps maps{};
    if (cudaError_t e = dz_map(&maps.a, a, kHalf); e != cudaSuccess) return e;
    if (cudaError_t e = piece_map(&maps.b, c, p, first, kTileK); e != cudaSuccess) return e;
    if (cudaError_t e = dz_map(&maps.aw, a, kTileK); e != cudaSuccess) return e;
    if (cudaError_t e = make_map(&maps.bw, at<uint16_t>(c, p.hidden), c.dim, p.rows, p.pitch, kTileK);
        e != cudaSuccess)
        return e;
    const int64_t tiles =
        (a.want_h ? p.rows / kPairTile * tiles_of(c.dim, a.width_h) * p.splits : 0) +
        (a.want_w ? tiles_of(a.vocab, kPairTile) * tiles_of(c.dim, a.width_w) : 0);
    const int64_t steps_h = tiles_of(tiles_of(p.piece, kTileK), p.splits);
    return steps_h <= kSumSteps && tiles_of(c.n_tokens, kTileK) <= kSumSteps
               ? launch_product<kProducts>(maps, a, tiles, stream)
               : launch_product<kProductsLong>(maps, a, tiles, stream);
}

cudaError_t launch_head_finish(const HeadCall& c, const HeadPlan& p, cudaStream_t stream) {
    const int64_t sections = (c.dim + kCopyColumns - 1) / kCopyColumns;
    const bool wide = aligned_to(c.grad_hidden, 8) && c.grad_hidden_stride % 4 == 0;
    const bool many = p.splits > 4;
    const int64_t units = c.n_tokens * sections;
    const unsigned grid =
        static_cast<unsigned>(many ? units : (units + kFinishWarps - 1) / kFinishWarps);
    const auto kernel = many ? (wide ? head_finish_kernel<true, true> : head_finish_kernel<false, true>)
                             : (wide ? head_finish_kernel<true, false> : head_finish_kernel<false, false>);
    return launch_after(kernel, grid, 32 * kFinishWarps, 0, stream, at<int32_t>(c, p.counts),
                        at<int32_t>(c, p.slot), at<float>(c, p.sums), p.rows, p.splits,
                        c.n_tokens, c.dim, sections, c.grad_hidden, c.grad_hidden_stride);
}

cudaError_t launch_tile_wait_selftest(uint64_t limit_ns, cudaStream_t stream) {
    int* status = nullptr;
    if (cudaError_t e = device_status_word(&status); e != cudaSuccess) return e;
    wait_selftest_kernel<<<1, 64, 0, stream>>>(status, limit_ns);
    return cudaGetLastError();
}

}  // namespace zf
