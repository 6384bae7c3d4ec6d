// Launch plans that are plain arithmetic, without CUDA.
#pragma once

#include <cstdint>

namespace zf {

constexpr int kSortCtas = 8;        // of the cluster that sorts a table gradient's tokens
constexpr int kSortWarps = 32;      // of each of them

// Clusters of the sort launch: the one that sorts, and, where every row of the
// table is written, those that write the zeros meanwhile: a warp a row at most,
// two CTAs an SM, at least one.
inline int sort_clusters(int64_t vocab, bool accumulate, int sms) {
    if (accumulate) return 1;
    const int64_t rows = (vocab + kSortWarps - 1) / kSortWarps;
    const int64_t need = (rows + kSortCtas - 1) / kSortCtas;
    const int64_t most = 2 * sms / kSortCtas - 1 > 1 ? 2 * sms / kSortCtas - 1 : 1;
    return 1 + static_cast<int>(need < most ? need : most);
}

}  // namespace zf
