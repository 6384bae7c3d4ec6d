// Softmax cross entropy of the head in pieces of the vocabulary (zero_head.cu): the plan
// of a call and its launches.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace zf {

// What a call works with.  Only live tokens take part: those with a label in [0, vocab)
// and, in the backward pass, a gradient other than zero.
struct HeadCall {
    const uint16_t* hidden;       // rows of hidden_stride
    const uint16_t* table;        // [vocab][dim]
    const void* labels;           // int32 or int64
    float* loss;                  // forward
    float* lse;                   // forward written (may be null), backward read
    const float* grad_loss;       // backward
    uint16_t* grad_hidden;        // backward; may be null
    uint16_t* grad_table;         // backward; may be null
    int64_t n_tokens;
    int64_t vocab;
    int64_t dim;
    int64_t hidden_stride;
    int64_t grad_hidden_stride;
    int32_t label64;
    int32_t accumulate;
    void* workspace;
};

// Places in the workspace, in bytes from its start.
struct HeadPlan {
    int64_t rows;                 // n_tokens rounded up to whole tiles
    int64_t pitch;                // elements of a row of the hidden states' copy
    int64_t piece;                // rows of the table worked on at a time
    int32_t width_z, width_h, width_w;    // columns of a tile of each product
    int32_t parts_a_piece;        // maxima and sums of a row, forward
    int32_t parts_a_row;
    int32_t splits;               // of the sum over the vocabulary in the hidden gradient
    int64_t counts, index, slot, label, lse, grad, hidden, table, parts, picked, dz, sums;
    int64_t bytes;
};
HeadPlan head_plan(int64_t n_tokens, int64_t vocab, int64_t dim, bool back, bool in_place);
// What calls of up to n_tokens tokens need for a table that is read in place, or for one that
// is not.
int64_t head_bytes(int64_t n_tokens, int64_t vocab, int64_t dim, bool back, bool in_place);

// Whether TMA reaches the table where it is.
bool head_table_in_place(const HeadCall& c);

// Whether the forward pass takes all tokens as they lie, without the first two launches.
bool head_rows_as_they_are(const HeadCall& c);

// The launches of a call, in order.
cudaError_t launch_head_rows(const HeadCall& c, const HeadPlan& p, bool back, cudaStream_t stream);
cudaError_t launch_head_gather(const HeadCall& c, const HeadPlan& p, cudaStream_t stream);
// forward: a piece of the vocabulary, then the rows' join
cudaError_t launch_head_loss(const HeadCall& c, const HeadPlan& p, int64_t first,
                             cudaStream_t stream);
cudaError_t launch_head_join(const HeadCall& c, const HeadPlan& p, cudaStream_t stream);
// backward: a piece's gradient of the logits, its share of the hidden states' gradient with
// the piece of the table's gradient; then the hidden states' gradient
cudaError_t launch_head_dz(const HeadCall& c, const HeadPlan& p, int64_t first,
                           cudaStream_t stream);
cudaError_t launch_head_products(const HeadCall& c, const HeadPlan& p, int64_t first,
                                 cudaStream_t stream);
cudaError_t launch_head_finish(const HeadCall& c, const HeadPlan& p, cudaStream_t stream);

// One CTA whose wait, the one that these kernels and the norm's use, runs out.
cudaError_t launch_tile_wait_selftest(uint64_t limit_ns, cudaStream_t stream);

}  // namespace zf
