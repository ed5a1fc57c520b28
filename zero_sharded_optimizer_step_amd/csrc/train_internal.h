// train_internal.h -- declarations shared by the sources of
// libzero_train_mi355x.so.  Not part of the public ABI.
#pragma once

#include "zero/train.h"
#include "zero_internal.h"

namespace zero {

// One tensor of a list as the kernels read it (64 bytes, scalar loads).
struct TensorRec {
    const void* grad;
    float* master;
    void* m;                  // exp_avg, or state8
    void* v;                  // exp_avg_sq, or scale8
    void* param;
    int64_t numel;
    int64_t first_chunk;
    uint32_t first_block;     // ordinal in the list of its first block of 256 (mod 2^32)
    int32_t group;
};
static_assert(sizeof(TensorRec) == 64, "one tensor is one line of the table");

// Work is dealt in chunks of one tensor: 1024 elements, one quad for each of
// 256 threads, so a wave holds exactly one block of an 8-bit state.  The
// table is the records, then for every chunk the index of its tensor.
constexpr int kChunk = 1024;
constexpr int kChunkThreads = kChunk / kQuad;
static_assert(kChunkThreads / 64 * ZERO_STATE8_BLOCK == kChunk, "one wave, one block");
constexpr size_t table_map_offset(int32_t n_tensors) {
    return sizeof(TensorRec) * static_cast<size_t>(n_tensors);
}

// Workspace of a list: one partials slot and one zero_global_t.
constexpr size_t kTensorsWorkspace = round_up(kSlotBytes, 256) + 256;

// Checks *a (see zero_tensors_step) and fills the launch constants; without
// `peers` the peers' fields are not looked at, without `buffers` the
// workspace and result are not.
int tensors_constants(const zero_tensors_args* a, bool peers, bool buffers, zero_tensors_scalars_t* k);

int check_xent_args(const zero_xent_args* a, bool backward);
// Bytes of workspace that calls of these sizes use; 0 for out-of-range ones.
size_t xent_needs(int64_t tokens, int64_t dim, int64_t vocab);

// x is what is encoded, or what codes are decoded into.
int check_rows8(const void* x, int64_t x_stride, int32_t dtype, int64_t rows, int64_t dim, const void* codes,
                int64_t codes_stride, const float* scale);
int check_glu8_args(const zero_glu8_args* a, bool backward);
int check_linear8_args(const zero_linear8_args* a, bool backward);
// Bytes of workspace that this call uses; 0 for out-of-range sizes.
size_t linear8_needs(const zero_linear8_args* a, bool backward);

// How `most` blocks are shared by two lists of tiles, one a block where there
// are no more than that, else by their work (of a tile: work_a and work_b).
inline void share_blocks(int64_t a, int64_t b, double work_a, double work_b, int64_t most, int64_t* first,
                         int64_t* second) {
    *first = a;
    *second = b;
    if (a + b <= most) return;
    const double wa = static_cast<double>(a) * work_a, wb = static_cast<double>(b) * work_b;
    *first = a == 0 ? 0 : (b == 0 ? most : static_cast<int64_t>(static_cast<double>(most) * (wa / (wa + wb)) + 0.5));
    if (a > 0 && *first < 1) *first = 1;
    if (b > 0 && *first > most - 1) *first = most - 1;
    // what one has no tile for is the other's (gradient of 128 tokens x 512 x 16384 27.9 us, left idle 30.2)
    if (*first > a) *first = a;
    *second = most - *first < b ? most - *first : b;
    *first = most - *second < a ? most - *second : a;
}

}  // namespace zero
