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

}  // namespace zero
