// train_xent.hip -- softmax cross entropy of a large vocabulary and its
// gradient (include/zero/train.h), without keeping the logits.
//
//   forward    L = w x^T tile by tile on the matrix cores; each tile leaves,
//              per token and wave row, its largest logit and the sum of
//              exponentials below it (one pass of a running softmax), and
//              the target's logit; a second kernel joins them into lse and
//              loss, a third sums the losses.  Up to 8 tokens: w is read
//              straight into registers, and one kernel joins it all.
//   backward   the tokens that have a target are gathered; then piece by
//              piece of the vocabulary: L again, P = exp(L - lse) - onehot
//              rounded to 16 bits into the workspace, then dx += P w (fp32
//              in the workspace) and dw = P^T x.
//
// One tile product serves all of it.  An operand lies with its rows along k
// (x and w in the logits, P in dx) or with k as the row (w in dx; x and P in
// dw); the second kind is turned on the way from LDS to the registers, so
// nothing is ever transposed in memory.
#include "train_product.h"

namespace zero {
namespace {

// kLse of up to 8 tokens: w is read once and nothing else counts, so the
// fragments go from memory to registers, many loads at a time.  A block takes
// 16 rows of w; its four waves take every fourth 64 of k, and the sums meet
// in LDS in a fixed order.  Whole forward at dim 4096 in bf16, w from memory,
// and that of the 128 x 128 tiles: 1 token x 32000 51.8 us (5.1 TB/s) and 67.9,
// 1 x 128000 176 us (6.0 TB/s) and 204, 4 x 32000 54.7 and 68.7, 8 62.3 and
// 67.7, 12 69.7 and 69.4, but 16 85.9 and 71.0, since every block reads x again.
template <int DT>
__global__ __launch_bounds__(256) void few_kernel(const Product q) {
    constexpr int kGroup = 2;                              // of 64 k a wave and turn
    __shared__ f32x4 s_sum[4][64];
    const int lane = threadIdx.x & 63, s = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int m0 = blockIdx.x * 16;
    auto records = [](int64_t bytes) { return static_cast<int>(bytes < 0x7ffffff0 ? bytes : 0x7ffffff0); };
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(q.a + m0 * q.lda), 0, records((q.m - m0) * q.lda), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(q.b), 0,
                                                                        records(q.n * q.ldb), 0x00020000);
    const uint32_t oa = static_cast<uint32_t>(s * q.lda), ob = static_cast<uint32_t>(s * q.ldb);
    struct Pieces {
        u32x4 a[kGroup][2], b[kGroup][2];
    };
    // k of this lane's piece p of block `block` of 64: both operands agree on it
    auto load = [&](Pieces& f, int block) __attribute__((always_inline)) -> void {
        #pragma unroll
        for (int u = 0; u < kGroup; ++u)
            #pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int k = (block + 4 * u) * 64 + g * 16 + p * 8;
                f.a[u][p] = __builtin_amdgcn_raw_buffer_load_b128(ra, k < q.k ? oa + k * 2 : kNowhere, 0, 0);
                f.b[u][p] = __builtin_amdgcn_raw_buffer_load_b128(rb, k < q.k ? ob + k * 2 : kNowhere, 0, 0);
            }
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Pieces& f) __attribute__((always_inline)) -> void {
        #pragma unroll
        for (int u = 0; u < kGroup; ++u)
            #pragma unroll
            for (int p = 0; p < 2; ++p) {
                if constexpr (DT == ZERO_BF16)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.a[u][p]),
                                                                  __builtin_bit_cast(bf16x8, f.b[u][p]), acc, 0, 0, 0);
                else
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, f.a[u][p]),
                                                                 __builtin_bit_cast(f16x8, f.b[u][p]), acc, 0, 0, 0);
            }
    };
    const int blocks = (q.k + 63) / 64;
    Pieces f0, f1;
    load(f0, wave);
    for (int b = wave; b < blocks; b += 8 * kGroup) {
        load(f1, b + 4 * kGroup);
        multiply(f0);
        load(f0, b + 8 * kGroup);
        multiply(f1);
    }
    s_sum[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    const f32x4 c1 = s_sum[1][lane], c2 = s_sum[2][lane], c3 = s_sum[3][lane];
    float x[4], top = -__builtin_inff(), sum = 0.0f;
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = (acc[e] + c1[e]) + (c2[e] + c3[e]);
        if (m0 + g * 4 + e >= q.m) x[e] = -__builtin_inff();
        top = fmaxf(top, x[e]);
    }
    top = fmaxf(other_row(top).x, other_row(top).y);
    top = fmaxf(other_half(top).x, other_half(top).y);
    const float base = infinite(top) ? 0.0f : top;
    #pragma unroll
    for (int e = 0; e < 4; ++e) sum += __expf(x[e] - base);
    sum = other_row(sum).x + other_row(sum).y;
    sum = other_half(sum).x + other_half(sum).y;
    if (s >= q.n) return;
    if (g == 0)
        reinterpret_cast<f32x2*>(q.partial)[static_cast<int64_t>(q.slot0 + blockIdx.x) * q.n + s] = f32x2{top, sum};
    const int64_t at = q.target[s] - q.first_m - m0 - g * 4;
    #pragma unroll
    for (int e = 0; e < 4; ++e)
        if (at == e && m0 + g * 4 + e < q.m) q.target_logit[s] = x[e];
}

// ------------------------------------------------------- joining the partials
__device__ __forceinline__ void write_mean(double sum, int64_t count, int beyond, zero_xent_result_t* out) {
    const double n = count > 1 ? static_cast<double>(count) : 1.0;
    out->loss_sum = sum;
    out->count = count;
    out->out_of_range = beyond;
    out->reserved = 0;
    out->mean = static_cast<float>(sum / n);
    out->inv_count = static_cast<float>(1.0 / n);
}

// A maximum and the sum of exponentials below it, with another such pair.
__device__ __forceinline__ void join(float& t, float& s, float t2, float s2) {
    const float m = fmaxf(t, t2);
    // equal maxima (also two infinite ones) keep their sums as they are
    s = s * (t == m ? 1.0f : __expf(t - m)) + s2 * (t2 == m ? 1.0f : __expf(t2 - m));
    t = m;
}

// 16 tokens by 64 slices of the slots in a block; every order is fixed.
__global__ __launch_bounds__(1024) void xent_rows_kernel(const f32x2* __restrict__ partial, int slots, int tokens,
                                                         const float* __restrict__ target_logit,
                                                         const int64_t* __restrict__ target, int64_t vocab,
                                                         float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ float s_top[64][17], s_sum[64][17];
    const int col = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int n = blockIdx.x * 16 + col;
    float top = -__builtin_inff(), sum = 0.0f;
    if (n < tokens)
        for (int s = slice; s < slots; s += 64) {
            const f32x2 p = partial[static_cast<int64_t>(s) * tokens + n];
            join(top, sum, p.x, p.y);
        }
    s_top[slice][col] = top;
    s_sum[slice][col] = sum;
    __syncthreads();
    for (int half = 32; half > 0; half >>= 1) {
        if (slice < half) {
            join(s_top[slice][col], s_sum[slice][col], s_top[slice + half][col], s_sum[slice + half][col]);
        }
        __syncthreads();
    }
    if (slice == 0 && n < tokens) {
        const float l = s_top[0][col] + logf(s_sum[0][col]);
        const int64_t t = target[n];
        lse[n] = l;
        loss[n] = t >= 0 && t < vocab ? l - target_logit[n] : 0.0f;
    }
}

// Up to kFewTokens tokens (it has room for 16): one block joins the slots of
// all of them and the mean in 4.1 us, where the two kernels above and below
// take 4.7 and 3.9 and the gap between them.
__global__ __launch_bounds__(1024) void xent_few_kernel(const f32x2* __restrict__ partial, int slots, int tokens,
                                                        const float* __restrict__ target_logit,
                                                        const int64_t* __restrict__ target, int64_t vocab,
                                                        float* __restrict__ loss, float* __restrict__ lse,
                                                        zero_xent_result_t* __restrict__ out) {
    __shared__ f32x2 s_part[16];
    __shared__ float s_loss[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    int share = 1;                                     // waves of one token
    while (share * 2 * tokens <= 16) share *= 2;
    const int n = wave / share;
    float top = -__builtin_inff(), sum = 0.0f;
    if (n < tokens) {
        #pragma unroll 4
        for (int s = (wave % share) * 64 + lane; s < slots; s += share * 64) {
            const f32x2 p = partial[static_cast<int64_t>(s) * tokens + n];
            join(top, sum, p.x, p.y);
        }
    }
    #pragma unroll
    for (int off = 1; off < 64; off *= 2) {
        const float t = __shfl_xor(top, off, 64), u = __shfl_xor(sum, off, 64);
        join(top, sum, t, u);
    }
    if (lane == 0) s_part[wave] = f32x2{top, sum};
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(tokens)) {
        const int i = threadIdx.x;
        top = s_part[i * share].x;
        sum = s_part[i * share].y;
        for (int k = 1; k < share; ++k) join(top, sum, s_part[i * share + k].x, s_part[i * share + k].y);
        const float l = top + logf(sum);
        const int64_t t = target[i];
        lse[i] = l;
        loss[i] = s_loss[i] = t >= 0 && t < vocab ? l - target_logit[i] : 0.0f;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
        int count = 0, beyond = 0;
        for (int i = 0; i < tokens; ++i) {
            const int64_t t = target[i];
            total += static_cast<double>(s_loss[i]);
            count += t >= 0 && t < vocab;
            beyond += t >= vocab;
        }
        write_mean(total, count, beyond, out);
    }
}

__global__ __launch_bounds__(1024) void xent_mean_kernel(const float* __restrict__ loss,
                                                         const int64_t* __restrict__ target, int64_t tokens,
                                                         int64_t vocab, zero_xent_result_t* __restrict__ out) {
    __shared__ double s_sum[1024];
    __shared__ int64_t s_count[1024];
    __shared__ int s_beyond[1024];
    double sum = 0.0;
    int64_t count = 0;
    int beyond = 0;
    for (int64_t i = threadIdx.x; i < tokens; i += 1024) {
        const int64_t t = target[i];
        sum += static_cast<double>(loss[i]);
        count += t >= 0 && t < vocab;
        beyond += t >= vocab;
    }
    s_sum[threadIdx.x] = sum;
    s_count[threadIdx.x] = count;
    s_beyond[threadIdx.x] = beyond;
    __syncthreads();
    for (unsigned half = 512; half > 0; half >>= 1) {
        if (threadIdx.x < half) {
            s_sum[threadIdx.x] += s_sum[threadIdx.x + half];
            s_count[threadIdx.x] += s_count[threadIdx.x + half];
            s_beyond[threadIdx.x] += s_beyond[threadIdx.x + half];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) write_mean(s_sum[0], s_count[0], s_beyond[0], out);
}

// The slabs' sum times the factor, 16 bits; slabs in order.  With `rank` a
// row's sum is in row rank[r], and 0 where that is negative.
template <int DT>
__global__ __launch_bounds__(256) void slab_sum_kernel(const float* __restrict__ slabs, int n_slabs, int64_t slab,
                                                       int64_t rows, int64_t dim, int64_t ld,
                                                       const zero_xent_result_t* __restrict__ result, float scale,
                                                       const int32_t* __restrict__ rank,
                                                       unsigned short* __restrict__ out, int64_t out_stride) {
    typedef u32x2 quad __attribute__((aligned(2)));
    const int64_t quads = ld / 4;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < rows * quads;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = at / quads, d = (at - r * quads) * 4;
        if (d >= dim) continue;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        const int64_t from = rank ? rank[r] : r;
        for (int s = 0; s < (from < 0 ? 0 : n_slabs); ++s) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(slabs + s * slab + from * ld + d);
            #pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += y[e];
        }
        const float f = scale * result->inv_count;
        unsigned short* o = out + r * out_stride + d;
        if (d + 4 <= dim) {
            u32x2 v;
            v.x = pack2<DT>(x[0] * f, x[1] * f);
            v.y = pack2<DT>(x[2] * f, x[3] * f);
            *reinterpret_cast<quad*>(o) = v;
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < dim) o[e] = pack1<DT>(x[e] * f);
        }
    }
}

// Rows of any stride and alignment into rows of ld elements (a multiple of
// 64), zeros past dim: what the products read where the caller's rows are
// not whole 16-byte pieces.
__global__ __launch_bounds__(256) void repack_kernel(const unsigned short* __restrict__ src, int64_t stride,
                                                     int64_t rows, int64_t dim, int64_t ld,
                                                     unsigned short* __restrict__ dst) {
    const int64_t pieces = ld / 8;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < rows * pieces;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = at / pieces, d = (at - r * pieces) * 8;
        *reinterpret_cast<u32x4*>(dst + r * ld + d) = row_piece(src + r * stride, d, dim);
    }
}

// ------------------------------------------------------------------ launches
// The tokens that have a target, one after another: their rows of x (as
// repack_kernel lays them), targets and lse, how many they are, and every
// token's place among them (-1: none).  The gradient's products then run
// over these alone: a masked token costs nothing there, and what its row
// holds, be it NaN, reaches no sum.  A block places `chunk` tokens and
// counts those before them by itself.
__global__ __launch_bounds__(256) void gather_kernel(const unsigned short* __restrict__ x, int64_t stride, int64_t dim,
                                                     int64_t ld, const int64_t* __restrict__ target,
                                                     const float* __restrict__ lse, int64_t vocab, int tokens,
                                                     int chunk, unsigned short* __restrict__ x_out,
                                                     int64_t* __restrict__ target_out, float* __restrict__ lse_out,
                                                     int32_t* __restrict__ rank, int32_t* __restrict__ kept) {
    __shared__ int s_count[4], s_rank[256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int first = blockIdx.x * chunk, last = first + chunk < tokens ? first + chunk : tokens;
    auto has = [&](int i, int end) { return i < end && target[i] >= 0 && target[i] < vocab; };
    // the four waves' counts as one; every thread calls it
    auto join = [&](int mine, int* before) {
        __syncthreads();
        if (lane == 0) s_count[wave] = mine;
        __syncthreads();
        int all = 0;
        *before = 0;
        for (int k = 0; k < 4; ++k) {
            *before += k < wave ? s_count[k] : 0;
            all += s_count[k];
        }
        return all;
    };
    int mine = 0, before = 0;
    for (int i = 0; i < first; i += 256) mine += __popcll(__builtin_amdgcn_ballot_w64(has(i + threadIdx.x, first)));
    int base = join(mine, &before);
    for (int b = first; b < last; b += 256) {
        const int i = b + threadIdx.x;
        const bool here = has(i, last);
        const uint64_t mask = __builtin_amdgcn_ballot_w64(here);
        const int all = join(__popcll(mask), &before);
        const int at = base + before + __popcll(mask & ((uint64_t(1) << lane) - 1));
        base += all;
        s_rank[threadIdx.x] = here ? at : -1;
        if (i < last) rank[i] = here ? at : -1;
        if (here) {
            target_out[at] = target[i];
            lse_out[at] = lse[i];
        }
        __syncthreads();
        const int n = last - b < 256 ? last - b : 256;
        for (int r = wave; r < n; r += 4) {
            const int64_t to = s_rank[r];
            if (to < 0) continue;
            for (int64_t d = lane * 8; d < ld; d += 512)
                *reinterpret_cast<u32x4*>(x_out + to * ld + d) = row_piece(x + (b + r) * stride, d, dim);
        }
    }
    if (last == tokens && threadIdx.x == 0) *kept = base;
}

// No token: nothing to add up, dw is zero.
__global__ __launch_bounds__(256) void zero_rows_kernel(unsigned short* __restrict__ out, int64_t stride,
                                                        int64_t rows, int64_t dim) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t d = threadIdx.x; d < dim; d += 256) out[r * stride + d] = 0;
}

// ------------------------------------------------------------------ launches
// How a problem is cut.  Everything depends on the three sizes only, and on
// whether w is repacked.
struct Cut {
    int64_t dim_pad;          // row of a repacked operand and of a slab
    int64_t piece;            // vocabulary of one piece of the backward, a multiple of 256
    int64_t p_row;            // row of P
    int64_t slots;            // most partials per token of the forward
    int32_t dx_slices, dw_slices;
    size_t x_bytes, row_bytes, w_bytes, p_bytes, slab_bytes, part_bytes;
    size_t total;
};

constexpr int64_t kMaxTokens = int64_t(1) << 20, kMaxDim = int64_t(1) << 20, kMaxVocab = int64_t(1) << 24;
constexpr int64_t kFewTokens = 8;             // few_kernel's rule
// Beside a row of P, so that the rows of one column lie in unlike channels of
// memory (gradient of 4096 x 4096 x 128000: 9.53 ms without, 9.45 with).
constexpr int64_t kPPad = 192;
// Of P, and of a piece of w repacked.  A larger piece costs room and saves
// dx's slab a trip: there, of 64 MB of P 12.5 ms with the forward, of 256 MB
// 12.3.
constexpr int64_t kPBytes = int64_t(256) << 20, kPackedBytes = int64_t(128) << 20;

void cut_piece(int64_t tokens, int64_t dim, int64_t vocab, bool packed, Cut* c) {
    c->dim_pad = up(dim > 0 ? dim : 1, 64);
    const int64_t t = tokens > 0 ? tokens : 1, v = up(vocab > 0 ? vocab : 1, 256);
    int64_t piece = (packed ? kPackedBytes : kPBytes) / (2 * t);
    if (packed && kPackedBytes / (2 * c->dim_pad) < piece) piece = kPackedBytes / (2 * c->dim_pad);
    piece = piece / 256 * 256;
    c->piece = piece < 256 ? 256 : (piece > v ? v : piece);
    c->slots = t <= kFewTokens ? v / 16 : v / 64;
    // slices of k where the tiles of 128 x 128 alone would leave CUs idle
    const int64_t dim_tiles = up(dim, 128) / 128;
    auto slices = [](int64_t tiles, int64_t k) {
        int64_t s = 512 / (tiles > 0 ? tiles : 1);
        if (s > k / 512) s = k / 512;
        return static_cast<int32_t>(s < 1 ? 1 : (s > 64 ? 64 : s));
    };
    c->dx_slices = slices(dim_tiles * (up(t, 128) / 128), c->piece);
    c->dw_slices = slices(dim_tiles * (up(c->piece, 128) / 128), t);
    c->x_bytes = round_up(static_cast<size_t>(t * c->dim_pad) * 2, 256);
    c->row_bytes = 256 + round_up(static_cast<size_t>(t) * 16, 256);
    c->w_bytes = packed ? round_up(static_cast<size_t>(c->piece * c->dim_pad) * 2, 256) : 0;
    c->p_row = c->piece + kPPad;
    c->p_bytes = round_up(static_cast<size_t>(t * c->p_row) * 2, 256);
    size_t slab = static_cast<size_t>(c->dx_slices) * t * c->dim_pad * 4;
    if (c->dw_slices > 1) slab += static_cast<size_t>(c->dw_slices) * c->piece * c->dim_pad * 4;
    c->slab_bytes = round_up(slab, 256);
    c->part_bytes = round_up(static_cast<size_t>(c->slots) * t * 8, 256) + round_up(static_cast<size_t>(t) * 4, 256);
    const size_t back = c->row_bytes + c->p_bytes + c->slab_bytes;
    c->total = c->x_bytes + c->w_bytes + (back > c->part_bytes ? back : c->part_bytes);
}

// False for sizes out of range.
bool cut(int64_t tokens, int64_t dim, int64_t vocab, bool packed, Cut* c) {
    if (tokens < 0 || tokens > kMaxTokens || dim < 0 || dim > kMaxDim || vocab < 0 || vocab > kMaxVocab)
        return false;
    if (tokens > 0 && (dim < 1 || vocab < 1)) return false;
    cut_piece(tokens, dim, vocab, packed, c);
    return true;
}

// Blocks of 256 threads for n items, each walking the rest of the grid.
unsigned blocks_for(int64_t n) {
    const int64_t b = (n + 255) / 256;
    return static_cast<unsigned>(b < (1 << 20) ? b : (1 << 20));
}

// One 16-bit matrix as the products read it: the caller's own rows where
// they are whole 16-byte pieces, else rows repacked into the workspace.
void launch_repack(const void* src, int64_t stride, int64_t rows, int64_t dim, int64_t ld, void* dst, hipStream_t st) {
    const int64_t n = rows * (ld / 8);
    hipLaunchKernelGGL(repack_kernel, dim3(blocks_for(n)), dim3(256), 0, st,
                       static_cast<const unsigned short*>(src), stride, rows, dim, ld,
                       static_cast<unsigned short*>(dst));
}

struct Matrix {
    const char* p;
    int64_t stride;           // bytes
    int32_t dim;              // readable elements of a row, a multiple of 8
};
Matrix prepared(const void* src, int64_t stride, int64_t first, int64_t rows, int64_t dim, int64_t dim_pad,
                void* room, hipStream_t st) {
    const unsigned short* at = static_cast<const unsigned short*>(src) + first * stride;
    if (whole_pieces(src, stride, dim)) return {reinterpret_cast<const char*>(at), stride * 2, static_cast<int32_t>(dim)};
    launch_repack(at, stride, rows, dim, dim_pad, room, st);
    return {static_cast<const char*>(room), dim_pad * 2, static_cast<int32_t>(dim_pad)};
}

template <int DT>
int forward(const zero_xent_args* a, const Cut& c, hipStream_t st) {
    char* ws = static_cast<char*>(a->workspace);
    char* xr = ws;
    char* wr = ws + c.x_bytes;
    float* partial = reinterpret_cast<float*>(wr + c.w_bytes);
    float* hit = reinterpret_cast<float*>(reinterpret_cast<char*>(partial) +
                                          round_up(static_cast<size_t>(c.slots) * a->tokens * 8, 256));
    const Matrix x = prepared(a->x, a->x_stride, 0, a->tokens, a->dim, c.dim_pad, xr, st);
    // the caller's w whole, a repacked one piece by piece
    // (at most 2^22 tiles a launch)
    const int64_t most = (int64_t(1) << 22) / (up(a->tokens, 128) / 128) * 128;
    const int64_t whole = most < a->vocab ? most : a->vocab;
    const int64_t piece = whole_pieces(a->w, a->w_stride, a->dim) ? whole : c.piece;
    int slots = 0;
    for (int64_t v = 0; v < a->vocab; v += piece) {
        const int64_t rows = a->vocab - v < piece ? a->vocab - v : piece;
        const Matrix w = prepared(a->w, a->w_stride, v, rows, a->dim, c.dim_pad, wr, st);
        Product q = {};
        q.a = w.p;
        q.lda = w.stride;
        q.b = x.p;
        q.ldb = x.stride;
        q.m = static_cast<int32_t>(rows);
        q.n = static_cast<int32_t>(a->tokens);
        q.k = w.dim < x.dim ? w.dim : x.dim;
        q.slice = static_cast<int32_t>(up(q.k, kTileK));
        q.first_m = static_cast<int32_t>(v);
        q.slot0 = slots;
        q.target = a->target;
        q.partial = partial;
        q.target_logit = hit;
        q.vocab = static_cast<int32_t>(a->vocab);
        if (a->tokens <= kFewTokens) {
            hipLaunchKernelGGL((few_kernel<DT>), dim3(static_cast<unsigned>((rows + 15) / 16)), dim3(256), 0, st, q);
            slots += static_cast<int>((rows + 15) / 16);
        } else if (large_tiles(q, 1)) {
            launch_tiles<DT, kRows, kRows, kLse, 256, 256, 2, 2>(q, 1, st);
            slots += static_cast<int>(up(rows, 256) / 256 * 2);
        } else {
            launch_tiles<DT, kRows, kRows, kLse, 128, 128, 2, 2>(q, 1, st);
            slots += static_cast<int>(up(rows, 128) / 128 * 2);
        }
    }
    if (a->tokens <= kFewTokens) {
        hipLaunchKernelGGL(xent_few_kernel, dim3(1), dim3(1024), 0, st, reinterpret_cast<const f32x2*>(partial), slots,
                           static_cast<int>(a->tokens), hit, a->target, a->vocab, a->loss, a->lse, a->result);
        return launch_error("loss kernel launch");
    }
    hipLaunchKernelGGL(xent_rows_kernel, dim3(static_cast<unsigned>((a->tokens + 15) / 16)), dim3(1024), 0, st,
                       reinterpret_cast<const f32x2*>(partial), slots, static_cast<int>(a->tokens), hit, a->target,
                       a->vocab, a->loss, a->lse);
    return launch_error("loss kernel launch");
}

template <int DT>
int backward(const zero_xent_args* a, const Cut& c, hipStream_t st) {
    char* ws = static_cast<char*>(a->workspace);
    unsigned short* xg = reinterpret_cast<unsigned short*>(ws);
    int32_t* kept = reinterpret_cast<int32_t*>(ws + c.x_bytes);
    int64_t* target = reinterpret_cast<int64_t*>(ws + c.x_bytes + 256);
    float* lse = reinterpret_cast<float*>(target + a->tokens);
    int32_t* rank = reinterpret_cast<int32_t*>(lse + a->tokens);
    char* wr = ws + c.x_bytes + c.row_bytes;
    char* p16 = wr + c.w_bytes;
    float* dx_slab = reinterpret_cast<float*>(p16 + c.p_bytes);
    float* dw_slab = dx_slab + static_cast<int64_t>(c.dx_slices) * a->tokens * c.dim_pad;
    const int tokens = static_cast<int>(a->tokens);
    const int chunk = tokens / 1024 > 16 ? tokens / 1024 : 16;
    hipLaunchKernelGGL(gather_kernel, dim3(static_cast<unsigned>((tokens + chunk - 1) / chunk)), dim3(256), 0, st,
                       static_cast<const unsigned short*>(a->x), a->x_stride, a->dim, c.dim_pad, a->target, a->lse,
                       a->vocab, tokens, chunk, xg, target, lse, rank, kept);
    const Matrix x = {reinterpret_cast<const char*>(xg), c.dim_pad * 2, static_cast<int32_t>(c.dim_pad)};
    // fp16 holds 2^-24 at best, a probability of a large vocabulary is often
    // less: P is held times 2^15 there (at most 32768, below fp16's 65504)
    const float pscale = DT == ZERO_FP16 ? 32768.0f : 1.0f;
    const float grad = static_cast<float>(a->grad_scale / pscale);
    for (int64_t v = 0; v < a->vocab; v += c.piece) {
        const int64_t rows = a->vocab - v < c.piece ? a->vocab - v : c.piece;
        const Matrix w = prepared(a->w, a->w_stride, v, rows, a->dim, c.dim_pad, wr, st);
        const int32_t kdim = w.dim < x.dim ? w.dim : x.dim;
        Product q = {};
        q.a = w.p;
        q.lda = w.stride;
        q.b = x.p;
        q.ldb = x.stride;
        q.m = static_cast<int32_t>(rows);
        q.n = static_cast<int32_t>(a->tokens);
        q.k = kdim;
        q.slice = static_cast<int32_t>(up(q.k, kTileK));
        q.first_m = static_cast<int32_t>(v);
        q.target = target;
        q.lse = lse;
        q.kept = kept;
        q.vocab = static_cast<int32_t>(a->vocab);
        q.c = p16;
        q.ldc = c.p_row;
        q.scale = pscale;
        launch_product<DT, kRows, kRows, kProb>(q, 1, st);

        // dx += P w: k is the piece's vocabulary
        Product d = {};
        d.a = w.p;
        d.lda = w.stride;
        d.b = p16;
        d.ldb = c.p_row * 2;
        d.m = w.dim;
        d.n = q.n;
        d.k = q.m;
        d.slice = static_cast<int32_t>(up(up(d.k, c.dx_slices) / c.dx_slices, kTileK));
        d.c = reinterpret_cast<char*>(dx_slab);
        d.ldc = c.dim_pad;
        d.slab = a->tokens * c.dim_pad;
        d.add = v > 0;
        d.kept = kept;
        launch_product<DT, kCols, kRows, kSlab>(d, c.dx_slices, st);

        // dw = P^T x: k is the tokens
        Product e = {};
        e.a = x.p;
        e.lda = x.stride;
        e.b = p16;
        e.ldb = c.p_row * 2;
        e.m = x.dim;
        e.n = q.m;
        e.k = q.n;
        e.kept = kept;
        unsigned short* dw = static_cast<unsigned short*>(a->dw) + v * a->dw_stride;
        if (c.dw_slices > 1) {
            e.slice = static_cast<int32_t>(up(up(e.k, c.dw_slices) / c.dw_slices, kTileK));
            e.c = reinterpret_cast<char*>(dw_slab);
            e.ldc = c.dim_pad;
            e.slab = c.piece * c.dim_pad;
            // more than one slice only where tiles times slices are at most 512
            // of 128 x 128, one round of the chip: large_tiles is false
            launch_tiles<DT, kCols, kCols, kSlab, 128, 128, 2, 2>(e, c.dw_slices, st);
            hipLaunchKernelGGL((slab_sum_kernel<DT>),
                               dim3(blocks_for(rows * (c.dim_pad / 4))), dim3(256), 0, st,
                               dw_slab, c.dw_slices, e.slab, rows, a->dim, c.dim_pad, a->result, grad, nullptr,
                               dw, a->dw_stride);
        } else {
            e.slice = static_cast<int32_t>(up(e.k, kTileK));
            e.c = reinterpret_cast<char*>(dw);
            e.ldc = a->dw_stride;
            e.valid_m = static_cast<int32_t>(a->dim);
            e.result = a->result;
            e.scale = grad;
            launch_product<DT, kCols, kCols, kGrad>(e, 1, st);
        }
    }
    hipLaunchKernelGGL((slab_sum_kernel<DT>),
                       dim3(blocks_for(a->tokens * (c.dim_pad / 4))), dim3(256), 0, st,
                       dx_slab, c.dx_slices, a->tokens * c.dim_pad, a->tokens, a->dim, c.dim_pad, a->result, grad,
                       rank, static_cast<unsigned short*>(a->dx), a->dx_stride);
    return launch_error("loss gradient kernel launch");
}

}  // namespace

size_t xent_needs(int64_t tokens, int64_t dim, int64_t vocab) {
    // room for either layout of w
    Cut whole, packed;
    if (!cut(tokens, dim, vocab, false, &whole) || !cut(tokens, dim, vocab, true, &packed)) return 0;
    return dim % 8 == 0 && whole.total > packed.total ? whole.total : packed.total;
}

}  // namespace zero

using namespace zero;

extern "C" {

size_t zero_xent_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab) {
    size_t most = xent_needs(tokens, dim, vocab);
    if (!most) return 0;
    // Fewer tokens may need more: they are cut into more slices, have wider
    // pieces of the vocabulary or, few of them, more partials.  Between two of
    // these numbers nothing but the tokens grows.
    int64_t last = 0;
    auto look = [&](int64_t t) {
        if (t < 1 || t >= tokens || t == last) return;
        last = t;
        const size_t b = xent_needs(t, dim, vocab);
        most = b > most ? b : most;
    };
    look(kFewTokens);
    for (int64_t t = 128; t < tokens; t += 128) look(t);
    for (const int64_t room : {kPBytes, kPackedBytes})
        for (int64_t piece = 256; piece <= up(vocab, 256); piece += 256) look(room / 2 / piece);
    return most;
}

int zero_xent_forward(const zero_xent_args* a, void* stream) {
    clear_error();
    int rc = check_xent_args(a, false);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->tokens > 0) {
        Cut c;
        cut(a->tokens, a->dim, a->vocab, !whole_pieces(a->w, a->w_stride, a->dim), &c);
        rc = a->dtype == ZERO_BF16 ? forward<ZERO_BF16>(a, c, st) : forward<ZERO_FP16>(a, c, st);
        if (rc || a->tokens <= kFewTokens) return rc;
    }
    hipLaunchKernelGGL(xent_mean_kernel, dim3(1), dim3(1024), 0, st, a->loss, a->target, a->tokens, a->vocab,
                       a->result);
    return launch_error("loss mean kernel launch");
}

int zero_xent_backward(const zero_xent_args* a, void* stream) {
    clear_error();
    const int rc = check_xent_args(a, true);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->tokens == 0) {
        if (a->vocab > 0 && a->dim > 0)
            hipLaunchKernelGGL(zero_rows_kernel, dim3(static_cast<unsigned>(a->vocab < 4096 ? a->vocab : 4096)),
                               dim3(256), 0, st, static_cast<unsigned short*>(a->dw), a->dw_stride, a->vocab, a->dim);
        return launch_error("loss gradient kernel launch");
    }
    Cut c;
    cut(a->tokens, a->dim, a->vocab, !whole_pieces(a->w, a->w_stride, a->dim), &c);
    return a->dtype == ZERO_BF16 ? backward<ZERO_BF16>(a, c, st) : backward<ZERO_FP16>(a, c, st);
}

}  // extern "C"
