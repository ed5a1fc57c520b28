// train_xent.hip -- softmax cross entropy of a large vocabulary and its
// gradient (include/zero/train.h), without keeping the logits.
//
//   forward    L = w x^T tile by tile on the matrix cores; each tile leaves,
//              per token and wave row, its largest logit and the sum of
//              exponentials below it (one pass of a running softmax), and
//              the target's logit; a second kernel joins them into lse and
//              loss, a third sums the losses.
//   backward   piece by piece of the vocabulary: L again, P = exp(L - lse) -
//              onehot rounded to 16 bits into the workspace, then
//              dx += P w (fp32 in the workspace) and dw = P^T x.
//
// One tile product serves all of it.  An operand lies with its rows along k
// (x and w in the logits, P in dx) or with k as the row (w in dx; x and P in
// dw); the second kind is turned on the way from LDS to the registers, so
// nothing is ever transposed in memory.
#include <hip/hip_runtime.h>

#include "train_internal.h"
#include "zero_device.h"

namespace zero {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

#define ZERO_LDS __attribute__((address_space(3)))

constexpr int kTileK = 64;
constexpr uint32_t kNowhere = 0x80000000u;   // past every descriptor: loads 0

enum Layout { kRows, kCols };   // the operand's rows lie along k, or k is the row

// What a product writes.
enum Epilogue {
    kLse,       // partial maxima and sums of exponentials, target logits
    kProb,      // P, 16 bits
    kSlab,      // fp32 partial products of one slice of k
    kGrad       // the product times a factor, 16 bits
};

// C[n][m] = sum_k A(m, k) B(n, k): m is the contiguous axis of the result.
struct Product {
    const char* a;
    const char* b;
    int64_t lda, ldb;         // bytes from row to row
    int32_t m, n, k;          // extents; along a kCols operand's m or n whole 16 bytes are read
    int32_t tiles_m, tiles_n;
    int32_t slice;            // k of one slice, a multiple of kTileK
    // epilogues
    char* c;                  // P, slabs or gradient
    int64_t ldc;              // elements
    int64_t slab;             // elements from slab to slab
    int32_t add;              // kSlab: add to what is there
    int32_t valid_m;          // columns m beyond it are not stored (kGrad)
    int32_t first_m;          // vocabulary index of m = 0 (kLse, kProb)
    int32_t slot0;            // kLse: first slot
    const int64_t* target;
    const float* lse;
    float* partial;           // kLse: float2[slot][n]
    float* target_logit;      // kLse
    const zero_xent_result_t* result;   // kGrad: inv_count
    float scale;              // kProb: applied before rounding; kGrad: undone, times grad_scale
    int32_t vocab;
};

// Where 16-byte piece c of a tile's row lies: rows-along-k tiles (8 pieces a
// row) swap pieces by the row, so that 16 lanes reading one piece of 16 rows
// meet 16 different 16-byte bank groups; k-as-row tiles swap pairs of pieces
// by k, so that the 4 x 16 blocks of a turning read spread over the banks.
__device__ __forceinline__ int swap_rows(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swap_cols(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }

template <int DT>
__device__ __forceinline__ f32x4 mfma(const s16x8 a, const s16x8 b, const f32x4 c) {
    if constexpr (DT == ZERO_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// One operand's tile of R rows (m or n) by kTileK: this thread's share of
// the loads into LDS, and its fragments out of it.
template <Layout L, int R, int THREADS>
struct Operand {
    static constexpr int kPieces = R * kTileK / 8;          // of 16 bytes
    static_assert(kPieces % 64 == 0, "whole waves load");
    static constexpr int kLoads = (kPieces + THREADS - 1) / THREADS;
    static constexpr int kRowPieces = L == kRows ? kTileK / 8 : R / 8;
    static constexpr int kRowsALoad = THREADS / kRowPieces;
    // a thread's later loads are the same piece of later rows
    static_assert(kLoads == 1 || kRowsALoad % 16 == 0, "swaps repeat every 16 rows");
    uint32_t off;             // of the first piece, or kNowhere
    int32_t along;            // kRows: its first k
    uint32_t next;            // bytes from load to load
    int64_t row, rows;        // bytes of a row; kRows: of the rows from the tile's first on

    __device__ __forceinline__ void setup(int64_t ld, int rows_left) {
        const int r = threadIdx.x / kRowPieces, c = threadIdx.x % kRowPieces;
        row = ld;
        next = static_cast<uint32_t>(kRowsALoad * ld);
        if constexpr (L == kRows) {
            const int piece = c ^ swap_rows(r);
            off = static_cast<uint32_t>(r * ld + piece * 16);
            along = piece * 8;
            rows = rows_left * ld;
        } else {
            const int piece = c ^ swap_cols(r);
            off = piece * 8 < rows_left ? static_cast<uint32_t>(r * ld + piece * 16) : kNowhere;
        }
    }
    // `base`: the tile's first byte at this step of k, `into` bytes into its
    // row; k_left: k from here on.  The descriptor ends with the last row, so
    // rows past it load 0; so does a piece of k past the end.
    __device__ __forceinline__ void load(const char* base, int64_t into, int k_left, ZERO_LDS char* lds) const {
        int64_t bytes = (L == kRows ? rows : k_left * row) - into;
        bytes = bytes < 0x7ffffff0 ? bytes : 0x7ffffff0;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(base), 0, static_cast<int>(bytes), 0x00020000);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        if constexpr (kPieces < THREADS) {
            if (wave * 64 >= kPieces) return;
        }
        uint32_t o = L == kCols || along < k_left ? off : kNowhere;
        #pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (ZERO_LDS void*)(lds + (j * THREADS + wave * 64) * 16),
                                                     16, o, 0, 0, 0);
            o += next;
        }
    }
    // Lane l's 8 values of the fragment at row r0 (a multiple of 16), half h
    // of the tile's k: row r0 + l % 16, k = 32 h + 8 (l / 16) + 0..7.
    __device__ __forceinline__ static s16x8 fragment(const ZERO_LDS char* lds, int r0, int h) {
        const int l = threadIdx.x & 63, s = l & 15, g = l >> 4;
        if constexpr (L == kRows) {
            const int c = (h * 4 + g) ^ swap_rows(s);
            return *(const ZERO_LDS s16x8*)(lds + (r0 + s) * (kTileK * 2) + c * 16);
        } else {
            // the 16 lanes of group g give 4 rows of k by 16 of m and get them turned
            const int k = h * 32 + g * 8 + (s >> 2);
            const int u = (r0 / 16) ^ (swap_cols(k) >> 1);
            const ZERO_LDS char* at = lds + k * (R * 2) + u * 32 + (s & 3) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_LDS s16x4*)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_LDS s16x4*)(at + 4 * R * 2));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

__device__ __forceinline__ bool infinite(float x) { return __builtin_fabsf(x) == __builtin_inff(); }

template <int DT, Layout LA, Layout LB, Epilogue E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void product_kernel(const Product q) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;     // fragments of a wave
    typedef Operand<LA, BM, kThreads> OpA;
    typedef Operand<LB, BN, kThreads> OpB;
    __shared__ __attribute__((aligned(1024))) char a0[BM * kTileK * 2];
    __shared__ __attribute__((aligned(1024))) char b0[BN * kTileK * 2];
    __shared__ __attribute__((aligned(1024))) char a1[BM * kTileK * 2];
    __shared__ __attribute__((aligned(1024))) char b1[BN * kTileK * 2];

    // Each XCD takes a contiguous run of tiles, ordered in strips of 4 along
    // n, so the tiles its 32 CUs hold at a time share rows of both operands.
    const int tiles = q.tiles_m * q.tiles_n;
    int id = blockIdx.x;
    {
        const int per = tiles / kXcds, extra = tiles % kXcds;
        const int x = id % kXcds, i = id / kXcds;
        id = x * per + (x < extra ? x : extra) + i;
    }
    constexpr int kStrip = 4;
    const int strip = id / (kStrip * q.tiles_m);
    const int width = q.tiles_n - strip * kStrip < kStrip ? q.tiles_n - strip * kStrip : kStrip;
    const int in_strip = id - strip * kStrip * q.tiles_m;
    const int tn = strip * kStrip + in_strip % width, tm = in_strip / width;
    const int m0 = tm * BM, n0 = tn * BN;

    const int k_lo = static_cast<int>(blockIdx.y) * q.slice;
    const int k_hi = q.k < k_lo + q.slice ? q.k : k_lo + q.slice;
    const int steps = k_hi > k_lo ? (k_hi - k_lo + kTileK - 1) / kTileK : 0;

    OpA oa;
    OpB ob;
    oa.setup(q.lda, q.m - m0);
    ob.setup(q.ldb, q.n - n0);
    // bytes from one step of k to the next
    const int64_t sa = LA == kRows ? kTileK * 2 : kTileK * q.lda;
    const int64_t sb = LB == kRows ? kTileK * 2 : kTileK * q.ldb;
    const char* pa = q.a + (LA == kRows ? m0 * q.lda + k_lo * 2 : k_lo * q.lda + m0 * 2);
    const char* pb = q.b + (LB == kRows ? n0 * q.ldb + k_lo * 2 : k_lo * q.ldb + n0 * 2);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
    f32x4 acc[FM][FN];
    #pragma unroll
    for (int i = 0; i < FM; ++i)
        #pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto load = [&](char* sha, char* shb, int step) {
        const int left = k_hi - k_lo - step * kTileK;
        oa.load(pa + step * sa, LA == kRows ? (k_lo + step * kTileK) * 2 : m0 * 2, left, (ZERO_LDS char*)sha);
        ob.load(pb + step * sb, LB == kRows ? (k_lo + step * kTileK) * 2 : n0 * 2, left, (ZERO_LDS char*)shb);
    };
    auto multiply = [&](const char* sha, const char* shb) {
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            // both halves' fragments at once would not fit the registers
            __builtin_amdgcn_sched_barrier(0);
            s16x8 fa[FM], fb[FN];
            #pragma unroll
            for (int i = 0; i < FM; ++i) fa[i] = OpA::fragment((const ZERO_LDS char*)sha, wm + i * 16, h);
            #pragma unroll
            for (int j = 0; j < FN; ++j) fb[j] = OpB::fragment((const ZERO_LDS char*)shb, wn + j * 16, h);
            #pragma unroll
            for (int i = 0; i < FM; ++i)
                #pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma<DT>(fa[i], fb[j], acc[i][j]);
        }
    };
    // a stage is read only after its loads arrived in every wave, and loaded
    // again only after every wave has read it
    auto turn = [] {
        __builtin_amdgcn_s_waitcnt(0x0f70);            // vmcnt(0): the loads into LDS
        __syncthreads();
    };
    if (steps > 0) load(a0, b0, 0);
    int s = 0;
    for (; s + 2 <= steps; s += 2) {
        turn();
        load(a1, b1, s + 1);
        multiply(a0, b0);
        turn();
        if (s + 2 < steps) load(a0, b0, s + 2);
        multiply(a1, b1);
    }
    if (s < steps) {
        turn();
        multiply(a0, b0);
    }

    // acc[i][j][e] is C at n = n0 + wn + 16 j + lane % 16,
    // m = m0 + wm + 16 i + 4 (lane / 16) + e
    const int lane = threadIdx.x & 63, nl = lane & 15, ml = (lane >> 4) * 4;
    if constexpr (E == kLse) {
        const int slot = q.slot0 + tm * WM + wave % WM;
        #pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = n0 + wn + j * 16 + nl;
            const bool live = n < q.n;
            // position of the target among this lane's m, if it is there
            const int64_t tgt = live ? q.target[n] : -1;
            const int64_t at = tgt - q.first_m - m0 - wm - ml;
            float top = -__builtin_inff(), hit = 0.0f;
            bool found = false;
            #pragma unroll
            for (int i = 0; i < FM; ++i)
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (m0 + wm + i * 16 + ml + e >= q.m) acc[i][j][e] = -__builtin_inff();
                    top = fmaxf(top, acc[i][j][e]);
                    if (at == i * 16 + e) {
                        hit = acc[i][j][e];
                        found = true;
                    }
                }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float base = infinite(top) ? 0.0f : top;
            float sum = 0.0f;
            #pragma unroll
            for (int i = 0; i < FM; ++i)
                #pragma unroll
                for (int e = 0; e < 4; ++e) sum += __expf(acc[i][j][e] - base);
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            if (live && lane < 16)
                reinterpret_cast<f32x2*>(q.partial)[static_cast<int64_t>(slot) * q.n + n] = f32x2{top, sum};
            if (found && tgt < q.vocab) q.target_logit[n] = hit;
        }
    } else if constexpr (E == kProb) {
        #pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = n0 + wn + j * 16 + nl;
            if (n >= q.n) continue;
            const int64_t tgt = q.target[n];
            const bool kept = tgt >= 0 && tgt < q.vocab;
            const float lse = q.lse[n];
            const int64_t at = tgt - q.first_m - m0 - wm - ml;
            unsigned short* row = reinterpret_cast<unsigned short*>(q.c) + n * q.ldc + m0 + wm + ml;
            #pragma unroll
            for (int i = 0; i < FM; ++i) {
                float p[4];
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = __expf(acc[i][j][e] - lse) - (at == i * 16 + e ? 1.0f : 0.0f);
                    p[e] = kept && m0 + wm + i * 16 + ml + e < q.m ? p[e] * q.scale : 0.0f;
                }
                u32x2 o;
                o.x = pack2<DT>(p[0], p[1]);
                o.y = pack2<DT>(p[2], p[3]);
                *reinterpret_cast<u32x2*>(row + i * 16) = o;
            }
        }
    } else if constexpr (E == kSlab) {
        float* c = reinterpret_cast<float*>(q.c) + static_cast<int64_t>(blockIdx.y) * q.slab;
        #pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = n0 + wn + j * 16 + nl;
            if (n >= q.n) continue;
            #pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int m = m0 + wm + i * 16 + ml;
                if (m >= q.m) continue;                   // q.m and ldc are whole quads
                f32x4* at = reinterpret_cast<f32x4*>(c + n * q.ldc + m);
                f32x4 x = acc[i][j];
                if (q.add) {
                    const f32x4 y = *at;
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = y[e] + x[e];
                }
                *at = x;
            }
        }
    } else {
        const float f = q.scale * q.result->inv_count;
        typedef u32x2 quad __attribute__((aligned(2)));
        #pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = n0 + wn + j * 16 + nl;
            if (n >= q.n) continue;
            unsigned short* row = reinterpret_cast<unsigned short*>(q.c) + n * q.ldc;
            #pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int m = m0 + wm + i * 16 + ml;
                const f32x4 x = acc[i][j];
                if (m + 4 <= q.valid_m) {
                    u32x2 o;
                    o.x = pack2<DT>(x[0] * f, x[1] * f);
                    o.y = pack2<DT>(x[2] * f, x[3] * f);
                    *reinterpret_cast<quad*>(row + m) = o;
                } else {
                    #pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (m + e < q.valid_m) row[m + e] = pack1<DT>(x[e] * f);
                }
            }
        }
    }
}

// ------------------------------------------------------- joining the partials
// 16 tokens by 64 slices of the slots in a block; every order is fixed.
__global__ __launch_bounds__(1024) void xent_rows_kernel(const f32x2* __restrict__ partial, int slots, int tokens,
                                                         const float* __restrict__ target_logit,
                                                         const int64_t* __restrict__ target, int64_t vocab,
                                                         float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ float s_top[64][17], s_sum[64][17];
    const int col = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int n = blockIdx.x * 16 + col;
    float top = -__builtin_inff(), sum = 0.0f;
    auto join = [](float& t, float& s, float t2, float s2) {
        const float m = fmaxf(t, t2);
        // equal maxima (also two infinite ones) keep their sums as they are
        s = s * (t == m ? 1.0f : __expf(t - m)) + s2 * (t2 == m ? 1.0f : __expf(t2 - m));
        t = m;
    };
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
    if (threadIdx.x == 0) {
        const double n = s_count[0] > 1 ? static_cast<double>(s_count[0]) : 1.0;
        out->loss_sum = s_sum[0];
        out->count = s_count[0];
        out->out_of_range = s_beyond[0];
        out->reserved = 0;
        out->mean = static_cast<float>(s_sum[0] / n);
        out->inv_count = static_cast<float>(1.0 / n);
    }
}

// The slabs' sum times the factor, 16 bits; slabs in order.
template <int DT>
__global__ __launch_bounds__(256) void slab_sum_kernel(const float* __restrict__ slabs, int n_slabs, int64_t slab,
                                                       int64_t rows, int64_t dim, int64_t ld,
                                                       const zero_xent_result_t* __restrict__ result, float scale,
                                                       unsigned short* __restrict__ out, int64_t out_stride) {
    typedef u32x2 quad __attribute__((aligned(2)));
    const int64_t quads = ld / 4;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < rows * quads;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = at / quads, d = (at - r * quads) * 4;
        if (d >= dim) continue;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < n_slabs; ++s) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(slabs + s * slab + r * ld + d);
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
    typedef u32x4 piece __attribute__((aligned(2)));
    const int64_t pieces = ld / 8;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < rows * pieces;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = at / pieces, d = (at - r * pieces) * 8;
        const unsigned short* s = src + r * stride + d;
        u32x4 o = {0u, 0u, 0u, 0u};
        if (d + 8 <= dim) {
            o = *reinterpret_cast<const piece*>(s);
        } else {
            unsigned w[4] = {0u, 0u, 0u, 0u};
            #pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d + e < dim) w[e / 2] |= static_cast<unsigned>(s[e]) << (16 * (e % 2));
            o = u32x4{w[0], w[1], w[2], w[3]};
        }
        *reinterpret_cast<u32x4*>(dst + r * ld + d) = o;
    }
}

// No token: nothing to add up, dw is zero.
__global__ __launch_bounds__(256) void zero_rows_kernel(unsigned short* __restrict__ out, int64_t stride,
                                                        int64_t rows, int64_t dim) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t d = threadIdx.x; d < dim; d += 256) out[r * stride + d] = 0;
}

// ------------------------------------------------------------------ launches
int launch_error(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(ZERO_EDEVICE, "%s: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

constexpr int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// How a problem is cut.  Everything depends on the three sizes only.
struct Cut {
    int64_t dim_pad;          // row of a repacked operand and of a slab
    int64_t piece;            // vocabulary of one piece of the backward, a multiple of 256
    int64_t slots;            // most partials per token of the forward
    int32_t dx_slices, dw_slices;
    size_t x_bytes, w_bytes, p_bytes, slab_bytes, part_bytes;
    size_t total;
};

constexpr int64_t kMaxTokens = int64_t(1) << 20, kMaxDim = int64_t(1) << 20, kMaxVocab = int64_t(1) << 24;
constexpr int64_t kFewTokens = 16;            // one tile of tokens in the forward
constexpr int64_t kPBytes = int64_t(64) << 20, kWBytes = int64_t(256) << 20;

bool cut(int64_t tokens, int64_t dim, int64_t vocab, Cut* c) {
    if (tokens < 0 || tokens > kMaxTokens || dim < 0 || dim > kMaxDim || vocab < 0 || vocab > kMaxVocab)
        return false;
    if (tokens > 0 && (dim < 1 || vocab < 1)) return false;
    c->dim_pad = up(dim > 0 ? dim : 1, 64);
    const int64_t t = tokens > 0 ? tokens : 1, v = up(vocab > 0 ? vocab : 1, 256);
    int64_t piece = kPBytes / (2 * t);
    if (kWBytes / (2 * c->dim_pad) < piece) piece = kWBytes / (2 * c->dim_pad);
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
    c->w_bytes = round_up(static_cast<size_t>(c->piece * c->dim_pad) * 2, 256);
    c->p_bytes = round_up(static_cast<size_t>(t * c->piece) * 2, 256);
    size_t slab = static_cast<size_t>(c->dx_slices) * t * c->dim_pad * 4;
    if (c->dw_slices > 1) slab += static_cast<size_t>(c->dw_slices) * c->piece * c->dim_pad * 4;
    c->slab_bytes = round_up(slab, 256);
    c->part_bytes = round_up(static_cast<size_t>(c->slots) * t * 8, 256) + round_up(static_cast<size_t>(t) * 4, 256);
    const size_t back = c->p_bytes + c->slab_bytes;
    c->total = c->x_bytes + c->w_bytes + (back > c->part_bytes ? back : c->part_bytes);
    return true;
}

// Blocks of 256 threads for n items, each walking the rest of the grid.
unsigned blocks_for(int64_t n) {
    const int64_t b = (n + 255) / 256;
    return static_cast<unsigned>(b < (1 << 20) ? b : (1 << 20));
}

template <int DT, Layout LA, Layout LB, Epilogue E, int BM, int BN, int WM, int WN>
void launch_tiles(Product q, int slices, hipStream_t st) {
    q.tiles_m = (q.m + BM - 1) / BM;
    q.tiles_n = (q.n + BN - 1) / BN;
    hipLaunchKernelGGL((product_kernel<DT, LA, LB, E, BM, BN, WM, WN>),
                       dim3(static_cast<unsigned>(q.tiles_m * q.tiles_n), static_cast<unsigned>(slices)),
                       dim3(WM * WN * 64), 0, st, q);
}

int64_t tiles_of(const Product& q, int64_t bm, int64_t bn) { return up(q.m, bm) / bm * (up(q.n, bn) / bn); }

// Returns the wave rows of a tile and their extent in m (for kLse's slots).
template <int DT, Layout LA, Layout LB, Epilogue E>
void launch_product(const Product& q, int slices, hipStream_t st) {
    if (tiles_of(q, 256, 256) * slices >= 192) launch_tiles<DT, LA, LB, E, 256, 256, 2, 4>(q, slices, st);
    else launch_tiles<DT, LA, LB, E, 128, 128, 2, 2>(q, slices, st);
}

// One 16-bit matrix as the products read it: the caller's own rows where
// they are whole 16-byte pieces, else rows repacked into the workspace.
bool whole_pieces(const void* p, int64_t stride, int64_t dim) {
    return aligned16(p) && stride % 8 == 0 && dim % 8 == 0 && stride <= (int64_t(1) << 21);
}
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
        if (tiles_of(q, 256, 256) >= 192) {
            launch_tiles<DT, kRows, kRows, kLse, 256, 256, 2, 4>(q, 1, st);
            slots += static_cast<int>(up(rows, 256) / 256 * 2);
        } else if (a->tokens <= kFewTokens) {
            launch_tiles<DT, kRows, kRows, kLse, 64, 16, 4, 1>(q, 1, st);
            slots += static_cast<int>(up(rows, 64) / 64 * 4);
        } else {
            launch_tiles<DT, kRows, kRows, kLse, 128, 128, 2, 2>(q, 1, st);
            slots += static_cast<int>(up(rows, 128) / 128 * 2);
        }
    }
    hipLaunchKernelGGL(xent_rows_kernel, dim3(static_cast<unsigned>((a->tokens + 15) / 16)), dim3(1024), 0, st,
                       reinterpret_cast<const f32x2*>(partial), slots, static_cast<int>(a->tokens), hit, a->target,
                       a->vocab, a->loss, a->lse);
    return launch_error("loss kernel launch");
}

template <int DT>
int backward(const zero_xent_args* a, const Cut& c, hipStream_t st) {
    char* ws = static_cast<char*>(a->workspace);
    char* xr = ws;
    char* wr = ws + c.x_bytes;
    char* p16 = wr + c.w_bytes;
    float* dx_slab = reinterpret_cast<float*>(p16 + c.p_bytes);
    float* dw_slab = dx_slab + static_cast<int64_t>(c.dx_slices) * a->tokens * c.dim_pad;
    // fp16 holds 2^-24 at best, a probability of a large vocabulary is often
    // less: P is held times 2^15 there (at most 32768, below fp16's 65504)
    const float pscale = DT == ZERO_FP16 ? 32768.0f : 1.0f;
    const float grad = static_cast<float>(a->grad_scale / pscale);
    const Matrix x = prepared(a->x, a->x_stride, 0, a->tokens, a->dim, c.dim_pad, xr, st);
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
        q.target = a->target;
        q.lse = a->lse;
        q.vocab = static_cast<int32_t>(a->vocab);
        q.c = p16;
        q.ldc = c.piece;
        q.scale = pscale;
        launch_product<DT, kRows, kRows, kProb>(q, 1, st);

        // dx += P w: k is the piece's vocabulary
        Product d = {};
        d.a = w.p;
        d.lda = w.stride;
        d.b = p16;
        d.ldb = c.piece * 2;
        d.m = w.dim;
        d.n = q.n;
        d.k = q.m;
        d.slice = static_cast<int32_t>(up(up(d.k, c.dx_slices) / c.dx_slices, kTileK));
        d.c = reinterpret_cast<char*>(dx_slab);
        d.ldc = c.dim_pad;
        d.slab = a->tokens * c.dim_pad;
        d.add = v > 0;
        launch_product<DT, kCols, kRows, kSlab>(d, c.dx_slices, st);

        // dw = P^T x: k is the tokens
        Product e = {};
        e.a = x.p;
        e.lda = x.stride;
        e.b = p16;
        e.ldb = c.piece * 2;
        e.m = x.dim;
        e.n = q.m;
        e.k = q.n;
        unsigned short* dw = static_cast<unsigned short*>(a->dw) + v * a->dw_stride;
        if (c.dw_slices > 1) {
            e.slice = static_cast<int32_t>(up(up(e.k, c.dw_slices) / c.dw_slices, kTileK));
            e.c = reinterpret_cast<char*>(dw_slab);
            e.ldc = c.dim_pad;
            e.slab = c.piece * c.dim_pad;
            launch_product<DT, kCols, kCols, kSlab>(e, c.dw_slices, st);
            hipLaunchKernelGGL((slab_sum_kernel<DT>),
                               dim3(blocks_for(rows * (c.dim_pad / 4))), dim3(256), 0, st,
                               dw_slab, c.dw_slices, e.slab, rows, a->dim, c.dim_pad, a->result, grad, dw,
                               a->dw_stride);
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
                       static_cast<unsigned short*>(a->dx), a->dx_stride);
    return launch_error("loss gradient kernel launch");
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

size_t zero_xent_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab) {
    Cut c;
    return cut(tokens, dim, vocab, &c) ? c.total : 0;
}

int zero_xent_forward(const zero_xent_args* a, void* stream) {
    clear_error();
    int rc = check_xent_args(a, false);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->tokens > 0) {
        Cut c;
        cut(a->tokens, a->dim, a->vocab, &c);
        rc = a->dtype == ZERO_BF16 ? forward<ZERO_BF16>(a, c, st) : forward<ZERO_FP16>(a, c, st);
        if (rc) return rc;
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
    cut(a->tokens, a->dim, a->vocab, &c);
    return a->dtype == ZERO_BF16 ? backward<ZERO_BF16>(a, c, st) : backward<ZERO_FP16>(a, c, st);
}

}  // extern "C"
