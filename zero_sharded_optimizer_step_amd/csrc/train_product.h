// train_product.h -- the tiled matrix product of the training operators, its
// operands' layouts and epilogues, and the choice of the tile.  Not part of
// the public ABI.
//
// An operand lies with its rows along k (x and w in the loss's logits, P in
// its dx) or with k as the row (w in dx; x and P in dw); the second kind is
// turned on the way from LDS to the registers, so nothing is ever transposed
// in memory.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

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
constexpr int kCus = 256, kLdsBytes = 160 << 10;
constexpr uint32_t kNowhere = 0x80000000u;   // past every descriptor: loads 0

enum Layout { kRows, kCols };   // the operand's rows lie along k, or k is the row

// What a product writes.
enum Epilogue {
    kLse,       // partial maxima and sums of exponentials, target logits
    kProb,      // P, 16 bits
    kSlab,      // fp32 partial products of one slice of k
    kGrad,      // the product times a factor, 16 bits
    kPlain,     // the product of all n and k, 16 bits
    kEither,    // that; of more than one slice each one's fp32 part
    // of 8-bit codes: whole sums times both rows' scales, and a bias; of more
    // than one slice each one's whole sums
    kScaledFp16,
    kScaledBf16
};

// Beside ZERO_FP16 and ZERO_BF16: two 8-bit codes in an element of 16 bits, so
// a step is 128 of k and everything else as it is.  Operands are kRows.
constexpr int kCodes = 100;

// C[n][m] = sum_k A(m, k) B(n, k): m is the contiguous axis of the result.
struct Product {
    const char* a;
    const char* b;
    int64_t lda, ldb;         // bytes from row to row
    int32_t m, n, k;          // extents; along a kCols operand's m or n whole 16 bytes are read
    int32_t tiles_m;
    int32_t slices, slice;    // slices of k, and k of one: a multiple of kTileK
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
    const int32_t* kept;      // kProb, kSlab, kGrad: how many tokens there are; n or k is their most
    // kScaled
    const float* scale_m;
    const float* scale_n;
    const unsigned short* bias;   // of m, 16 bits, or NULL
};

// f(0), f(1) .. f(N - 1), each number a constant.
template <int... I, typename F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, const F& f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(const F& f) { each_of(std::make_integer_sequence<int, N>{}, f); }

// Where 16-byte piece c of a tile's row lies: rows-along-k tiles (8 pieces a
// row) swap pieces by the row, so that 16 lanes reading one piece of 16 rows
// meet 16 different 16-byte bank groups; k-as-row tiles swap pairs of pieces
// by k, so that the 4 x 16 blocks of a turning read spread over the banks.
__device__ __forceinline__ int swap_rows(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swap_cols(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }

// c += a b, in place: 64 accumulators fill the accumulation registers, and
// left to the compiler's own allocation they wander through copies.
template <int DT>
__device__ __forceinline__ void mfma(f32x4& c, const s16x8 a, const s16x8 b) {
    if constexpr (DT == ZERO_BF16) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else if constexpr (DT == kCodes) asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// Element e of an accumulator, taken here: the compiler's own copies move all
// 256 at once and spill what stands in their way.
__device__ __forceinline__ float taken(const f32x4& c, int e) {
    float o;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(o) : "a"(c[e]));
    return o;
}
__device__ __forceinline__ f32x4 taken(const f32x4& c) { return f32x4{taken(c, 0), taken(c, 1), taken(c, 2), taken(c, 3)}; }

// One operand's tile of R rows (m or n) by kTileK: this thread's share of
// the loads into LDS, and its fragments out of it.
template <Layout L, int R, int THREADS>
struct Operand {
    static constexpr int kPieces = R * kTileK / 8;          // of 16 bytes
    static_assert(kPieces % THREADS == 0, "every thread loads");
    static constexpr int kLoads = kPieces / THREADS;
    static constexpr int kRowPieces = L == kRows ? kTileK / 8 : R / 8;
    static constexpr int kRowsALoad = THREADS / kRowPieces;
    // a thread's later loads are the same piece of later rows, or in turn two pieces
    static_assert(kLoads == 1 || kRowsALoad % 8 == 0, "swaps repeat every 16 rows");
    static constexpr bool kTwo = L == kCols && kLoads > 1 && kRowsALoad % 16 != 0;
    uint32_t off, off1;       // of the even and the odd loads' piece, or kNowhere
    int32_t along;            // kRows: its first k
    uint32_t next;            // bytes from load to load
    int64_t row;              // bytes of a row
    const char* base;         // the tile's first byte
    int64_t bytes;            // from there to the end of its rows (kRows), of k (kCols)

    // `p`: the operand at this slice's first k and the tile's first row or column r0.
    __device__ __forceinline__ void setup(const char* p, int64_t ld, int rows_left, int r0, int k_lo, int k) {
        const int r = threadIdx.x / kRowPieces, c = threadIdx.x % kRowPieces;
        row = ld;
        next = static_cast<uint32_t>(kRowsALoad * ld);
        base = p;
        if constexpr (L == kRows) {
            const int piece = c ^ swap_rows(r);
            off = static_cast<uint32_t>(r * ld + piece * 16);
            along = piece * 8;
            bytes = rows_left * ld - k_lo * 2;
        } else {
            const int piece = c ^ swap_cols(r);
            off = piece * 8 < rows_left ? static_cast<uint32_t>(r * ld + piece * 16) : kNowhere;
            const int other = c ^ swap_cols(r + kRowsALoad);
            off1 = other * 8 < rows_left ? static_cast<uint32_t>(r * ld + other * 16) : kNowhere;
            bytes = k * ld - r0 * 2;
        }
    }
    // What the loads of one step need.  The descriptor ends with the last row
    // (kRows) or the last k (kCols): rows past it load 0; so does a piece of k
    // past the end.
    struct Step {
        const char* at;
        int bytes;
        uint32_t o, o1;
    };
    __device__ __forceinline__ Step step(int t, int k) const {
        Step s;
        int64_t left = L == kRows ? bytes : bytes - t * (kTileK * row);
        left = left < 0 ? 0 : (left < 0x7ffffff0 ? left : 0x7ffffff0);
        s.at = L == kRows ? base : base + t * (kTileK * row);
        s.bytes = static_cast<int>(left);
        // a tile's 256 rows of at most 4 MB end before kNowhere
        s.o = L == kCols ? off : (along + t * kTileK < k ? off + t * (kTileK * 2) : kNowhere);
        s.o1 = kTwo ? off1 : s.o;
        return s;
    }
    __device__ __forceinline__ void load(const Step& s, ZERO_LDS char* lds, int j) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(s.at), 0, s.bytes, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (ZERO_LDS void*)(lds + (j * THREADS + wave * 64) * 16), 16,
                                                 (j % 2 ? s.o1 : s.o) + j * next, 0, 0, 0);
    }
    // Lane l's 8 values of fragment i of the wave whose rows start at r0, half
    // h of the tile's k, are row r0 + 16 i + l % 16, k = 32 h + 8 (l / 16) +
    // 0..7.  `first` is where those of i = h = 0 lie in the tile.
    __device__ __forceinline__ static uint32_t first(int r0) {
        const int l = threadIdx.x & 63, s = l & 15, g = l >> 4;
        if constexpr (L == kRows) return (r0 + s) * (kTileK * 2) + (g ^ swap_rows(s)) * 16;
        // the 16 lanes of group g give 4 rows of k by 16 of m and get them turned
        const int k = g * 8 + (s >> 2);
        return k * (R * 2) + ((r0 / 16) ^ (swap_cols(k) >> 1)) * 32 + (s & 3) * 8;
    }
    __device__ __forceinline__ static s16x8 fragment(const ZERO_LDS char* lds, uint32_t first, int i, int h) {
        if constexpr (L == kRows) {
            return *(const ZERO_LDS s16x8*)(lds + (first ^ (h * 64)) + i * (16 * kTileK * 2));
        } else {
            const ZERO_LDS char* at = lds + (first ^ (i * 32)) + h * (32 * R * 2);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_LDS s16x4*)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_LDS s16x4*)(at + 4 * R * 2));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kNotKept = INT32_MIN;

// As the instruction has it: a NaN beside a number gives the number.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float o;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(o) : "v"(a), "v"(b), "v"(c));
    return o;
}
// {x of the lane's even row of 16, x of its odd row}, {of the lower half, of the upper}
__device__ __forceinline__ f32x2 other_row(float x) {
    const auto o = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return f32x2{__uint_as_float(o[0]), __uint_as_float(o[1])};
}
__device__ __forceinline__ f32x2 other_half(float x) {
    const auto o = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return f32x2{__uint_as_float(o[0]), __uint_as_float(o[1])};
}
// Is element `at` (16 i + e) among a lane's FM x 4?  And the element itself.
template <int FM>
__device__ __forceinline__ bool here(int at) { return (at & ~((FM - 1) * 16 + 3)) == 0; }
template <int FM>
__device__ __forceinline__ float pick(const f32x4 (&x)[FM], int at) {
    float v[FM];
    const bool b0 = at & 1, b1 = at & 2;
    #pragma unroll
    for (int i = 0; i < FM; ++i) {
        const float lo = b0 ? x[i][1] : x[i][0], hi = b0 ? x[i][3] : x[i][2];
        v[i] = b1 ? hi : lo;
    }
    #pragma unroll
    for (int w = 1; w < FM; w *= 2) {
        const bool b = at & (16 * w);
        #pragma unroll
        for (int i = 0; i < FM; i += 2 * w) v[i] = b ? v[i + w] : v[i];
    }
    return v[0];
}
// Two fragments' values one above the other in m, times f, in 16 bits: a lane
// gives 4 consecutive m of each and gets 8 of one, for 16-byte stores.
template <int DT>
__device__ __forceinline__ u32x4 pair(const f32x4 a, const f32x4 b, float f) {
    const auto lo = __builtin_amdgcn_permlane16_swap(pack2<DT>(a[0] * f, a[1] * f), pack2<DT>(b[0] * f, b[1] * f),
                                                     false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(pack2<DT>(a[2] * f, a[3] * f), pack2<DT>(b[2] * f, b[3] * f),
                                                     false, false);
    return u32x4{lo[0], hi[0], lo[1], hi[1]};
}
__device__ __forceinline__ bool infinite(float x) { return __builtin_fabsf(x) == __builtin_inff(); }

// The product's tile by tile.  What bounds a large one is the matrix cores'
// power: at 4096 tokens x 4096 x 128000 in bf16 the clock falls to 1.85 GHz,
// and the forward takes 2.87 to 3.0 ms (1.43 to 1.5 PFLOP/s) with values of a
// normal distribution and 2.51 ms with zeros.  Hence
//   - four waves with 128 x 128 of a 256 x 256 tile each, one a SIMD, so that
//     a value out of LDS serves 8 products of 16 x 16 x 32 (eight waves of
//     128 x 64 read half as much again: 3.35 ms with all of the below lacking);
//   - the accumulators in the 256 accumulation registers, both halves'
//     fragments in the others, every product with at most one other
//     instruction behind it (in clumps of eight: 3.40 ms);
//   - five slots of LDS for the operands' steps of 64 k, so a step's loads
//     have one to three halves of a step to arrive and no wait drains them;
//   - blocks that stay: a tile's first loads run under the epilogue of the
//     tile before (as separate blocks, and with an epilogue that spilled
//     registers: 3.10 ms).
// s0 to s4 are the five slots; the caller's, so that one kernel may hold two
// products.  This block is `block` of `grid`.
template <int BM, int BN>
constexpr int kProductSlot = (BM > BN ? BM : BN) * kTileK * 2;
template <int DT, Layout LA, Layout LB, Epilogue E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void product(const Product& q, int block, int grid, char* s0, char* s1, char* s2, char* s3,
                                        char* s4) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;     // fragments of a wave
    static_assert(FM % 2 == 0 && FN >= 4, "the epilogues' pairs and shares");
    typedef Operand<LA, BM, kThreads> OpA;
    typedef Operand<LB, BN, kThreads> OpB;

    // The grid is what the chip holds at once; a block walks the tiles of all
    // slices.
    constexpr bool kTokensAreK = LB == kCols && (E == kSlab || E == kGrad);
    constexpr bool kTokensAreN = E == kProb || (E == kSlab && !kTokensAreK);
    constexpr bool kScaled = E == kScaledFp16 || E == kScaledBf16;
    constexpr int OT = E == kScaledFp16 ? ZERO_FP16 : (E == kScaledBf16 ? ZERO_BF16 : DT);   // of a 16-bit result
    static_assert(kScaled == (DT == kCodes), "codes have whole sums");
    const int size_n = kTokensAreN ? *q.kept : q.n, size_k = kTokensAreK ? *q.kept : q.k;
    const int tiles_n = (size_n + BN - 1) / BN;
    const int tiles = q.tiles_m * tiles_n, total = tiles * q.slices;
    if (block >= total) return;
    struct Place {
        int tm, m0, n0, slice, k_lo, k;                    // k: this slice's
    };
    auto place = [&](int id) -> Place {
        Place w;
        w.slice = id / tiles;
        id -= w.slice * tiles;
        // Each XCD takes a contiguous run of tiles, ordered in strips of 4 along
        // n, so the tiles its 32 CUs hold at a time share rows of both operands.
        const int per = tiles / kXcds, extra = tiles % kXcds;
        const int x = id % kXcds, i = id / kXcds;
        id = x * per + (x < extra ? x : extra) + i;
        constexpr int kStrip = 4;
        const int strip = id / (kStrip * q.tiles_m);
        const int width = tiles_n - strip * kStrip < kStrip ? tiles_n - strip * kStrip : kStrip;
        const int in_strip = id - strip * kStrip * q.tiles_m;
        w.tm = in_strip / width;
        w.m0 = w.tm * BM;
        w.n0 = (strip * kStrip + in_strip % width) * BN;
        w.k_lo = w.slice * q.slice;
        w.k = (size_k < w.k_lo + q.slice ? size_k : w.k_lo + q.slice) - w.k_lo;
        w.k = w.k > 0 ? w.k : 0;
        return w;
    };

    const int lane = threadIdx.x & 63, nl = lane & 15, ml = (lane >> 4) * 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);

    OpA oa;
    OpB ob;
    Place w;
    auto load = [&](const auto& op, int t, char* to) -> void {
        const auto st = op.step(t, w.k);
        #pragma unroll
        for (int j = 0; j < std::decay_t<decltype(op)>::kLoads; ++j) op.load(st, (ZERO_LDS char*)to, j);
    };
    // Share g of 4 of the loads of the first two steps; step 1's a comes last.
    auto first_loads = [&](int g) -> void {
        if (g == 0) load(oa, 0, s0);
        else if (g == 1) load(ob, 0, s1);
        else if (g == 2) load(ob, 1, s3);
        else load(oa, 1, s2);
    };
    auto begin = [&](int id) -> void {
        w = place(id);
        oa.setup(q.a + (LA == kRows ? w.m0 * q.lda + w.k_lo * 2 : w.k_lo * q.lda + w.m0 * 2), q.lda, q.m - w.m0,
                 w.m0, w.k_lo, w.k);
        ob.setup(q.b + (LB == kRows ? w.n0 * q.ldb + w.k_lo * 2 : w.k_lo * q.ldb + w.n0 * 2), q.ldb, size_n - w.n0,
                 w.n0, w.k_lo, w.k);
    };
    // of the 8 consecutive m that a lane holds after pair()
    [[maybe_unused]] const int pair_m = ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
    f32x4 acc[FM][FN];

    struct Frags {
        s16x8 a[FM], b[FN];
    };
    const uint32_t at_a = OpA::first(wm), at_b = OpB::first(wn);
    auto read = [&](Frags& f, const char* sha, const char* shb, uint32_t fa, uint32_t fb, int h, int r) {
        if (r < FN) f.b[r] = OpB::fragment((const ZERO_LDS char*)shb, fb, r, h);
        else f.a[r - FN] = OpA::fragment((const ZERO_LDS char*)sha, fa, r - FN, h);
    };
    // The products of one half of a step's k.  With one wave a SIMD the matrix
    // core idles wherever two other instructions stand in a row, so the reads
    // of the next half's fragments and the loads of a later step go one by one
    // between them, over the first half of them: the last have arrived when
    // the next half begins (forward of 4096 x 4096 x 128000 over the first
    // half 3.04 ms, three quarters 3.07, all 3.15).
    auto half = [&](const Frags& use, Frags& fill, const char* sha, const char* shb, int h, const auto& op, int t,
                    char* to) __attribute__((always_inline)) -> void {
        constexpr int kItems = FM + FN + std::decay_t<decltype(op)>::kLoads;
        constexpr int kLoads = std::decay_t<decltype(op)>::kLoads;
        constexpr int kSpan = FM * FN / 2;
        // hidden, or every address of every slot takes a register of its own
        uint32_t fa = at_a, fb = at_b;
        asm volatile("" : "+v"(fa), "+v"(fb));
        const auto st = op.step(t, w.k);
        each<FM * FN>([&](auto slot) __attribute__((always_inline)) -> void {
            constexpr int s = decltype(slot)::value;
            __builtin_amdgcn_sched_barrier(0);
            mfma<DT>(acc[s / FN][s % FN], use.a[s / FN], use.b[s % FN]);
            constexpr int from = s < kSpan ? s * kItems / kSpan : kItems;
            constexpr int to_x = s < kSpan ? (s + 1) * kItems / kSpan : kItems;
            each<to_x - from>([&](auto item) __attribute__((always_inline)) -> void {
                constexpr int x = from + decltype(item)::value, l = x * kLoads / kItems;
                if constexpr ((x + 1) * kLoads / kItems > l) op.load(st, (ZERO_LDS char*)to, l);
                else read(fill, sha, shb, fa, fb, h, x - l);
            });
        });
        __builtin_amdgcn_sched_barrier(0);
    };
    Frags f0, f1;
    // Step t lies in slots a and b, step t + 1 in a1 and b1.  Slot a2 was
    // step t - 1's b: every wave's reads of it ended before the turn of step
    // t - 1.  The reads of a end before the turn here, after which it takes
    // step t + 2's b.
    auto step = [&](int t, char* a, char* b, char* a1, char* b1, char* a2) __attribute__((always_inline)) {
        half(f0, f1, a, b, 1, oa, t + 2, a2);
        // all but the loads of a2 have arrived, in every wave
        __builtin_amdgcn_s_waitcnt(0x0070 | OpA::kLoads);
        __builtin_amdgcn_s_barrier();
        half(f1, f0, a1, b1, 0, ob, t + 2, a);
    };
    static_assert(OpA::kLoads < 16, "the wait's low bits");
    // acc[i][j][e] is C at n = n0 + wn + 16 j + lane % 16,
    // m = m0 + wm + 16 i + 4 (lane / 16) + e
    // The epilogues' code is kept short: it runs once a tile, and straight-line
    // code past the instruction cache costs more to fetch than to run.
    auto epilogue = [&](int tm, int m0, int n0, int slice, const int64_t (&target)[FN], const float (&lse)[FN],
                        const f32x4 (&by)[FM], bool more) __attribute__((always_inline)) -> void {
        // the next tile's first loads, a share with each of the first four columns
        auto columns = [&](auto column) __attribute__((always_inline)) -> void {
            each<FN>([&](auto index) __attribute__((always_inline)) -> void {
                constexpr int j = decltype(index)::value;
                __builtin_amdgcn_sched_barrier(0);
                if (more) {
                    each<4>([&](auto share) __attribute__((always_inline)) -> void {
                        constexpr int g = decltype(share)::value;
                        if constexpr (g == j) first_loads(g);
                    });
                }
                column(index);
            });
        };
        [[maybe_unused]] const int end = q.m - (m0 + wm + ml);   // the lane's elements 16 i + e below it exist
        // the target's place from this lane's first m on
        [[maybe_unused]] int at[FN];
        if constexpr (E == kLse || E == kProb) {
            #pragma unroll
            for (int j = 0; j < FN; ++j)
                at[j] = target[j] >= 0 && target[j] < q.vocab
                            ? static_cast<int>(target[j]) - q.first_m - (m0 + wm + ml) : kNotKept;
        }
        [[maybe_unused]] auto split = [&](auto column) __attribute__((always_inline)) -> void {
            if (m0 + BM > q.m)
                columns([&](auto index) __attribute__((always_inline)) -> void { column(std::true_type{}, index); });
            else
                columns([&](auto index) __attribute__((always_inline)) -> void { column(std::false_type{}, index); });
        };
        // kLse, kProb: an element, -inf beyond the last m where a tile has such
        auto logit = [&](auto edge, int i, int j, int e) __attribute__((always_inline)) -> float {
            const float x = taken(acc[i][j], e);
            return !decltype(edge)::value || i * 16 + e < end ? x : -__builtin_inff();
        };
        if constexpr (E == kLse) {
            const int slot = q.slot0 + tm * WM + wave % WM;
            auto column = [&](auto edge, auto index) __attribute__((always_inline)) -> void {
                constexpr int j = decltype(index)::value;
                const int n = n0 + wn + j * 16 + nl;
                f32x4 x[FM];
                #pragma unroll
                for (int i = 0; i < FM; ++i)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) x[i][e] = logit(edge, i, j, e);
                float top = max3(x[0][0], x[0][1], max3(x[0][2], x[0][3], x[0][3]));
                #pragma unroll
                for (int i = 1; i < FM; ++i) top = max3(x[i][0], x[i][1], max3(x[i][2], x[i][3], top));
                top = fmaxf(other_row(top).x, other_row(top).y);
                top = fmaxf(other_half(top).x, other_half(top).y);
                const bool hit = n < size_n && here<FM>(at[j]);
                if (__builtin_amdgcn_ballot_w64(hit) != 0) {
                    const float v = pick(x, at[j]);
                    if (hit) q.target_logit[n] = v;
                }
                // exp(x - top) as 2^(x log2 e - c) 2^(c - top log2 e): the second
                // factor is c's rounding, between 2^-1/16 and 2^1/16 up to kFar.
                // Beyond it the factors would leave fp32's range (0 times inf),
                // past 2.36e38 c itself: there top is subtracted first.
                float base = infinite(top) ? 0.0f : top;
                constexpr float kFar = 1 << 20;
                if (__builtin_amdgcn_ballot_w64(__builtin_fabsf(base) > kFar) != 0) {
                    #pragma unroll
                    for (int i = 0; i < FM; ++i)
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) x[i][e] -= base;
                    base = 0.0f;
                }
                const float c = base * kLog2e, rest = __builtin_fmaf(base, -kLog2e, c);
                f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f}, y[FM];
                #pragma unroll
                for (int i = 0; i <= FM; ++i) {
                    // a row's sums go with the next row's exponentials
                    __builtin_amdgcn_sched_barrier(0);
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (i < FM) y[i][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i][e], kLog2e, -c));
                        if (i > 0) part[e] += y[i - 1][e];
                    }
                }
                float sum = ((part[0] + part[1]) + (part[2] + part[3])) * __builtin_amdgcn_exp2f(rest);
                sum = other_row(sum).x + other_row(sum).y;
                sum = other_half(sum).x + other_half(sum).y;
                if (n < size_n && lane < 16)
                    reinterpret_cast<f32x2*>(q.partial)[static_cast<int64_t>(slot) * size_n + n] = f32x2{top, sum};
            };
            split(column);
        } else if constexpr (E == kProb) {
            // In 16 bits, as the matrix cores of the two products take it: half
            // a step each, independent, beside the half step that dx and dw are
            // rounded by at the end.  Errors of the gradients against 64 bits
            // (relative, all of them): bf16, 4096 x 4096 x 128000 1.7e-3, with P
            // in fp32 1.7e-3; fp16, 509 x 1000 x 10007 2.2e-4 and 2.1e-4.
            const float bias = q.scale > 1.0f ? 15.0f : 0.0f;      // log2 of the scale
            auto column = [&](auto edge, auto index) __attribute__((always_inline)) -> void {
                constexpr int j = decltype(index)::value;
                const int n = n0 + wn + j * 16 + nl;
                f32x4 p[FM];
                #pragma unroll
                for (int i = 0; i < FM; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    #pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[i][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(logit(edge, i, j, e) - lse[j], kLog2e, bias));
                }
                const bool kept = at[j] != kNotKept, hit = n < size_n && here<FM>(at[j]);
                if (__builtin_amdgcn_ballot_w64(hit) != 0) {
                    #pragma unroll
                    for (int i = 0; i < FM; ++i)
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) p[i][e] -= at[j] == i * 16 + e ? q.scale : 0.0f;
                }
                unsigned short* row = reinterpret_cast<unsigned short*>(q.c) + n * q.ldc + m0 + wm;
                #pragma unroll
                for (int i = 0; i < FM; i += 2) {
                    const u32x4 o = pair<DT>(p[i], p[i + 1], 1.0f);
                    if (n < size_n) *reinterpret_cast<u32x4*>(row + i * 16 + pair_m) = kept ? o : u32x4{0u, 0u, 0u, 0u};
                }
            };
            split(column);
        } else if (E == kSlab || ((E == kEither || kScaled) && q.slices > 1)) {
            float* c = reinterpret_cast<float*>(q.c) + static_cast<int64_t>(slice) * q.slab;
            columns([&](auto index) __attribute__((always_inline)) -> void {
                constexpr int j = decltype(index)::value;
                const int n = n0 + wn + j * 16 + nl;
                f32x4* row = reinterpret_cast<f32x4*>(c + n * q.ldc + m0 + wm + ml);
                f32x4 y[FM];
                #pragma unroll
                for (int i = 0; i < FM; ++i) {
                    y[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    // q.m and ldc are whole quads
                    if (E == kSlab && q.add && n < size_n && i * 16 < end) y[i] = row[i * 4];
                }
                #pragma unroll
                for (int i = 0; i < FM; ++i) {
                    f32x4 x = taken(acc[i][j]);
                    if constexpr (E == kSlab) {
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = y[i][e] + x[e];
                    }
                    if (n < size_n && i * 16 < end) row[i * 4] = x;
                }
            });
        } else if constexpr (E != kSlab) {
            float f = 1.0f;
            if constexpr (E == kGrad) f = q.scale * q.result->inv_count;
            typedef u32x4 eight __attribute__((aligned(2)));
            // 16 rows of a wave's m, each 16 bytes longer, so that a column of them meets all banks
            constexpr int kRoomRow = FM * 32 + 16, kRoomLanes = FM * 2;
            static_assert(16 * kRoomRow * WM * WN <= kProductSlot<BM, BN>, "a slot holds the waves' rows");
            ZERO_LDS char* room = (ZERO_LDS char*)s4 + wave * 16 * kRoomRow;
            // of the lane's m; past the last m the descriptor gives 0
            [[maybe_unused]] f32x4 plus[FM];
            if constexpr (kScaled) {
                const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
                    const_cast<unsigned short*>(q.bias), 0, q.m * 2, 0x00020000);
                #pragma unroll
                for (int i = 0; i < FM; ++i) {
                    plus[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    if (q.bias) {
                        #pragma unroll
                        for (int e = 0; e < 4; ++e)
                            plus[i][e] = lo_to_f32<OT>(
                                __builtin_amdgcn_raw_buffer_load_b16(rb, (m0 + wm + i * 16 + ml + e) * 2, 0, 0));
                    }
                }
            }
            columns([&](auto index) __attribute__((always_inline)) -> void {
                constexpr int j = decltype(index)::value;
                // an accumulator as it is written; a whole sum is rounded to fp32 first
                auto result = [&](int i) __attribute__((always_inline)) -> f32x4 {
                    f32x4 x = taken(acc[i][j]);
                    if constexpr (kScaled) {
                        #pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = __builtin_fmaf(static_cast<float>(__float_as_int(x[e])) * lse[j], by[i][e], plus[i][e]);
                    }
                    return x;
                };
                // A lane has 4 of m in 16 rows of m apart; stored so, every lane is an
                // address of its own.  Turned by way of the free slot, 16 bytes a lane
                // lie one behind the other along a row.
                #pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const f32x4 x = result(i);
                    *(ZERO_LDS u32x2*)(room + nl * kRoomRow + i * 32 + ml * 2) =
                        u32x2{pack2<OT>(x[0] * f, x[1] * f), pack2<OT>(x[2] * f, x[3] * f)};
                }
                #pragma unroll
                for (int r = lane / kRoomLanes; r < 16; r += 64 / kRoomLanes) {
                    const u32x4 o = *(const ZERO_LDS u32x4*)(room + r * kRoomRow + lane % kRoomLanes * 16);
                    const int n = n0 + wn + j * 16 + r, m = m0 + wm + lane % kRoomLanes * 8;
                    unsigned short* row = reinterpret_cast<unsigned short*>(q.c) + n * q.ldc;
                    if (n >= size_n || m >= q.valid_m) continue;
                    if (m + 8 <= q.valid_m) {
                        *reinterpret_cast<eight*>(row + m) = o;
                    } else {
                        #pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (m + e < q.valid_m) row[m + e] = static_cast<unsigned short>(o[e / 2] >> (16 * (e % 2)));
                    }
                }
            });
        }
    };

    begin(block);
    #pragma unroll
    for (int g = 0; g < 4; ++g) first_loads(g);
    for (int id = block;;) {
        #pragma unroll
        for (int i = 0; i < FM; ++i)
            #pragma unroll
            for (int j = 0; j < FN; ++j) {
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                asm volatile("" : "+a"(acc[i][j]));        // written here, well before the first product
            }
        // The loads of step 1's a, which came last, may still be under way (so
        // may stores of the last tile's epilogue, which came after them).
        __builtin_amdgcn_s_waitcnt(0x0070 | OpA::kLoads);
        __builtin_amdgcn_s_barrier();
        // what the epilogue needs of each token is here long before it
        [[maybe_unused]] int64_t target[FN];
        [[maybe_unused]] float lse[FN];
        if constexpr (E == kLse || E == kProb || kScaled) {
            #pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n = w.n0 + wn + j * 16 + nl;
                if constexpr (!kScaled) target[j] = q.target[n < size_n ? n : size_n - 1];
                if constexpr (E == kProb) lse[j] = q.lse[n < size_n ? n : size_n - 1];
                if constexpr (kScaled) lse[j] = q.scale_n[n < size_n ? n : size_n - 1];   // the row's scale
            }
        }
        [[maybe_unused]] f32x4 by[FM];                     // the scales of the lane's m
        if constexpr (kScaled) {
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<float*>(q.scale_m), 0, q.m * 4, 0x00020000);
            #pragma unroll
            for (int i = 0; i < FM; ++i)
                by[i] = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (w.m0 + wm + i * 16 + ml) * 4, 0, 0));
        }
        #pragma unroll
        for (int x = 0; x < FM + FN; ++x) read(f0, s0, s1, at_a, at_b, 0, x);
        const int steps = (w.k + kTileK - 1) / kTileK;
        for (int t = 0; t < steps; t += 5) {
            step(t, s0, s1, s2, s3, s4);
            if (t + 1 < steps) step(t + 1, s2, s3, s4, s0, s1);
            if (t + 2 < steps) step(t + 2, s4, s0, s1, s2, s3);
            if (t + 3 < steps) step(t + 3, s1, s2, s3, s4, s0);
            if (t + 4 < steps) step(t + 4, s3, s4, s0, s1, s2);
        }
        __builtin_amdgcn_s_waitcnt(0x0070);                // no load outlives the tile
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 15\n\ts_nop 15");              // the last products' results, which the compiler does not time
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        const int tm = w.tm, m0 = w.m0, n0 = w.n0, slice = w.slice;
        id += grid;
        if (id < total) begin(id);
        epilogue(tm, m0, n0, slice, target, lse, by, id < total);
        if (id >= total) break;
    }
}

template <int DT, Layout LA, Layout LB, Epilogue E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void product_kernel(const Product q) {
    constexpr int kSlot = kProductSlot<BM, BN>;
    __shared__ __attribute__((aligned(1024))) char s0[kSlot];
    __shared__ __attribute__((aligned(1024))) char s1[kSlot];
    __shared__ __attribute__((aligned(1024))) char s2[kSlot];
    __shared__ __attribute__((aligned(1024))) char s3[kSlot];
    __shared__ __attribute__((aligned(1024))) char s4[kSlot];
    product<DT, LA, LB, E, BM, BN, WM, WN>(q, blockIdx.x, gridDim.x, s0, s1, s2, s3, s4);
}

// Two products that share B's rows' memory but not the way it is read, as one
// grid: the first `first` blocks walk one's tiles, the others the other's.
template <int DT, Epilogue E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void two_products_kernel(const Product qa, const Product qb, int first) {
    constexpr int kSlot = kProductSlot<BM, BN>;
    __shared__ __attribute__((aligned(1024))) char s0[kSlot];
    __shared__ __attribute__((aligned(1024))) char s1[kSlot];
    __shared__ __attribute__((aligned(1024))) char s2[kSlot];
    __shared__ __attribute__((aligned(1024))) char s3[kSlot];
    __shared__ __attribute__((aligned(1024))) char s4[kSlot];
    const int block = blockIdx.x;
    if (block < first) product<DT, kCols, kRows, E, BM, BN, WM, WN>(qa, block, first, s0, s1, s2, s3, s4);
    else product<DT, kCols, kCols, E, BM, BN, WM, WN>(qb, block - first, gridDim.x - first, s0, s1, s2, s3, s4);
}

int launch_error(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(ZERO_EDEVICE, "%s: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

constexpr int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

template <int DT, Layout LA, Layout LB, Epilogue E, int BM, int BN, int WM, int WN>
void launch_tiles(Product q, int slices, hipStream_t st) {
    q.tiles_m = (q.m + BM - 1) / BM;
    q.slices = slices;
    // as many blocks as the CUs' LDS holds at once
    constexpr int kBlocks = kCus * (kLdsBytes / (5 * (BM > BN ? BM : BN) * kTileK * 2));
    const int total = q.tiles_m * ((q.n + BN - 1) / BN) * slices;
    hipLaunchKernelGGL((product_kernel<DT, LA, LB, E, BM, BN, WM, WN>),
                       dim3(static_cast<unsigned>(total < kBlocks ? total : kBlocks)), dim3(WM * WN * 64), 0, st, q);
}

int64_t tiles_of(const Product& q, int64_t bm, int64_t bn) { return up(q.m, bm) / bm * (up(q.n, bn) / bn); }

// 256 x 256 or 128 x 128: by how often each fills the chip, the larger one
// block a CU, the smaller two.  Microseconds for 128 x 128 and 256 x 256, bf16:
//   - of 1024 of k or more a round of the larger takes 1.6 times one of the
//     smaller, and a round takes its time however few blocks are in it.
//     Forward of 2048 tokens x 4096: 4096 of the vocabulary (128 large tiles)
//     68 and 87, 5120 (160) 103 and 86, 8192 (256) 124 and 103, 8448 (264) 153
//     and 174, 16384 (512) 238 and 196;
//   - of less, 1.8 times, and the smaller's last round takes its share only:
//     a block alone on its CU is the faster, and so it is with few steps
//     between a tile's start and its epilogue.  Forward of 2048 x 256 x 6016
//     12.8 and 17.1, 4096 x 512 x 10007 45 and 53, x 32000 150 and 134; dw of
//     509 tokens x 1000 x 10007 18.6 and 20.6, x 16384 23.2 and 22.7.
// Against the better of the two each time, over 64 to 4096 of k, this loses
// 0.4 % on average (648 forwards and Ps, 270 dws, the worst 25 %: 14.0 us for
// 11.2); the first half alone would lose 1.6 %.
bool large_tiles(const Product& q, int slices) {
    const int64_t small = tiles_of(q, 128, 128) * slices;
    const int64_t large = (tiles_of(q, 256, 256) * slices + kCus - 1) / kCus;
    if (q.slice < 1024) return 9 * large * (2 * kCus) <= 5 * small;
    return 8 * large <= 5 * ((small + 2 * kCus - 1) / (2 * kCus));
}

template <int DT, Layout LA, Layout LB, Epilogue E>
void launch_product(const Product& q, int slices, hipStream_t st) {
    if (large_tiles(q, slices)) launch_tiles<DT, LA, LB, E, 256, 256, 2, 2>(q, slices, st);
    else launch_tiles<DT, LA, LB, E, 128, 128, 2, 2>(q, slices, st);
}

// Rows that the products read where they lie: whole 16-byte pieces.  Others
// are copied first.
bool whole_pieces(const void* p, int64_t stride, int64_t dim) {
    return aligned16(p) && stride % 8 == 0 && dim % 8 == 0 && stride <= (int64_t(1) << 21);
}

}  // namespace
}  // namespace zero
