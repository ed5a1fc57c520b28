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
    kGrad       // the product times a factor, 16 bits
};

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
    const int32_t* kept;      // the backward: how many tokens there are; n or k is their most
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
template <int DT, Layout LA, Layout LB, Epilogue E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void product_kernel(const Product q) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;     // fragments of a wave
    static_assert(FM % 2 == 0 && FN >= 4, "the epilogues' pairs and shares");
    typedef Operand<LA, BM, kThreads> OpA;
    typedef Operand<LB, BN, kThreads> OpB;
    constexpr int kSlot = (BM > BN ? BM : BN) * kTileK * 2;
    __shared__ __attribute__((aligned(1024))) char s0[kSlot];
    __shared__ __attribute__((aligned(1024))) char s1[kSlot];
    __shared__ __attribute__((aligned(1024))) char s2[kSlot];
    __shared__ __attribute__((aligned(1024))) char s3[kSlot];
    __shared__ __attribute__((aligned(1024))) char s4[kSlot];

    // The grid is what the chip holds at once; a block walks the tiles of all
    // slices.
    constexpr bool kTokensAreK = LB == kCols, kTokensAreN = E == kProb || (E == kSlab && !kTokensAreK);
    const int size_n = kTokensAreN ? *q.kept : q.n, size_k = kTokensAreK ? *q.kept : q.k;
    const int tiles_n = (size_n + BN - 1) / BN;
    const int tiles = q.tiles_m * tiles_n, total = tiles * q.slices;
    if (static_cast<int>(blockIdx.x) >= total) return;
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
                        bool more) __attribute__((always_inline)) -> void {
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
        } else if constexpr (E == kSlab) {
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
                    if (q.add && n < size_n && i * 16 < end) y[i] = row[i * 4];
                }
                #pragma unroll
                for (int i = 0; i < FM; ++i) {
                    f32x4 x = taken(acc[i][j]);
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = y[i][e] + x[e];
                    if (n < size_n && i * 16 < end) row[i * 4] = x;
                }
            });
        } else {
            const float f = q.scale * q.result->inv_count;
            typedef u32x4 eight __attribute__((aligned(2)));
            columns([&](auto index) __attribute__((always_inline)) -> void {
                constexpr int j = decltype(index)::value;
                const int n = n0 + wn + j * 16 + nl;
                unsigned short* row = reinterpret_cast<unsigned short*>(q.c) + n * q.ldc;
                #pragma unroll
                for (int i = 0; i < FM; i += 2) {
                    const u32x4 o = pair<DT>(taken(acc[i][j]), taken(acc[i + 1][j]), f);
                    const int m = m0 + wm + i * 16 + pair_m;
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

    begin(blockIdx.x);
    #pragma unroll
    for (int g = 0; g < 4; ++g) first_loads(g);
    for (int id = blockIdx.x;;) {
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
        if constexpr (E == kLse || E == kProb) {
            #pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n = w.n0 + wn + j * 16 + nl;
                target[j] = q.target[n < size_n ? n : size_n - 1];
                if constexpr (E == kProb) lse[j] = q.lse[n < size_n ? n : size_n - 1];
            }
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
        id += gridDim.x;
        if (id < total) begin(id);
        epilogue(tm, m0, n0, slice, target, lse, id < total);
        if (id >= total) break;
    }
}

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

// Elements [d, d + 8) of a row of any alignment, zeros past dim.
__device__ __forceinline__ u32x4 row_piece(const unsigned short* __restrict__ s, int64_t d, int64_t dim) {
    typedef u32x4 piece __attribute__((aligned(2)));
    if (d + 8 <= dim) return *reinterpret_cast<const piece*>(s + d);
    unsigned w[4] = {0u, 0u, 0u, 0u};
    #pragma unroll
    for (int e = 0; e < 8; ++e)
        if (d + e < dim) w[e / 2] |= static_cast<unsigned>(s[d + e]) << (16 * (e % 2));
    return u32x4{w[0], w[1], w[2], w[3]};
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
int launch_error(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(ZERO_EDEVICE, "%s: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

constexpr int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

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
}  // namespace zero

using namespace zero;

extern "C" {

size_t zero_xent_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab) {
    // room for either layout of w
    Cut whole, packed;
    if (!cut(tokens, dim, vocab, false, &whole) || !cut(tokens, dim, vocab, true, &packed)) return 0;
    return dim % 8 == 0 && whole.total > packed.total ? whole.total : packed.total;
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
