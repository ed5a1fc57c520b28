// train_linear8.hip -- the product of 8-bit rows with 8-bit weights and its
// gradient (include/zero/train.h).
//
//   forward    y = x8 w8^T in whole numbers on the matrix cores, scaled and
//              rounded once in the epilogue: by the tiles that the loss uses
//              (8192 x 4096 x 16384 in 422 us, 2.6 POP/s, bound by the matrix
//              cores' power), where they are few in slices of k; few tokens
//              by a kernel whose waves need no barrier between their loads.
//   backward   x^ and w^ are written out in 16 bits (exact with the encoder's
//              scales), as many columns of dim at a time as 512 MB hold; then
//              dx = dy w^ and dw = dy^T x^.  Small results are cut along
//              their sum into slices, joined in a fixed order.  Up to 64
//              tokens one pass over w8's rows makes dw's beside dx's sums,
//              with no copy in 16 bits.
#include "train_product.h"

namespace zero {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Few {
    const char* w;
    const char* x;
    int64_t ldw, ldx;         // bytes
    int32_t out, tokens, k;   // k: bytes of a row, a multiple of 16
    const float *w_scale, *x_scale;
    const unsigned short* bias;
    unsigned short* y;
    int64_t ldy;              // elements
};

// Few tokens: w8 is read once and nothing else counts.  A block takes 16 rows
// of w8 at a time, `groups` times, and 16 NF tokens; its four waves take every
// fourth 128 of k, each on its own, and their sums, whole numbers, meet in
// LDS.  The loads of the next rows are under way meanwhile.  They go to LDS
// with 8 lanes along a row: as fragments straight into registers, a row to a
// lane, every lane is an address of its own, and the 16 bytes a cycle and CU
// that this gives bound the kernel: 1 token x 4096 x 16384 took 15.7 us and 64
// 46, now 11.6 (5.8 TB/s) and 23 to 28.  Blocks begin at unlike k, or all of
// them would meet in the same channels of memory (1 token 17.4 and 15.7 then).
constexpr int kFewWaves = 4, kMostGroups = 16;
template <int OT, int NF>
__global__ __launch_bounds__(kFewWaves * 64) void few8_kernel(const Few q) {
    constexpr int W = kFewWaves, kRowsBytes = 16 * 128, kSlot = (1 + NF) * kRowsBytes, kLoads = 2 * (1 + NF);
    __shared__ __attribute__((aligned(1024))) char s0[W][kSlot];
    __shared__ __attribute__((aligned(1024))) char s1[W][kSlot];
    __shared__ __attribute__((aligned(1024))) char s2[W][kSlot];
    __shared__ i32x4 s_sum[2][W][NF][64];
    __shared__ f32x4 s_scale[kMostGroups][4], s_bias[kMostGroups][4];
    const int lane = threadIdx.x & 63, s = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int n0 = blockIdx.y * (16 * NF);
    const int step_m = gridDim.x * 16;                     // from group to group
    const int groups = (q.out - static_cast<int>(blockIdx.x) * 16 + step_m - 1) / step_m;
    // a thread has an output channel of each group
    {
        const int i = threadIdx.x / 16, m = blockIdx.x * 16 + i * step_m + threadIdx.x % 16;
        if (i < groups) {
            const int at = m < q.out ? m : q.out - 1;
            s_scale[i][s / 4][s % 4] = q.w_scale[at];
            s_bias[i][s / 4][s % 4] = q.bias ? lo_to_f32<OT>(q.bias[at]) : 0.0f;
        }
    }
    // a wave finishes 16 tokens
    const int n = n0 + wave * 16 + s;
    const bool mine = wave < NF && n < q.tokens;
    const float sx = mine ? q.x_scale[n] : 0.0f;
    __syncthreads();
    auto records = [](int64_t bytes) { return static_cast<int>(bytes < 0x7ffffff0 ? bytes : 0x7ffffff0); };
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(q.x + n0 * q.ldx), 0, records((q.tokens - n0) * q.ldx), 0x00020000);
    const int blocks = q.k > 0 ? (q.k + 127) / 128 : 1;    // of 128 of k
    const int mine_k = (blocks + W - 1) / W;               // steps of a group
    const int turn = static_cast<int>(static_cast<unsigned>(blockIdx.x / kXcds * W) % static_cast<unsigned>(blocks));
    // Row r's piece c of 16 bytes lies where piece c ^ swap_rows(r) would: a
    // load's 8 rows below the first 8 have bit 2 of it the other way.
    const int row = lane / 8, piece = (lane % 8) ^ swap_rows(row);
    const uint32_t oa = static_cast<uint32_t>(row * q.ldw), ob = static_cast<uint32_t>(row * q.ldx);
    // the next step's loads: two of 8 rows for each 16; past the last group all give 0
    int load_m = blockIdx.x * 16, load_i = wave;
    auto load = [&](char* slot) __attribute__((always_inline)) -> void {
        const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(q.w + load_m * q.ldw), 0, load_m < q.out ? records((q.out - load_m) * q.ldw) : 0, 0x00020000);
        const int block = load_i + turn < blocks ? load_i + turn : load_i + turn - blocks;
        #pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int k = block * 128 + (piece ^ (p * 4)) * 16;
            const bool in = load_i < blocks && k < q.k;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZERO_LDS void*)(slot + p * 1024), 16,
                                                     in ? oa + p * 8 * static_cast<uint32_t>(q.ldw) + k : kNowhere, 0, 0, 0);
            #pragma unroll
            for (int j = 0; j < NF; ++j)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rb, (ZERO_LDS void*)(slot + (1 + j) * kRowsBytes + p * 1024), 16,
                    in ? ob + (j * 16 + p * 8) * static_cast<uint32_t>(q.ldx) + k : kNowhere, 0, 0, 0);
        }
        load_i += W;
        if (load_i >= mine_k * W) {
            load_i = wave;
            load_m += step_m;
        }
    };
    i32x4 acc[NF] = {};
    const uint32_t at = s * 128 + (g ^ swap_rows(s)) * 16;
    int group = 0, done = 0;
    auto finish = [&]() __attribute__((always_inline)) -> void {
        i32x4 (&sums)[W][NF][64] = s_sum[group & 1];
        #pragma unroll
        for (int j = 0; j < NF; ++j) {
            sums[wave][j][lane] = acc[j];
            acc[j] = i32x4{0, 0, 0, 0};
        }
        // the loads under way stay so: nothing but LDS is waited for
        __builtin_amdgcn_s_waitcnt(0xc07f);
        __builtin_amdgcn_s_barrier();
        if (mine) {
            i32x4 sum = sums[0][wave][lane];
            #pragma unroll
            for (int w = 1; w < W; ++w) sum += sums[w][wave][lane];
            const f32x4 sw = s_scale[group][g], b = s_bias[group][g];
            const int m = blockIdx.x * 16 + group * step_m + g * 4;
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < q.out)
                    q.y[n * q.ldy + m + e] = pack1<OT>(__builtin_fmaf(static_cast<float>(sum[e]) * sx, sw[e], b[e]));
        }
        ++group;
        done = 0;
    };
    auto step = [&](const char* use, char* fill) __attribute__((always_inline)) -> void {
        load(fill);
        __builtin_amdgcn_s_waitcnt(0x0f70 | ((2 * kLoads) & 15) | ((2 * kLoads) >> 4) << 14);
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
            const ZERO_LDS char* from = (const ZERO_LDS char*)use + (at ^ (h * 64));
            const i32x4 a = *(const ZERO_LDS i32x4*)from;
            #pragma unroll
            for (int j = 0; j < NF; ++j)
                acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, *(const ZERO_LDS i32x4*)(from + (1 + j) * kRowsBytes),
                                                               acc[j], 0, 0, 0);
        }
        // read before it is filled again
        __builtin_amdgcn_s_waitcnt(0xc07f);
        if (++done == mine_k) finish();
    };
    char *a0 = s0[wave], *a1 = s1[wave], *a2 = s2[wave];
    load(a0);
    load(a1);
    const int steps = groups * mine_k;
    for (int i = 0; i < steps; i += 3) {
        step(a0, a2);
        if (i + 1 < steps) step(a1, a0);
        if (i + 2 < steps) step(a2, a1);
    }
    // no load outlives the block
    __builtin_amdgcn_s_waitcnt(0x0f70);
}

// What the gradient's products read, made in one launch, each part a range of
// blocks: w^ and x^ in 16 bits, dy's rows where they are not whole pieces, and
// sums of dy's columns over shares of its rows.
struct Held {
    const char* codes;        // at the first column
    int64_t stride;
    const float* scale;
    int64_t rows;
    int32_t wide, pieces;     // columns, and pieces of 8 of them
    unsigned short* out;
    int64_t ld;               // elements
};
struct Prepare {
    Held held[2];
    const unsigned short* dy;
    int64_t dy_stride, tokens, out;
    unsigned short* dyr;
    int64_t dyr_ld;
    int64_t share;            // rows of one share of the column sums
    int32_t column_blocks;    // of 256 columns
    int32_t past;             // dy is more than the caches hold: read past them
    float* part;              // [shares][out], or
    unsigned short* db;       // the only share's sums in 16 bits
    uint32_t ends[4];         // the blocks' ranges end here
};

// A block's pieces, of 256 threads: enough for their loads to be on their way
// together.
constexpr int kPrepPieces = 2;

template <int DT>
__device__ __forceinline__ void write_held(const Held& h, uint32_t block) {
    // the block's first piece; from there 32 bits do
    const int64_t first = static_cast<int64_t>(block) * (256 * kPrepPieces);
    const int64_t row0 = first / h.pieces;
    const uint32_t in_row = static_cast<uint32_t>(first - row0 * h.pieces);
    u32x2 c[kPrepPieces];
    float s[kPrepPieces];
    int64_t r[kPrepPieces];
    int d[kPrepPieces];
    #pragma unroll
    for (int i = 0; i < kPrepPieces; ++i) {
        const uint32_t at = in_row + i * 256 + threadIdx.x, down = at / static_cast<uint32_t>(h.pieces);
        r[i] = row0 + down;
        d[i] = static_cast<int>(at - down * h.pieces) * 8;
        if (r[i] >= h.rows) continue;
        c[i] = *reinterpret_cast<const u32x2*>(h.codes + r[i] * h.stride + d[i]);
        s[i] = h.scale[r[i]];
    }
    #pragma unroll
    for (int i = 0; i < kPrepPieces; ++i) {
        if (r[i] >= h.rows) continue;
        float x[8];
        #pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(static_cast<int8_t>(c[i][e / 4] >> (8 * (e % 4)))) * s[i];
        *reinterpret_cast<u32x4*>(h.out + r[i] * h.ld + d[i]) =
            u32x4{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7])};
    }
}

// 256 columns a block, eight rows at a time.
template <int DT>
__device__ __forceinline__ void column_sums(const Prepare& q, uint32_t block) {
    __shared__ float s_sum[8][256];
    const int col = threadIdx.x & 31, row = threadIdx.x >> 5;
    const uint32_t across = block % q.column_blocks;
    const int64_t down = block / q.column_blocks;
    // eight columns a thread; past the last the last eight again
    int64_t d = static_cast<int64_t>(across) * 256 + col * 8;
    if (q.out >= 8 && d > q.out - 8) d = q.out - 8;
    const int64_t first = down * q.share, last = first + q.share < q.tokens ? first + q.share : q.tokens;
    float sum[8] = {};
    // kDeep rows' loads on their way together; past the last row its own again, for nothing
    constexpr int kDeep = 8;
    auto add = [&](auto piece) __attribute__((always_inline)) -> void {
        for (int64_t r = first + row; r < last; r += 8 * kDeep) {
            u32x4 w[kDeep];
            #pragma unroll
            for (int i = 0; i < kDeep; ++i) w[i] = piece(q.dy + (r + 8 * i < last ? r + 8 * i : r) * q.dy_stride);
            #pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                float x[8];
                decode4<DT>(u32x2{w[i].x, w[i].y}, x);
                decode4<DT>(u32x2{w[i].z, w[i].w}, x + 4);
                #pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += r + 8 * i < last ? x[e] : 0.0f;
            }
        }
    };
    typedef u32x4 eight __attribute__((aligned(2)));
    if (q.past) add([&](const unsigned short* at) { return u32x4(__builtin_nontemporal_load(reinterpret_cast<const eight*>(at + d))); });
    else if (q.out >= 8) add([&](const unsigned short* at) { return u32x4(*reinterpret_cast<const eight*>(at + d)); });
    else add([&](const unsigned short* at) { return row_piece(at, d, q.out); });
    // columns of two threads have the same sums twice
    const int64_t from = d - static_cast<int64_t>(across) * 256;
    #pragma unroll
    for (int e = 0; e < 8; ++e)
        if (from + e >= 0) s_sum[row][from + e] = sum[e];
    __syncthreads();
    const int64_t n = static_cast<int64_t>(across) * 256 + threadIdx.x;
    if (n >= q.out) return;
    float total = 0.0f;
    #pragma unroll
    for (int r = 0; r < 8; ++r) total += s_sum[r][threadIdx.x];
    if (q.db) q.db[n] = pack1<DT>(total);
    else q.part[down * q.out + n] = total;
}

template <int DT>
__global__ __launch_bounds__(256) void prepare_kernel(const Prepare q) {
    const uint32_t block = blockIdx.x;
    if (block < q.ends[0]) {
        column_sums<DT>(q, block);
    } else if (block < q.ends[1]) {
        write_held<DT>(q.held[0], block - q.ends[0]);
    } else if (block < q.ends[2]) {
        write_held<DT>(q.held[1], block - q.ends[1]);
    } else {
        const int64_t pieces = q.dyr_ld / 8, blocks = q.ends[3] - q.ends[2];
        for (int64_t at = static_cast<int64_t>(block - q.ends[2]) * 256 + threadIdx.x; at < q.tokens * pieces;
             at += blocks * 256) {
            const int64_t r = at / pieces, d = (at - r * pieces) * 8;
            *reinterpret_cast<u32x4*>(q.dyr + r * q.dyr_ld + d) = row_piece(q.dy + r * q.dy_stride, d, q.out);
        }
    }
}

// What is left of results cut into parts: slices of dx and of dw, shares of
// db, each joined in order, one launch.
struct Slabs {
    const float* slabs;
    int64_t slab, rows, ld;
    int32_t slices, wide;     // columns
    unsigned short* out;
    int64_t out_stride;
};
struct Finish {
    Slabs of[2];
    const float* part;
    int64_t out;
    int32_t shares;
    unsigned short* db;
    uint32_t ends[3];
};
template <int DT>
__global__ __launch_bounds__(256) void finish_kernel(const Finish q) {
    typedef u32x2 quad __attribute__((aligned(2)));
    const uint32_t block = blockIdx.x;
    if (block >= q.ends[1]) {
        const int64_t n = static_cast<int64_t>(block - q.ends[1]) * 256 + threadIdx.x;
        if (n >= q.out) return;
        float total = 0.0f;
        #pragma unroll 8
        for (int i = 0; i < q.shares; ++i) total += q.part[i * q.out + n];
        q.db[n] = pack1<DT>(total);
        return;
    }
    const Slabs& b = q.of[block >= q.ends[0]];
    const int64_t quads = b.ld / 4, at = static_cast<int64_t>(block - (block >= q.ends[0] ? q.ends[0] : 0)) * 256 + threadIdx.x;
    const int64_t r = at / quads, d = (at - r * quads) * 4;
    if (r >= b.rows || d >= b.wide) return;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    #pragma unroll 4
    for (int s = 0; s < b.slices; ++s) x += *reinterpret_cast<const f32x4*>(b.slabs + s * b.slab + r * b.ld + d);
    unsigned short* o = b.out + r * b.out_stride + d;
    if (d + 4 <= b.wide) {
        *reinterpret_cast<quad*>(o) = u32x2{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])};
    } else {
        #pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < b.wide) o[e] = pack1<DT>(x[e]);
    }
}

// The gradient of up to 64 tokens: w8 is read once and dw written once, and
// little else counts.  A wave takes 32 rows of both at a time and 128 columns.
// w^, whose sum runs over the rows, is turned in registers: a lane loads 8
// columns of 8 rows, and what it has of a column is its part of a fragment.
// dy goes to dx's products as it lies and to dw's turned by way of LDS, where
// x^'s fragments lie too; a lane's dw are 8 columns of a row, one store.
// Eight waves join their sums of dx in LDS, the shares of the rows by a
// second kernel, or where there is one share that is dx.
// Of 4096 x 16384 1 token takes 46 us (4.4 TB/s of w8 and dw), 16 49, 32 54 and
// 64 63: 8 us more of products and conversions, 4 of joining.  Up to 16 tokens
// two blocks share a CU (16 tokens: one 54).  33 to 48 tokens have a form of
// their own: 48 take 57.4 us, by that of 64 59.1, of 4096 x 4096 19.5 and 20.4.
// Neighbouring columns' blocks run on unlike XCDs; the other way round 1 token
// takes 52.  w8 read past the caches: 47; dw written through them: 50.
struct FewGradient {
    const char* w8;
    const char* x8;
    int64_t w_row, x_row;     // bytes
    const float *w_scale, *x_scale;
    const unsigned short* dy;
    int64_t dy_stride;
    int32_t share;            // rows of a share, a multiple of 32
    int32_t tokens, dim, out, want_dx;
    float* part;              // [shares][tokens][ld], or NULL: one share
    int64_t ld;
    unsigned short* dx;
    int64_t dx_stride;
    unsigned short* dw;       // or NULL
    int64_t dw_stride;
    unsigned short* db;       // or NULL
};
constexpr int kFewColumns = 128, kGradientWaves = 8, kFewRows = 32;

// Column i of eight columns of codes of eight rows: a fragment.
template <int DT>
__device__ __forceinline__ u32x4 turned8(const u32x2 (&c)[8], const float (&s)[8], int i) {
    u32x4 o;
    #pragma unroll
    for (int r = 0; r < 4; ++r)
        o[r] = pack2<DT>(static_cast<float>(static_cast<int8_t>(c[2 * r][i / 4] >> (8 * (i % 4)))) * s[2 * r],
                         static_cast<float>(static_cast<int8_t>(c[2 * r + 1][i / 4] >> (8 * (i % 4)))) * s[2 * r + 1]);
    return o;
}

template <int DT>
__device__ __forceinline__ f32x4 product16(const u32x4 a, const u32x4 b, const f32x4 c) {
    if constexpr (DT == ZERO_BF16) {
        typedef __bf16 frag __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
    } else {
        typedef _Float16 frag __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
    }
}

template <int DT, int NF>
__global__ __launch_bounds__(kGradientWaves * 64, NF == 1 ? 4 : 2) void few_gradient_kernel(const FewGradient q) {
    const int across = blockIdx.x, down = blockIdx.y;
    constexpr int W = kGradientWaves, KH = NF > 2 ? 2 : 1, kTurned = 32 * KH + 8, kJoinRow = kFewColumns + 4;
    constexpr int kHeldBytes = KH * 8 * 64 * 16, kLoopBytes = kHeldBytes + W * kFewRows * kTurned * 2;
    constexpr int kJoinBytes = W * 16 * kJoinRow * 4;
    __shared__ __attribute__((aligned(16))) char room[kLoopBytes > kJoinBytes ? kLoopBytes : kJoinBytes];
    u32x4* const s_x = reinterpret_cast<u32x4*>(room);     // [half][column of a lane's 8][lane]
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    unsigned short* const s_dy = reinterpret_cast<unsigned short*>(room + kHeldBytes) + wave * kFewRows * kTurned;
    const int d = across * kFewColumns + c * 8;
    const int first = down * q.share, last = first + q.share < q.out ? first + q.share : q.out;
    u32x2 w[8];
    f32x4 scale[2];
    u32x4 dy[NF];
    int past = 0;                                          // of dy's eight elements from the row's end on
    // the wave's next 32 rows; past the last of them all are 0
    auto load = [&](int row) __attribute__((always_inline)) -> void {
        const int rows = row < last ? (q.out - row < kFewRows ? q.out - row : kFewRows) : 0, from = rows > 0 ? row : 0;
        const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(q.w8 + from * q.w_row), 0, q.want_dx ? static_cast<int>(rows * q.w_row) : 0, 0x00020000);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float*>(q.w_scale + from), 0, q.want_dx ? static_cast<int>(rows * 4) : 0, 0x00020000);
        // offsets made here each time: kept from step to step they take registers that are not there
        uint32_t o = g * 8 * static_cast<uint32_t>(q.w_row) + d;
        asm volatile("" : "+v"(o));
        #pragma unroll
        for (int r = 0; r < 8; ++r)
            w[r] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                       rw, d < q.dim ? o + r * static_cast<uint32_t>(q.w_row) : kNowhere, 0, 0));
        #pragma unroll
        for (int r = 0; r < 2; ++r)
            scale[r] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, g * 32 + r * 16, 0, 0));
        // a row's end is taken out of its last eight elements
        const int n = row + g * 8, at = n + 8 <= q.out ? n : q.out - 8;
        past = n - at < 8 ? n - at : 8;
        #pragma unroll
        for (int j = 0; j < NF; ++j) {
            typedef u32x4 eight __attribute__((aligned(2)));
            const int t = j * 16 + c;
            dy[j] = *reinterpret_cast<const eight*>(q.dy + (t < q.tokens ? t : q.tokens - 1) * q.dy_stride + at);
        }
    };
    load(first + wave * kFewRows);
    if (q.dw && wave < KH) {
        u32x2 x[8];
        float s[8];
        #pragma unroll
        for (int r = 0; r < 8; ++r) {
            // codes of tokens past the last count nothing
            const int t = wave * 32 + g * 8 + r, at = t < q.tokens ? t : q.tokens - 1;
            x[r] = *reinterpret_cast<const u32x2*>(q.x8 + at * q.x_row + (d < q.dim ? d : 0));
            s[r] = t < q.tokens ? q.x_scale[at] : 0.0f;
        }
        #pragma unroll
        for (int i = 0; i < 8; ++i) s_x[(wave * 8 + i) * 64 + lane] = turned8<DT>(x, s, i);
    }
    __syncthreads();
    f32x4 acc[8][NF] = {};
    for (int row = first + wave * kFewRows; row < last; row += W * kFewRows) {
        #pragma unroll
        for (int j = 0; j < NF; ++j) dy[j] = past < 8 && j * 16 + c < q.tokens ? moved_down(dy[j], past) : u32x4{0u, 0u, 0u, 0u};
        #pragma unroll
        for (int j = 0; j < NF; ++j)
            #pragma unroll
            for (int e = 0; e < 8; ++e)
                s_dy[(g * 8 + e) * kTurned + j * 16 + c] = static_cast<unsigned short>(dy[j][e / 2] >> (16 * (e % 2)));
        if (q.want_dx) {
            const float s[8] = {scale[0].x, scale[0].y, scale[0].z, scale[0].w, scale[1].x, scale[1].y, scale[1].z, scale[1].w};
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u32x4 b = turned8<DT>(w, s, i);
                #pragma unroll
                for (int j = 0; j < NF; ++j) acc[i][j] = product16<DT>(dy[j], b, acc[i][j]);
            }
        }
        load(row + W * kFewRows);
        if (!q.dw && !(q.db && across == 0)) continue;
        // the wave's own rows of LDS, written above by its other lanes
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        int64_t to0 = static_cast<int64_t>(row + g * 4) * q.dw_stride + d;
        asm volatile("" : "+v"(to0));
        #pragma unroll
        for (int n = 0; n < 2; ++n) {
            u32x4 a[KH];
            #pragma unroll
            for (int h = 0; h < KH; ++h) {
                a[h] = *reinterpret_cast<const u32x4*>(s_dy + (n * 16 + c) * kTurned + h * 32 + g * 8);
                // nothing was written for the other half of the last product's sum
                if (NF % 2 == 1 && h == KH - 1 && g >= 2) a[h] = u32x4{0u, 0u, 0u, 0u};
            }
            if (q.db && across == 0) {
                float all = 0.0f;
                #pragma unroll
                for (int h = 0; h < KH; ++h)
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) all += lo_to_f32<DT>(a[h][e]) + hi_to_f32<DT>(a[h][e]);
                all += __shfl_xor(all, 16, 64);
                all += __shfl_xor(all, 32, 64);
                if (g == 0 && row + n * 16 + c < q.out) q.db[row + n * 16 + c] = pack1<DT>(all);
            }
            if (!q.dw) continue;
            // two columns at a time: what waits for the others is in 16 bits
            u32x4 v[4];
            #pragma unroll
            for (int i = 0; i < 8; i += 2) {
                f32x4 o[2] = {};
                #pragma unroll
                for (int e = 0; e < 2; ++e)
                    #pragma unroll
                    for (int h = 0; h < KH; ++h) o[e] = product16<DT>(a[h], s_x[(h * 8 + i + e) * 64 + lane], o[e]);
                #pragma unroll
                for (int r = 0; r < 4; ++r) v[r][i / 2] = pack2<DT>(o[0][r], o[1][r]);
            }
            #pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (row + n * 16 + g * 4 + r >= q.out || d >= q.dim) continue;
                typedef u32x4 eight __attribute__((aligned(2)));
                typedef u32x2 four __attribute__((aligned(2)));
                typedef uint32_t two __attribute__((aligned(2)));
                unsigned short* to = q.dw + (to0 + (n * 16 + r) * q.dw_stride);
                if (d + 8 <= q.dim) {
                    __builtin_nontemporal_store(v[r], reinterpret_cast<eight*>(to));
                } else {
                    u32x4 x = v[r];
                    const int left = q.dim - d;
                    if (left & 4) {
                        *reinterpret_cast<four*>(to) = u32x2{x.x, x.y};
                        x.x = x.z;
                        x.y = x.w;
                        to += 4;
                    }
                    if (left & 2) {
                        *reinterpret_cast<two*>(to) = x.x;
                        x.x = x.y;
                        to += 2;
                    }
                    if (left & 1) *to = static_cast<unsigned short>(x.x);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    if (!q.want_dx) return;
    float* const s_join = reinterpret_cast<float*>(room);  // [wave][16 tokens][kJoinRow]
    #pragma unroll
    for (int j = 0; j < NF; ++j) {
        __syncthreads();
        #pragma unroll
        for (int r = 0; r < 4; ++r)
            #pragma unroll
            for (int i = 0; i < 8; i += 4)
                *reinterpret_cast<f32x4*>(s_join + (wave * 16 + g * 4 + r) * kJoinRow + c * 8 + i) =
                    f32x4{acc[i][j][r], acc[i + 1][j][r], acc[i + 2][j][r], acc[i + 3][j][r]};
        __syncthreads();
        const int in = threadIdx.x / 32, at = threadIdx.x % 32 * 4, t = j * 16 + in, column = across * kFewColumns + at;
        f32x4 x = *reinterpret_cast<const f32x4*>(s_join + in * kJoinRow + at);
        #pragma unroll
        for (int v = 1; v < W; ++v) x += *reinterpret_cast<const f32x4*>(s_join + (v * 16 + in) * kJoinRow + at);
        if (t >= q.tokens) continue;
        if (q.part) {
            if (column < q.ld)
                *reinterpret_cast<f32x4*>(q.part + (static_cast<int64_t>(down) * q.tokens + t) * q.ld + column) = x;
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (column + e < q.dim) q.dx[t * q.dx_stride + column + e] = pack1<DT>(x[e]);
        }
    }
}

struct FewJoin {
    const float* part;        // [shares][rows][ld]
    int64_t ld;
    int32_t shares, rows, dim;
    unsigned short* out;
    int64_t out_stride;
};
// Four columns of a row to 16 threads, each with every 16th share.
template <int DT>
__global__ __launch_bounds__(256) void few_join_kernel(const FewJoin q) {
    typedef u32x2 quad __attribute__((aligned(2)));
    __shared__ f32x4 s_sum[16][17];
    const int mine = threadIdx.x % 16, group = threadIdx.x / 16;
    const int64_t quads = q.ld / 4, at = static_cast<int64_t>(blockIdx.x) * 16 + mine;
    const int64_t r = at / quads, d = (at - r * quads) * 4;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r < q.rows) {
        #pragma unroll 8
        for (int s = group; s < q.shares; s += 16)
            x += *reinterpret_cast<const f32x4*>(q.part + (static_cast<int64_t>(s) * q.rows + r) * q.ld + d);
    }
    s_sum[group][mine] = x;
    __syncthreads();
    if (group != 0 || r >= q.rows || d >= q.dim) return;
    #pragma unroll
    for (int s = 1; s < 16; ++s) x += s_sum[s][mine];
    unsigned short* o = q.out + r * q.out_stride + d;
    if (d + 4 <= q.dim) {
        *reinterpret_cast<quad*>(o) = u32x2{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])};
    } else {
        #pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < q.dim) o[e] = pack1<DT>(x[e]);
    }
}

// ------------------------------------------------------------------ launches
constexpr int64_t kMaxTokens = int64_t(1) << 20, kMaxOut = int64_t(1) << 20;
// few8_kernel's rule: up to 64 tokens; up to 1024 while its parts, 16 rows by
// 64 tokens, are at most two rounds of the CUs and dim is short.  Microseconds,
// and those of the tiles: 17 tokens x 4096 x 4096 6.9 and 11.6, x 16384 16 and
// 24; 64 x 4096 x 16384 23.3 and 25.0, x 1000 x 10007 9.5 and 9.4; 128 x 4096 x
// 4096 (512 parts) 13.6 and 15.0, 512 x 512 x 512 4.5 and 6.3, but 192 x 4096 x
// 4096 (768) 28.5 and 17.1, 128 x 16384 x 4096 41 and 27, x 4096 x 16384 40 and
// 25.  Few rows that are long leave its blocks one after another's loads, 0.3 to
// 0.5 us for 512 of k, and CUs idle that slices of tiles would use: 64 x 16384 x
// 1024 18.8 and 14.1, x 300 17.8 and 11.8, 17 x 16384 x 1024 13.6 and 12.7, 1 x
// 65536 x 128 33 and 16, x 32768 x 900 18.6 and 15.3, but 64 x 8192 x 1024 12.0
// and 12.0, 17 x 10000 x 512 9.9 and 11.3, 1 x 16384 x 1024 11.2 and 12.0, 32 x
// 16384 x 2048 14.2 and 15.4.
constexpr int64_t kFewTokens = 64, kMoreTokens = 1024, kFewParts = 512, kFewDim = 4096;
constexpr int kTilesAtOnce = 2 * kCus;        // of 128 x 128
constexpr int64_t kCacheBytes = int64_t(256) << 20;
constexpr int64_t kMostPacks = 1 << 22;       // blocks; with the others' the grid's 32 bits hold them
constexpr size_t kPieceBytes = size_t(512) << 20;

// What a gradient's call has to make, a copy of dy's rows among it where they
// are not read as they lie.
struct Wanted {
    bool dx, dw, db, copy_dy;
};
Wanted wanted(const zero_linear8_args* a) {
    Wanted w;
    w.dx = a->dx && a->tokens > 0 && a->dim > 0;
    w.dw = a->dw && a->out > 0 && a->dim > 0;
    w.db = a->db && a->out > 0;
    w.copy_dy = (w.dx || w.dw) && a->tokens > 0 && a->out > 0 && !whole_pieces(a->dy, a->dy_stride, a->out);
    return w;
}

// How a gradient is cut: by the three sizes alone; and its workspace.
struct Cut {
    int64_t piece;            // columns of dim at a time, a multiple of 256
    int32_t dx_slices, dw_slices;
    int32_t shares;           // of db's sum
    size_t x_bytes, w_bytes, dy_bytes, dx_slab, dw_slab, part_bytes;
    int32_t few_shares;       // few_gradient_kernel's
    size_t total;
};

// Whether few_gradient_kernel takes it: up to 32 tokens, and up to 64 of weights
// that are not small, where the tiles' three launches are the shorter chain.
// Microseconds, and those of the tiles: 64 tokens x 4096 x 16384 63 and 125, x
// 1024 x 16384 26 and 44, x 1000 x 4100 16.8 and 18.7, but x 1000 x 2053 18.7 and
// 16.5, x 200 x 300 12.7 and 9.5; x 2048 x 1000, 15.6 and 16.8, goes by the tiles
// all the same.  32 tokens x 1000 x 2053 14.1 and 15.8, x 200 x 300 9.3 and 9.2;
// 16 x 200 x 300 8.1 and 9.2, x 64 x 64 5.9 and 7.3; 1 x 1000 x 4100 11.6, where
// a kernel without matrix cores took 10.6, but x 64 x 64 5.7 and 7.0.
constexpr int64_t kFewGradientTokens = 32, kMoreGradientTokens = 64, kMoreWeights = int64_t(1) << 21;
bool few_gradient_rule(int64_t tokens, int64_t dim, int64_t out) {
    // a row of dy has whole pieces to take its end out of
    if (out < 8) return false;
    return tokens <= kFewGradientTokens || (tokens <= kMoreGradientTokens && dim * out >= kMoreWeights);
}

bool in_range(int64_t tokens, int64_t dim, int64_t out) {
    return tokens >= 0 && tokens <= kMaxTokens && dim >= 0 && dim <= ZERO_ROWS8_MAX_DIM && out >= 0 && out <= kMaxOut;
}

bool cut(int64_t tokens, int64_t dim, int64_t out, const Wanted& want, Cut* c) {
    if (!in_range(tokens, dim, out)) return false;
    const int64_t t = tokens > 0 ? tokens : 1, k = up(dim > 0 ? dim : 1, 256), n = out > 0 ? out : 1;
    int64_t piece = static_cast<int64_t>(kPieceBytes / (2 * static_cast<size_t>(t + n))) / 256 * 256;
    c->piece = piece < 256 ? 256 : (piece > k ? k : piece);
    // slices of the sum where the tiles of 128 x 128 alone would leave CUs idle
    const int64_t dim_tiles = c->piece / 128;
    auto slices = [](int64_t tiles, int64_t sum) {
        int64_t s = kTilesAtOnce / tiles;
        if (s > sum / 512) s = sum / 512;
        return static_cast<int32_t>(s < 1 ? 1 : (s > 64 ? 64 : s));
    };
    c->dx_slices = slices(dim_tiles * (up(t, 128) / 128), n);
    c->dw_slices = slices(dim_tiles * (up(n, 128) / 128), t);
    const int64_t columns = up(n, 256) / 256;
    int64_t shares = 1024 / columns;
    if (shares > t / 64) shares = t / 64;
    c->shares = static_cast<int32_t>(shares < 1 ? 1 : shares);
    auto bytes = [](bool needed, int64_t count, size_t of) {
        return needed ? round_up(static_cast<size_t>(count) * of, 256) : size_t(0);
    };
    c->x_bytes = bytes(want.dw, t * c->piece, 2);
    c->w_bytes = bytes(want.dx, n * c->piece, 2);
    c->dy_bytes = bytes(want.copy_dy, t * up(n, 64), 2);
    c->dx_slab = bytes(want.dx && c->dx_slices > 1, c->dx_slices * t * c->piece, 4);
    c->dw_slab = bytes(want.dw && c->dw_slices > 1, c->dw_slices * n * c->piece, 4);
    c->part_bytes = bytes(want.db && c->shares > 1, c->shares * n, 4);
    c->total = c->x_bytes + c->w_bytes + c->dy_bytes + c->dx_slab + c->dw_slab + c->part_bytes;
    // one or two blocks a CU, a step or more for each of their waves
    int64_t few = kCus * (t <= 16 ? 2 : 1) / (up(k, kFewColumns) / kFewColumns);
    if (few > n / (kGradientWaves * kFewRows)) few = n / (kGradientWaves * kFewRows);
    c->few_shares = static_cast<int32_t>(few < 1 ? 1 : few);
    if (few_gradient_rule(t, dim, n)) {
        // nothing is written out in 16 bits, and db is one share's
        c->x_bytes = c->w_bytes = c->dy_bytes = c->dx_slab = c->dw_slab = 0;
        c->total = bytes(want.dx && c->few_shares > 1, c->few_shares * t * k, 4);
    }
    return true;
}

// As many blocks as the CUs' LDS holds at once, if they come round at most 16
// times; a block's rows as many as another's.
template <int OT, int NF>
void few(const Few& q, hipStream_t st) {
    constexpr int kLds = 3 * kFewWaves * (1 + NF) * 2048 + 2 * kFewWaves * NF * 1024 + kMostGroups * 128;
    constexpr int most = kCus * (kLdsBytes / kLds);
    const int rows = (q.out + 15) / 16, tokens = (q.tokens + 16 * NF - 1) / (16 * NF);
    int times = (rows * tokens + most - 1) / most;
    times = times < kMostGroups ? times : kMostGroups;
    const int blocks = (rows + times - 1) / times;
    hipLaunchKernelGGL((few8_kernel<OT, NF>), dim3(blocks, tokens), dim3(kFewWaves * 64), 0, st, q);
}

// Slices of the forward's k: tiles that leave CUs idle take shares of it.  A
// step of 128 of k takes a tile 0.53 us, all of their operands come at 10 TB/s
// at best, a slice's sums are written and read once each, and joining them is
// a launch.  Microseconds with 1, 2, 3, 4 and 8 slices, and the rule's choice:
// 256 tokens x 4096 x 4096 23.0, 20.1, 18.7, 18.5, 23.0 (3); 256 x 16384 x 4096
// 67.5, 46.6, 37.4 (46 elsewhere in memory), 40.2, 39.6 (3); 512 x 4096 x 4096
// 23.5, 24.6, 26.6, 27.3, 43.9 (1); 700 x 8000 x 1500 43.3, 31.8, 26.4, 28.9,
// 32.8 (3).  It is not always the best: 512 x 16384 x 4096 71.2, 65.0, 61.9, 56.5,
// 70.2 (2), 1500 x 16000 x 600 72.7, 45.9, 36.0, 33.0, 34.0 (3).
int forward_slices(int64_t tokens, int64_t dim, int64_t out) {
    const int64_t tiles = up(tokens, 128) / 128 * (up(out, 128) / 128), steps = up(dim, 128) / 128;
    const double operands = static_cast<double>(tiles) * 256.0 * static_cast<double>(dim) * 1e-7;
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= 32 && s * tiles <= kTilesAtOnce && s <= steps; ++s) {
        const double latency = 0.53 * static_cast<double>((steps + s - 1) / s);
        const double join = s > 1 ? 3.0 + static_cast<double>(s * tokens) * static_cast<double>(out) * 1e-6 : 0.0;
        const double t = (latency > operands ? latency : operands) + join;
        if (t < least) {
            least = t;
            best = s;
        }
    }
    return best;
}
bool few_rows(int64_t tokens, int64_t dim, int64_t out) {
    const bool thin = out <= (tokens > 32 ? 2048 : 1024) && dim > (tokens > 32 ? 8192 : (tokens > 16 ? 12288 : 16384));
    if (tokens <= kFewTokens) return !thin;
    return tokens <= kMoreTokens && dim <= kFewDim && (out + 15) / 16 * ((tokens + 63) / 64) <= kFewParts;
}

struct Join {
    const int* slabs;
    int64_t slab, ld;
    int32_t slices, tokens, out;
    const float *w_scale, *x_scale;
    const unsigned short* bias;
    unsigned short* y;
    int64_t ldy;
};
// The slices' whole sums added, scaled and rounded; four channels a thread.
template <int OT>
__global__ __launch_bounds__(256) void join_kernel(const Join q) {
    typedef u32x2 quad __attribute__((aligned(2)));
    const int64_t quads = q.ld / 4, at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t n = at / quads, m = (at - n * quads) * 4;
    if (n >= q.tokens || m >= q.out) return;
    i32x4 sum = {0, 0, 0, 0};
    #pragma unroll 4
    for (int s = 0; s < q.slices; ++s) sum += *reinterpret_cast<const i32x4*>(q.slabs + s * q.slab + n * q.ld + m);
    const float sx = q.x_scale[n];
    float x[4];
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t i = m + e < q.out ? m + e : q.out - 1;
        x[e] = __builtin_fmaf(static_cast<float>(sum[e]) * sx, q.w_scale[i], q.bias ? lo_to_f32<OT>(q.bias[i]) : 0.0f);
    }
    unsigned short* o = q.y + n * q.ldy + m;
    if (m + 4 <= q.out) {
        *reinterpret_cast<quad*>(o) = u32x2{pack2<OT>(x[0], x[1]), pack2<OT>(x[2], x[3])};
    } else {
        #pragma unroll
        for (int e = 0; e < 4; ++e)
            if (m + e < q.out) o[e] = pack1<OT>(x[e]);
    }
}

// Bytes of workspace that a call uses, 256 at least.
constexpr size_t kLeastBytes = 256;
size_t forward_bytes(int64_t tokens, int64_t dim, int64_t out) {
    const int slices = few_rows(tokens, dim, out) ? 1 : forward_slices(tokens, dim, out);
    const size_t sums = slices > 1 ? static_cast<size_t>(slices) * tokens * up(out, 64) * 4 : 0;
    return sums > kLeastBytes ? round_up(sums, 256) : kLeastBytes;
}
size_t backward_bytes(int64_t tokens, int64_t dim, int64_t out, const Wanted& want) {
    Cut c;
    if (!cut(tokens, dim, out, want, &c)) return 0;
    return c.total > kLeastBytes ? c.total : kLeastBytes;
}

// And the most that calls of up to so many tokens use: fewer tokens may be cut
// into more slices, or have wider pieces of columns.
size_t most_forward_bytes(int64_t tokens, int64_t dim, int64_t out) {
    size_t most = kLeastBytes;
    if (out == 0) return most;
    // none with more tiles than half of the chip's is cut
    for (int64_t t = 1; t <= tokens && 2 * (up(t, 128) / 128) * (up(out, 128) / 128) <= kTilesAtOnce; ++t) {
        const size_t b = forward_bytes(t, dim, out);
        most = b > most ? b : most;
    }
    return most;
}
size_t most_backward_bytes(int64_t tokens, int64_t dim, int64_t out, bool copy_dy) {
    const Wanted all = {true, true, true, copy_dy};
    size_t most = backward_bytes(tokens, dim, out, all);
    // Between two of these nothing but the tokens grows: rules end at 16, 32 and
    // 64, tiles and shares change at multiples of 64 or behind them, and a
    // narrower piece begins where its width no longer divides kPieceBytes so.
    auto look = [&](int64_t t) {
        if (t < 1 || t >= tokens) return;
        const size_t b = backward_bytes(t, dim, out, all);
        most = b > most ? b : most;
    };
    look(16);
    look(32);
    for (int64_t t = 64; t <= tokens; t += 64) {
        look(t - 1);
        look(t);
    }
    const int64_t n = out > 0 ? out : 1;
    for (int64_t wide = 256; wide <= up(dim, 256); wide += 256)
        look(static_cast<int64_t>(kPieceBytes) / 2 / wide - n);
    return most;
}

template <int OT>
int forward(const zero_linear8_args* a, hipStream_t st) {
    const int64_t k = ZERO_ROWS8_BYTES(a->dim);
    if (few_rows(a->tokens, a->dim, a->out)) {
        Few q = {};
        q.w = static_cast<const char*>(a->w8);
        q.x = static_cast<const char*>(a->x8);
        q.ldw = a->w8_stride;
        q.ldx = a->x8_stride;
        q.out = static_cast<int32_t>(a->out);
        q.tokens = static_cast<int32_t>(a->tokens);
        q.k = static_cast<int32_t>(k);
        q.w_scale = a->w_scale;
        q.x_scale = a->x_scale;
        q.bias = static_cast<const unsigned short*>(a->bias);
        q.y = static_cast<unsigned short*>(a->y);
        q.ldy = a->y_stride;
        if (a->tokens <= 16) few<OT, 1>(q, st);
        else if (a->tokens <= 32) few<OT, 2>(q, st);
        else few<OT, 4>(q, st);
        return launch_error("product kernel launch");
    }
    constexpr Epilogue E = OT == ZERO_BF16 ? kScaledBf16 : kScaledFp16;
    Product q = {};
    q.a = static_cast<const char*>(a->w8);
    q.lda = a->w8_stride;
    q.b = static_cast<const char*>(a->x8);
    q.ldb = a->x8_stride;
    q.m = q.valid_m = static_cast<int32_t>(a->out);
    q.n = static_cast<int32_t>(a->tokens);
    q.k = static_cast<int32_t>(k / 2);
    q.slice = static_cast<int32_t>(up(q.k, kTileK));
    q.c = static_cast<char*>(a->y);
    q.ldc = a->y_stride;
    q.scale_m = a->w_scale;
    q.scale_n = a->x_scale;
    q.bias = static_cast<const unsigned short*>(a->bias);
    const int slices = forward_slices(a->tokens, a->dim, a->out);
    if (slices == 1) {
        launch_product<kCodes, kRows, kRows, E>(q, 1, st);
        return launch_error("product kernel launch");
    }
    q.slice = static_cast<int32_t>(up(up(q.k, slices) / slices, kTileK));
    q.c = static_cast<char*>(a->workspace);
    q.ldc = up(a->out, 64);
    q.slab = a->tokens * q.ldc;
    launch_tiles<kCodes, kRows, kRows, E, 128, 128, 2, 2>(q, slices, st);
    const Join j = {static_cast<const int*>(a->workspace), q.slab, q.ldc, slices, q.n, q.m, a->w_scale, a->x_scale,
                    q.bias, static_cast<unsigned short*>(a->y), a->y_stride};
    hipLaunchKernelGGL((join_kernel<OT>), dim3(static_cast<unsigned>((q.slab / 4 + 255) / 256)), dim3(256), 0, st, j);
    return launch_error("product kernel launch");
}

// A gradient's product: its slices' parts go to `slabs`, without slices its
// result where it belongs.
void place(Product* q, int slices, float* slabs, int64_t ld, int64_t rows, int64_t wide, void* out, int64_t out_stride) {
    q->slices = slices;
    q->slice = static_cast<int32_t>(up(up(q->k, slices) / slices, kTileK));
    q->valid_m = static_cast<int32_t>(wide);
    q->c = slices > 1 ? reinterpret_cast<char*>(slabs) : static_cast<char*>(out);
    q->ldc = slices > 1 ? ld : out_stride;
    q->slab = rows * ld;
}

// dx's and dw's tiles of 128 x 128 in one grid, either may have none: each
// leaves CUs idle by itself (509 tokens x 1000 x 2053 in fp16 13 and 9 us one
// after the other).
template <int DT>
void two_products(Product a, Product b, hipStream_t st) {
    a.tiles_m = (a.m + 127) / 128;
    b.tiles_m = (b.m + 127) / 128;
    const int64_t na = tiles_of(a, 128, 128) * a.slices, nb = tiles_of(b, 128, 128) * b.slices;
    int64_t first, second;
    share_blocks(na, nb, a.slice + kTileK, b.slice + kTileK, kTilesAtOnce, &first, &second);
    hipLaunchKernelGGL((two_products_kernel<DT, kEither, 128, 128, 2, 2>), dim3(static_cast<unsigned>(first + second)),
                       dim3(256), 0, st, a, b, static_cast<int>(first));
}

template <int DT>
int few_gradient(const zero_linear8_args* a, const Cut& c, hipStream_t st) {
    FewGradient q = {};
    q.w8 = static_cast<const char*>(a->w8);
    q.x8 = static_cast<const char*>(a->x8);
    q.w_row = a->w8_stride;
    q.x_row = a->x8_stride;
    q.w_scale = a->w_scale;
    q.x_scale = a->x_scale;
    q.dy = static_cast<const unsigned short*>(a->dy);
    q.dy_stride = a->dy_stride;
    q.out = static_cast<int32_t>(a->out);
    q.dim = static_cast<int32_t>(a->dim);
    q.share = static_cast<int32_t>(up(up(a->out, c.few_shares) / c.few_shares, kFewRows));
    q.tokens = static_cast<int32_t>(a->tokens);
    q.want_dx = a->dx != nullptr;
    q.part = a->dx && c.few_shares > 1 ? static_cast<float*>(a->workspace) : nullptr;
    q.ld = up(a->dim, 8);
    q.dx = static_cast<unsigned short*>(a->dx);
    q.dx_stride = a->dx_stride;
    q.dw = static_cast<unsigned short*>(a->dw);
    q.dw_stride = a->dw_stride;
    q.db = static_cast<unsigned short*>(a->db);
    const dim3 grid(static_cast<unsigned>(up(a->dim, kFewColumns) / kFewColumns), static_cast<unsigned>(c.few_shares));
    if (a->tokens <= 16) hipLaunchKernelGGL((few_gradient_kernel<DT, 1>), grid, dim3(kGradientWaves * 64), 0, st, q);
    else if (a->tokens <= 32) hipLaunchKernelGGL((few_gradient_kernel<DT, 2>), grid, dim3(kGradientWaves * 64), 0, st, q);
    else if (a->tokens <= 48) hipLaunchKernelGGL((few_gradient_kernel<DT, 3>), grid, dim3(kGradientWaves * 64), 0, st, q);
    else hipLaunchKernelGGL((few_gradient_kernel<DT, 4>), grid, dim3(kGradientWaves * 64), 0, st, q);
    if (q.part) {
        const FewJoin j = {q.part, q.ld, c.few_shares, q.tokens, q.dim, q.dx, q.dx_stride};
        hipLaunchKernelGGL((few_join_kernel<DT>), dim3(static_cast<unsigned>((a->tokens * (q.ld / 4) + 15) / 16)), dim3(256), 0,
                           st, j);
    }
    return launch_error("product gradient kernel launch");
}

template <int DT>
int backward(const zero_linear8_args* a, const Wanted& want, const Cut& c, hipStream_t st) {
    if (a->tokens > 0 && a->dim > 0 && (a->dx || a->dw) && few_gradient_rule(a->tokens, a->dim, a->out))
        return few_gradient<DT>(a, c, st);
    char* ws = static_cast<char*>(a->workspace);
    unsigned short* x16 = reinterpret_cast<unsigned short*>(ws);
    unsigned short* w16 = reinterpret_cast<unsigned short*>(ws + c.x_bytes);
    unsigned short* dyr = reinterpret_cast<unsigned short*>(ws + c.x_bytes + c.w_bytes);
    float* dx_slab = reinterpret_cast<float*>(ws + c.x_bytes + c.w_bytes + c.dy_bytes);
    float* dw_slab = dx_slab + c.dx_slab / 4;
    float* part = dw_slab + c.dw_slab / 4;
    const int64_t t = a->tokens, n = a->out;
    const bool whole = whole_pieces(a->dy, a->dy_stride, n);
    const int64_t dyr_ld = up(n, 64);
    const int64_t last = want.dx || want.dw ? a->dim : 1;   // db alone: once
    for (int64_t d = 0; d < last; d += c.piece) {
        const int64_t wide = a->dim - d < c.piece ? a->dim - d : c.piece;
        Prepare p = {};
        auto held = [&](Held* h, const void* codes, int64_t stride, const float* scale, int64_t rows,
                        unsigned short* out) -> uint32_t {
            *h = {static_cast<const char*>(codes) + d, stride, scale, rows, static_cast<int32_t>(wide),
                  static_cast<int32_t>(up(wide, 8) / 8), out, c.piece};
            return static_cast<uint32_t>((rows * h->pieces + 256 * kPrepPieces - 1) / (256 * kPrepPieces));
        };
        p.dy = static_cast<const unsigned short*>(a->dy);
        p.dy_stride = a->dy_stride;
        p.tokens = t;
        p.out = n;
        p.dyr = dyr;
        p.dyr_ld = dyr_ld;
        p.column_blocks = static_cast<int32_t>(up(n, 256) / 256);
        p.share = up(up(t, c.shares) / c.shares, 8);
        // 8192 x 16384 98 us for 107 with w^ and x^; 2048 x 4096, which the
        // products then find in the caches, 142 us in all for 140
        p.past = n >= 8 && t * n * 2 >= kCacheBytes;
        p.part = part;
        p.db = c.shares == 1 ? static_cast<unsigned short*>(a->db) : nullptr;
        p.ends[0] = d == 0 && want.db ? static_cast<uint32_t>(p.column_blocks * c.shares) : 0;
        p.ends[1] = p.ends[0] + (want.dx ? held(&p.held[0], a->w8, a->w8_stride, a->w_scale, n, w16) : 0);
        p.ends[2] = p.ends[1] + (want.dw ? held(&p.held[1], a->x8, a->x8_stride, a->x_scale, t, x16) : 0);
        const int64_t packs = (t * (dyr_ld / 8) + 255) / 256;
        p.ends[3] = p.ends[2] + (d == 0 && want.copy_dy ? static_cast<uint32_t>(packs < kMostPacks ? packs : kMostPacks) : 0);
        if (p.ends[3] > 0) hipLaunchKernelGGL((prepare_kernel<DT>), dim3(p.ends[3]), dim3(256), 0, st, p);

        Finish f = {};
        Product dx = {}, dw = {};
        auto both = [&](Product* q, const unsigned short* held16) {
            q->a = reinterpret_cast<const char*>(held16);
            q->lda = c.piece * 2;
            q->m = static_cast<int32_t>(up(wide, 8));
            // No row or no column: nothing of dy is read, nor of a copy that is not
            // made; but rows of any stride would lead kNowhere back into range.
            q->b = whole ? static_cast<const char*>(a->dy) : reinterpret_cast<const char*>(dyr);
            q->ldb = (whole ? a->dy_stride : dyr_ld) * 2;
        };
        if (want.dx) {
            unsigned short* out = static_cast<unsigned short*>(a->dx) + d;
            both(&dx, w16);
            dx.n = static_cast<int32_t>(t);
            dx.k = static_cast<int32_t>(n);
            place(&dx, c.dx_slices, dx_slab, c.piece, t, wide, out, a->dx_stride);
            f.of[0] = {dx_slab, dx.slab, t, c.piece, c.dx_slices, static_cast<int32_t>(wide), out, a->dx_stride};
            f.ends[0] = c.dx_slices > 1 ? static_cast<uint32_t>((t * (c.piece / 4) + 255) / 256) : 0;
        }
        f.ends[1] = f.ends[0];
        if (want.dw) {
            unsigned short* out = static_cast<unsigned short*>(a->dw) + d;
            both(&dw, x16);
            dw.n = static_cast<int32_t>(n);
            dw.k = static_cast<int32_t>(t);
            place(&dw, c.dw_slices, dw_slab, c.piece, n, wide, out, a->dw_stride);
            f.of[1] = {dw_slab, dw.slab, n, c.piece, c.dw_slices, static_cast<int32_t>(wide), out, a->dw_stride};
            f.ends[1] += c.dw_slices > 1 ? static_cast<uint32_t>((n * (c.piece / 4) + 255) / 256) : 0;
        }
        f.part = part;
        f.out = n;
        f.shares = c.shares;
        f.db = static_cast<unsigned short*>(a->db);
        f.ends[2] = f.ends[1] + (d == 0 && want.db && c.shares > 1 ? static_cast<uint32_t>((n + 255) / 256) : 0);
        // more than one slice only where they are one round of the small tiles
        const bool large_dx = want.dx && c.dx_slices == 1 && large_tiles(dx, 1);
        const bool large_dw = want.dw && c.dw_slices == 1 && large_tiles(dw, 1);
        if (large_dx) launch_tiles<DT, kCols, kRows, kPlain, 256, 256, 2, 2>(dx, 1, st);
        if (large_dw) launch_tiles<DT, kCols, kCols, kPlain, 256, 256, 2, 2>(dw, 1, st);
        if ((want.dx && !large_dx) || (want.dw && !large_dw))
            two_products<DT>(large_dx ? Product{} : dx, large_dw ? Product{} : dw, st);
        if (f.ends[2] > 0) hipLaunchKernelGGL((finish_kernel<DT>), dim3(f.ends[2]), dim3(256), 0, st, f);
    }
    return launch_error("product gradient kernel launch");
}

}  // namespace

size_t linear8_needs(const zero_linear8_args* a, bool backward) {
    if (!in_range(a->tokens, a->dim, a->out)) return 0;
    return backward ? backward_bytes(a->tokens, a->dim, a->out, wanted(a)) : forward_bytes(a->tokens, a->dim, a->out);
}

}  // namespace zero

using namespace zero;

extern "C" {

size_t zero_linear8_workspace_bytes_for(int64_t tokens, int64_t dim, int64_t out, int32_t uses) {
    constexpr int32_t kAll = ZERO_LINEAR8_FORWARD | ZERO_LINEAR8_BACKWARD | ZERO_LINEAR8_BACKWARD_ANY_DY;
    if (!in_range(tokens, dim, out) || uses <= 0 || (uses & ~kAll)) return 0;
    size_t most = kLeastBytes;
    auto with = [&](size_t b) { most = b > most ? b : most; };
    if (uses & ZERO_LINEAR8_FORWARD) with(most_forward_bytes(tokens, dim, out));
    if (uses & ZERO_LINEAR8_BACKWARD) with(most_backward_bytes(tokens, dim, out, false));
    if (uses & ZERO_LINEAR8_BACKWARD_ANY_DY) with(most_backward_bytes(tokens, dim, out, true));
    return most;
}

size_t zero_linear8_workspace_bytes(int64_t tokens, int64_t dim, int64_t out) {
    return zero_linear8_workspace_bytes_for(tokens, dim, out, ZERO_LINEAR8_FORWARD | ZERO_LINEAR8_BACKWARD_ANY_DY);
}

int zero_linear8_forward(const zero_linear8_args* a, void* stream) {
    clear_error();
    const int rc = check_linear8_args(a, false);
    if (rc || a->tokens == 0 || a->out == 0) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a->dtype == ZERO_BF16 ? forward<ZERO_BF16>(a, st) : forward<ZERO_FP16>(a, st);
}

int zero_linear8_backward(const zero_linear8_args* a, void* stream) {
    clear_error();
    const int rc = check_linear8_args(a, true);
    if (rc || (a->tokens == 0 && a->out == 0)) return rc;
    const Wanted want = wanted(a);
    Cut c;
    cut(a->tokens, a->dim, a->out, want, &c);
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a->dtype == ZERO_BF16 ? backward<ZERO_BF16>(a, want, c, st) : backward<ZERO_FP16>(a, want, c, st);
}

}  // extern "C"
