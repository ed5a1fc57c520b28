// train_linear8.hip -- the product of 8-bit rows with 8-bit weights and its
// gradient (include/zero/train.h).
//
//   forward    y = x8 w8^T in whole numbers on the matrix cores, scaled and
//              rounded once in the epilogue.  Up to 64 tokens w8 goes straight
//              from memory to registers.
//   backward   x^ and w^ are written out in 16 bits (exact with the encoder's
//              scales), as many columns of dim at a time as 512 MB hold; then
//              dx = dy w^ and dw = dy^T x^.  Small results are cut along
//              their sum into slices, joined in a fixed order.
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

// Up to 16 NF tokens: w8 is read once and nothing else counts, so the
// fragments go from memory to registers, many loads at a time.  A block takes
// 16 rows of w8; its four waves take every fourth 128 of k, and the sums,
// whole numbers, meet in LDS.
template <int OT, int NF>
__global__ __launch_bounds__(256) void few8_kernel(const Few q) {
    constexpr int kGroup = 2;                              // of 128 k a wave and turn
    __shared__ i32x4 s_sum[4][NF][64];
    const int lane = threadIdx.x & 63, s = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int m0 = blockIdx.x * 16;
    auto records = [](int64_t bytes) { return static_cast<int>(bytes < 0x7ffffff0 ? bytes : 0x7ffffff0); };
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(q.w + m0 * q.ldw), 0, records((q.out - m0) * q.ldw), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(q.x), 0,
                                                                        records(q.tokens * q.ldx), 0x00020000);
    const uint32_t oa = static_cast<uint32_t>(s * q.ldw), ob = static_cast<uint32_t>(s * q.ldx);
    const uint32_t next = static_cast<uint32_t>(16 * q.ldx);
    struct Pieces {
        u32x4 a[kGroup][2], b[kGroup][2][NF];
    };
    // k of this lane's piece p of block `block` of 128: both operands agree on it
    auto load = [&](Pieces& f, int block) __attribute__((always_inline)) -> void {
        #pragma unroll
        for (int u = 0; u < kGroup; ++u)
            #pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int k = (block + 4 * u) * 128 + g * 32 + p * 16;
                f.a[u][p] = __builtin_amdgcn_raw_buffer_load_b128(ra, k < q.k ? oa + k : kNowhere, 0, 0);
                #pragma unroll
                for (int j = 0; j < NF; ++j)
                    f.b[u][p][j] = __builtin_amdgcn_raw_buffer_load_b128(rb, k < q.k ? ob + j * next + k : kNowhere, 0, 0);
            }
    };
    i32x4 acc[NF] = {};
    auto multiply = [&](const Pieces& f) __attribute__((always_inline)) -> void {
        #pragma unroll
        for (int u = 0; u < kGroup; ++u)
            #pragma unroll
            for (int p = 0; p < 2; ++p)
                #pragma unroll
                for (int j = 0; j < NF; ++j)
                    acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, f.a[u][p]),
                                                                   __builtin_bit_cast(i32x4, f.b[u][p][j]), acc[j], 0, 0, 0);
    };
    const int blocks = (q.k + 127) / 128;
    Pieces f0, f1;
    load(f0, wave);
    for (int b = wave; b < blocks; b += 8 * kGroup) {
        load(f1, b + 4 * kGroup);
        multiply(f0);
        load(f0, b + 8 * kGroup);
        multiply(f1);
    }
    #pragma unroll
    for (int j = 0; j < NF; ++j) s_sum[wave][j][lane] = acc[j];
    __syncthreads();
    // a wave finishes 16 tokens
    const int n = wave * 16 + s;
    if (wave >= NF || n >= q.tokens) return;
    const i32x4 sum = s_sum[0][wave][lane] + s_sum[1][wave][lane] + s_sum[2][wave][lane] + s_sum[3][wave][lane];
    const float sx = q.x_scale[n];
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int m = m0 + g * 4 + e;
        if (m >= q.out) break;
        const float b = q.bias ? lo_to_f32<OT>(q.bias[m]) : 0.0f;
        q.y[n * q.ldy + m] = pack1<OT>(__builtin_fmaf(static_cast<float>(sum[e]) * sx, q.w_scale[m], b));
    }
}

// Sums of n columns over rows [first, last) of a block's share; 256 columns a
// block, eight rows at a time.
struct ColumnSum {
    const unsigned short* dy;
    int64_t ld;               // elements
    int64_t rows, out, share; // rows of one share
    float* part;              // [shares][out]
};
template <int DT>
__global__ __launch_bounds__(256) void column_sum_kernel(const ColumnSum q) {
    __shared__ float s_sum[8][256];
    const int col = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 256 + col * 8;
    const int64_t first = blockIdx.y * q.share, last = first + q.share < q.rows ? first + q.share : q.rows;
    float sum[8] = {};
    #pragma unroll 4
    for (int64_t r = first + row; r < last; r += 8) {
        const u32x4 w = row_piece(q.dy + r * q.ld, d, q.out);
        float x[8];
        decode4<DT>(u32x2{w.x, w.y}, x);
        decode4<DT>(u32x2{w.z, w.w}, x + 4);
        #pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += x[e];
    }
    #pragma unroll
    for (int e = 0; e < 8; ++e) s_sum[row][col * 8 + e] = sum[e];
    __syncthreads();
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (n >= q.out) return;
    float total = 0.0f;
    #pragma unroll
    for (int r = 0; r < 8; ++r) total += s_sum[r][threadIdx.x];
    q.part[blockIdx.y * q.out + n] = total;
}
template <int DT>
__global__ __launch_bounds__(256) void column_join_kernel(const float* __restrict__ part, int shares, int64_t out,
                                                          unsigned short* __restrict__ db) {
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (n >= out) return;
    float total = 0.0f;
    for (int i = 0; i < shares; ++i) total += part[i * out + n];
    db[n] = pack1<DT>(total);
}

// The slices' sum in 16 bits; slices in order.
template <int DT>
__global__ __launch_bounds__(256) void slice_sum_kernel(const float* __restrict__ slabs, int n_slabs, int64_t slab,
                                                        int64_t rows, int64_t dim, int64_t ld,
                                                        unsigned short* __restrict__ out, int64_t out_stride) {
    typedef u32x2 quad __attribute__((aligned(2)));
    const int64_t quads = ld / 4;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < rows * quads;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = at / quads, d = (at - r * quads) * 4;
        if (d >= dim) continue;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < n_slabs; ++s) x += *reinterpret_cast<const f32x4*>(slabs + s * slab + r * ld + d);
        unsigned short* o = out + r * out_stride + d;
        if (d + 4 <= dim) {
            *reinterpret_cast<quad*>(o) = u32x2{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])};
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < dim) o[e] = pack1<DT>(x[e]);
        }
    }
}

// ------------------------------------------------------------------ launches
constexpr int64_t kMaxTokens = int64_t(1) << 20, kMaxOut = int64_t(1) << 20;
constexpr int64_t kFewTokens = 64;            // few8_kernel's rule
constexpr size_t kPieceBytes = size_t(512) << 20;

// How a gradient is cut: by the three sizes alone.
struct Cut {
    int64_t piece;            // columns of dim at a time, a multiple of 256
    int32_t dx_slices, dw_slices;
    int32_t shares;           // of db's sum
    size_t x_bytes, w_bytes, dy_bytes, slab_bytes, part_bytes;
    size_t total;
};

bool cut(int64_t tokens, int64_t dim, int64_t out, Cut* c) {
    if (tokens < 0 || tokens > kMaxTokens || dim < 0 || dim > ZERO_ROWS8_MAX_DIM || out < 0 || out > kMaxOut)
        return false;
    const int64_t t = tokens > 0 ? tokens : 1, k = up(dim > 0 ? dim : 1, 256), n = out > 0 ? out : 1;
    int64_t piece = static_cast<int64_t>(kPieceBytes / (2 * static_cast<size_t>(t + n))) / 256 * 256;
    c->piece = piece < 256 ? 256 : (piece > k ? k : piece);
    // slices of the sum where the tiles of 128 x 128 alone would leave CUs idle
    const int64_t dim_tiles = c->piece / 128;
    auto slices = [](int64_t tiles, int64_t sum) {
        int64_t s = 512 / tiles;
        if (s > sum / 512) s = sum / 512;
        return static_cast<int32_t>(s < 1 ? 1 : (s > 64 ? 64 : s));
    };
    c->dx_slices = slices(dim_tiles * (up(t, 128) / 128), n);
    c->dw_slices = slices(dim_tiles * (up(n, 128) / 128), t);
    const int64_t columns = up(n, 256) / 256;
    int64_t shares = 1024 / columns;
    if (shares > t / 64) shares = t / 64;
    c->shares = static_cast<int32_t>(shares < 1 ? 1 : shares);
    c->x_bytes = round_up(static_cast<size_t>(t * c->piece) * 2, 256);
    c->w_bytes = round_up(static_cast<size_t>(n * c->piece) * 2, 256);
    c->dy_bytes = round_up(static_cast<size_t>(t * up(n, 64)) * 2, 256);
    const size_t dx_slab = c->dx_slices > 1 ? static_cast<size_t>(c->dx_slices) * t * c->piece * 4 : 0;
    const size_t dw_slab = c->dw_slices > 1 ? static_cast<size_t>(c->dw_slices) * n * c->piece * 4 : 0;
    c->slab_bytes = round_up(dx_slab > dw_slab ? dx_slab : dw_slab, 256);
    c->part_bytes = round_up(static_cast<size_t>(c->shares) * n * 4, 256);
    c->total = c->x_bytes + c->w_bytes + c->dy_bytes + c->slab_bytes + c->part_bytes;
    return true;
}

template <int OT>
int forward(const zero_linear8_args* a, hipStream_t st) {
    const int64_t k = ZERO_ROWS8_BYTES(a->dim);
    if (a->tokens <= kFewTokens) {
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
        const dim3 grid(static_cast<unsigned>((a->out + 15) / 16));
        if (a->tokens <= 16) hipLaunchKernelGGL((few8_kernel<OT, 1>), grid, dim3(256), 0, st, q);
        else if (a->tokens <= 32) hipLaunchKernelGGL((few8_kernel<OT, 2>), grid, dim3(256), 0, st, q);
        else hipLaunchKernelGGL((few8_kernel<OT, 4>), grid, dim3(256), 0, st, q);
        return launch_error("product kernel launch");
    }
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
    launch_product<kCodes, kRows, kRows, OT == ZERO_BF16 ? kScaledBf16 : kScaledFp16>(q, 1, st);
    return launch_error("product kernel launch");
}

// C = A B over k, in slices where there are more than one.
template <int DT, Layout LB>
void gradient(Product q, int slices, int64_t rows, int64_t dim, float* slabs, int64_t ld, void* out, int64_t out_stride,
              hipStream_t st) {
    if (slices > 1) {
        q.slice = static_cast<int32_t>(up(up(q.k, slices) / slices, kTileK));
        q.c = reinterpret_cast<char*>(slabs);
        q.ldc = ld;
        q.slab = rows * ld;
        // tiles times slices are at most 512 of 128 x 128, one round of the chip
        launch_tiles<DT, kCols, LB, kPart, 128, 128, 2, 2>(q, slices, st);
        hipLaunchKernelGGL((slice_sum_kernel<DT>), dim3(blocks_for(rows * (ld / 4))), dim3(256), 0, st, slabs, slices,
                           q.slab, rows, dim, ld, static_cast<unsigned short*>(out), out_stride);
        return;
    }
    q.slice = static_cast<int32_t>(up(q.k, kTileK));
    q.c = static_cast<char*>(out);
    q.ldc = out_stride;
    q.valid_m = static_cast<int32_t>(dim);
    launch_product<DT, kCols, LB, kPlain>(q, 1, st);
}

template <int DT>
int backward(const zero_linear8_args* a, const Cut& c, hipStream_t st) {
    char* ws = static_cast<char*>(a->workspace);
    char* x16 = ws;
    char* w16 = x16 + c.x_bytes;
    char* dyr = w16 + c.w_bytes;
    float* slabs = reinterpret_cast<float*>(dyr + c.dy_bytes);
    float* part = reinterpret_cast<float*>(dyr + c.dy_bytes + c.slab_bytes);
    const int64_t t = a->tokens, n = a->out;
    if (a->db && n > 0) {
        const ColumnSum q = {static_cast<const unsigned short*>(a->dy), a->dy_stride, t, n,
                             up(up(t, c.shares) / c.shares, 8), part};
        const unsigned blocks = static_cast<unsigned>(up(n, 256) / 256);
        hipLaunchKernelGGL((column_sum_kernel<DT>), dim3(blocks, c.shares), dim3(256), 0, st, q);
        hipLaunchKernelGGL((column_join_kernel<DT>), dim3(blocks), dim3(256), 0, st, part, c.shares, n,
                           static_cast<unsigned short*>(a->db));
    }
    const bool want_dx = a->dx && t > 0, want_dw = a->dw && n > 0;
    if (a->dim == 0 || (!want_dx && !want_dw)) return launch_error("product gradient kernel launch");
    // no row or no column: nothing of dy is read
    Matrix dy = {dyr, 128, 0};
    if (t > 0 && n > 0) dy = prepared(a->dy, a->dy_stride, 0, t, n, up(n, 64), dyr, st);
    for (int64_t d = 0; d < a->dim; d += c.piece) {
        const int64_t wide = a->dim - d < c.piece ? a->dim - d : c.piece;
        Product q = {};
        q.lda = c.piece * 2;
        q.m = static_cast<int32_t>(up(wide, 8));
        q.b = dy.p;
        q.ldb = dy.stride;
        int rc;
        if (want_dx) {
            if ((rc = zero_rows8_decode(static_cast<const char*>(a->w8) + d, a->w8_stride, a->w_scale, n, wide, w16,
                                        c.piece, DT, st)))
                return rc;
            q.a = w16;
            q.n = static_cast<int32_t>(t);
            q.k = static_cast<int32_t>(n);
            gradient<DT, kRows>(q, c.dx_slices, t, wide, slabs, c.piece, static_cast<unsigned short*>(a->dx) + d,
                                a->dx_stride, st);
        }
        if (want_dw) {
            if ((rc = zero_rows8_decode(static_cast<const char*>(a->x8) + d, a->x8_stride, a->x_scale, t, wide, x16,
                                        c.piece, DT, st)))
                return rc;
            q.a = x16;
            q.n = static_cast<int32_t>(n);
            q.k = static_cast<int32_t>(t);
            gradient<DT, kCols>(q, c.dw_slices, n, wide, slabs, c.piece, static_cast<unsigned short*>(a->dw) + d,
                                a->dw_stride, st);
        }
    }
    return launch_error("product gradient kernel launch");
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

size_t zero_linear8_workspace_bytes(int64_t tokens, int64_t dim, int64_t out) {
    Cut c;
    return cut(tokens, dim, out, &c) ? c.total : 0;
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
    Cut c;
    cut(a->tokens, a->dim, a->out, &c);
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a->dtype == ZERO_BF16 ? backward<ZERO_BF16>(a, c, st) : backward<ZERO_FP16>(a, c, st);
}

}  // extern "C"
