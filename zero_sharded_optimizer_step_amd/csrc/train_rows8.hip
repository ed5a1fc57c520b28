// train_rows8.hip -- rows of 8-bit codes and the gated activation that keeps
// its input in them (include/zero/train.h).
//
// All of it streams: what bounds a large call is HBM.  A row's scale needs
// its largest magnitude, so the encoders hold a row in registers between the
// maximum and the codes (a row longer than 16384 is read twice, the second
// time from the caches); the readers need no row at a time.
#include <hip/hip_runtime.h>

#include "train_internal.h"
#include "zero_device.h"

namespace zero {
namespace {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Elements of a row that a lane loads at a time: 16 bytes, so that lanes lie
// one behind the other.
template <int DT>
constexpr int kPiece = DT == ZERO_FP32 ? 4 : 8;

// ------------------------------------------------------------------- scales
// A row's largest magnitude is taken on the bits: they order as the values
// do, and an infinity or a NaN is above every number.
template <int DT>
constexpr uint32_t kInfinity = DT == ZERO_FP16 ? 0x7C00u : (DT == ZERO_BF16 ? 0x7F80u : 0x7F800000u);

struct Scale {
    float s, inv;             // 2^e and 2^-e; s is NaN where the row is not finite
    bool bad, edge;           // edge: e is the highest, a number may round to 128
};

template <int DT>
__device__ __forceinline__ Scale scale_of(uint32_t top) {
    constexpr int kLow = DT == ZERO_FP16 ? -24 : -126, kHigh = DT == ZERO_FP16 ? 9 : 121;
    uint32_t bits = top;
    if constexpr (DT != ZERO_FP32) bits = __float_as_uint(lo_to_f32<DT>(top));
    // the exponent of the top less 6, one more from 127.5 / 64 on
    int e = static_cast<int>((bits + 0x10000u) >> 23) - 127 - 6;
    e = e < kLow ? kLow : (e > kHigh ? kHigh : e);
    Scale r;
    r.bad = top >= kInfinity<DT>;
    r.edge = e == kHigh;
    r.s = r.bad ? __builtin_nanf("") : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    r.inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    return r;
}

// Four codes.  1.5 * 2^23 added to a number of [-127, 127] rounds it to
// nearest even and leaves it, in two's complement, in the low byte; x / 2^e
// is exact, so the multiply-add rounds the same.
__device__ __forceinline__ unsigned code4(const float x[4], const Scale& k) {
    unsigned b[4];
    #pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(__builtin_fmaf(x[e], k.inv, 12582912.0f));
    if (k.edge) {
        #pragma unroll
        for (int e = 0; e < 4; ++e)
            b[e] = __float_as_uint(__builtin_amdgcn_fmed3f(x[e] * k.inv, -127.0f, 127.0f) + 12582912.0f);
    }
    const unsigned lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const unsigned hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

__device__ __forceinline__ void value4(unsigned codes, float s, float o[4]) {
    #pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = static_cast<float>(static_cast<int8_t>(codes >> (8 * e))) * s;
}

// -------------------------------------------------------------------- pieces
// All of it is read and written once: past the caches' own order of keeping,
// a large call leaves to them what its caller has there.  Of 8192 x 16384 in
// bf16 the gated forward takes 165 us so and 182 without, its backward 168 and
// 186; 16384 x 4096 encoded 37.7 and 38.9, read back 37.1 and 38.9.
template <typename T>
__device__ __forceinline__ void put(void* at, T v) {
    __builtin_nontemporal_store(v, static_cast<T*>(at));
}
template <typename T, bool kOnce>
__device__ __forceinline__ T get(const void* at) {
    if constexpr (kOnce) return __builtin_nontemporal_load(static_cast<const T*>(at));
    else return *static_cast<const T*>(at);
}

template <int DT>
struct Piece {
    u32x4 w;
    typedef u32x4 piece __attribute__((aligned(2)));
    template <bool kOnce>
    __device__ __forceinline__ void load(const void* row, int64_t d, int64_t dim) {
        const unsigned short* s = static_cast<const unsigned short*>(row);
        w = d + 8 <= dim ? get<piece, kOnce>(s + d) : row_piece(s, d, dim);
    }
    __device__ __forceinline__ void values(float o[8]) const {
        decode4<DT>(u32x2{w.x, w.y}, o);
        decode4<DT>(u32x2{w.z, w.w}, o + 4);
    }
    // the larger of `so_far` and this piece's magnitudes, two at a time
    __device__ __forceinline__ uint32_t top(uint32_t so_far) const {
        u16x2 t = __builtin_bit_cast(u16x2, so_far);
        #pragma unroll
        for (int e = 0; e < 4; ++e) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, w[e] & 0x7FFF7FFFu));
        return __builtin_bit_cast(uint32_t, t);
    }
    static __device__ __forceinline__ uint32_t one(uint32_t t) { return t >> 16 > (t & 0xFFFFu) ? t >> 16 : t & 0xFFFFu; }
    __device__ __forceinline__ void round(const float o[8]) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack2<DT>(o[2 * e], o[2 * e + 1]);
    }
    // the same bits, which the compiler takes for others
    __device__ __forceinline__ void hide() {
        uint32_t a = w.x, b = w.y, c = w.z, d = w.w;
        asm volatile("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
        w = u32x4{a, b, c, d};
    }
    // elements [d, d + 8) of a row of any alignment, up to dim
    __device__ __forceinline__ void store(void* row, int64_t d, int64_t dim) const {
        unsigned short* o = static_cast<unsigned short*>(row) + d;
        if (d + 8 <= dim) {
            put<piece>(o, w);
        } else {
            #pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d + e < dim) o[e] = static_cast<unsigned short>(w[e / 2] >> (16 * (e % 2)));
        }
    }
};

template <>
struct Piece<ZERO_FP32> {
    f32x4 w;
    typedef f32x4 piece __attribute__((aligned(4)));
    template <bool kOnce>
    __device__ __forceinline__ void load(const void* row, int64_t d, int64_t dim) {
        const float* s = static_cast<const float*>(row);
        if (d + 4 <= dim) {
            w = get<piece, kOnce>(s + d);
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = d + e < dim ? s[d + e] : 0.0f;
        }
    }
    __device__ __forceinline__ void values(float o[4]) const {
        #pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = w[e];
    }
    __device__ __forceinline__ uint32_t top(uint32_t t) const {
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t b = __float_as_uint(w[e]) & 0x7FFFFFFFu;
            t = b > t ? b : t;
        }
        return t;
    }
    static __device__ __forceinline__ uint32_t one(uint32_t t) { return t; }
    __device__ __forceinline__ void round(const float o[4]) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = o[e];
    }
    __device__ __forceinline__ void store(void* row, int64_t d, int64_t dim) const {
        float* o = static_cast<float*>(row) + d;
        if (d + 4 <= dim) {
            put<piece>(o, w);
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < dim) o[e] = w[e];
        }
    }
};

// A piece's codes, 4 or 8 bytes; rows of codes are whole pieces up to a
// multiple of 16 past dim, zeros there.
template <int DT>
struct Codes {
    static constexpr int kWords = kPiece<DT> / 4;
    typedef unsigned int words __attribute__((ext_vector_type(kWords)));
    words c;
    __device__ __forceinline__ void load(const char* row, int64_t d, int64_t dim) {
        c = d < dim ? get<words, true>(row + d) : words(0u);
    }
    __device__ __forceinline__ void values(float s, float o[4 * kWords]) const {
        #pragma unroll
        for (int i = 0; i < kWords; ++i) value4(c[i], s, o + 4 * i);
    }
};
template <int DT>
__device__ __forceinline__ void store_codes(const Piece<DT>& p, const Scale& k, char* row, int64_t d) {
    typedef typename Codes<DT>::words words;
    float x[kPiece<DT>];
    p.values(x);
    words c;
    #pragma unroll
    for (int i = 0; i < Codes<DT>::kWords; ++i) c[i] = code4(x + 4 * i, k);
    put<words>(row + d, k.bad ? words(0u) : c);
}

// The largest of N values over the TR threads of a row.  Two buffers in turn
// (`turn`), so one barrier serves a row: a wave that writes one of them again
// has passed the barrier of the row between, as every reader had before it.
template <int TR, int N>
__device__ __forceinline__ void row_max(uint32_t (&t)[N], int turn) {
    static_assert(TR <= 64 || TR >= 256, "a wave has whole rows, or a row the whole block");
    #pragma unroll
    for (int off = (TR < 64 ? TR : 64) / 2; off > 0; off >>= 1)
        #pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t u = __shfl_xor(t[i], off, 64);
            t[i] = u > t[i] ? u : t[i];
        }
    if constexpr (TR > 64) {
        constexpr int kWaves = TR / 64;
        __shared__ uint32_t s_top[2][N][kWaves];
        if ((threadIdx.x & 63) == 0)
            #pragma unroll
            for (int i = 0; i < N; ++i) s_top[turn][i][threadIdx.x / 64] = t[i];
        __syncthreads();
        #pragma unroll
        for (int i = 0; i < N; ++i)
            #pragma unroll
            for (int w = 0; w < kWaves; ++w) t[i] = s_top[turn][i][w] > t[i] ? s_top[turn][i][w] : t[i];
    }
}

// How the threads of a block share rows: TR threads a row, P pieces each.
template <int TR>
constexpr int kThreads = TR < 256 ? 256 : TR;
template <int TR>
constexpr int kRowsABlock = kThreads<TR> / TR;

// ------------------------------------------------------------------- encode
struct Encode {
    const char* x;
    int64_t x_row;            // bytes
    int64_t rows, dim;
    char* codes;
    int64_t codes_row;
    float* scale;
};

template <int DT, int TR, int P, bool kHeld>
__global__ __launch_bounds__(kThreads<TR>) void rows8_encode_kernel(const Encode q) {
    const int t = threadIdx.x % TR;
    const int64_t end = (q.dim + 15) / 16 * 16;
    int turn = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRowsABlock<TR> + threadIdx.x / TR; r < q.rows;
         r += static_cast<int64_t>(gridDim.x) * kRowsABlock<TR>, turn ^= 1) {
        const char* x = q.x + r * q.x_row;
        char* codes = q.codes + r * q.codes_row;
        Piece<DT> p[P];
        uint32_t top[1] = {0u};
        for (int64_t base = 0; base < end; base += TR * P * kPiece<DT>) {
            #pragma unroll
            for (int i = 0; i < P; ++i) p[i].template load<kHeld>(x, base + (i * TR + t) * kPiece<DT>, q.dim);
            #pragma unroll
            for (int i = 0; i < P; ++i) top[0] = p[i].top(top[0]);
            if (kHeld) break;
        }
        top[0] = Piece<DT>::one(top[0]);
        row_max<TR>(top, turn);
        const Scale k = scale_of<DT>(top[0]);
        if (t == 0) q.scale[r] = k.s;
        for (int64_t base = 0; base < end; base += TR * P * kPiece<DT>) {
            #pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t d = base + (i * TR + t) * kPiece<DT>;
                if (!kHeld) p[i].template load<false>(x, d, q.dim);
                if (d < end) store_codes(p[i], k, codes, d);
            }
            if (kHeld) break;
        }
    }
}

// ------------------------------------------------------------------- decode
struct Decode {
    const char* codes;
    int64_t codes_row;
    const float* scale;
    int64_t rows, dim;
    char* y;
    int64_t y_row;            // bytes
    uint32_t parts;           // blocks of one row
};

template <int DT, int TR, int P>
__global__ __launch_bounds__(256) void rows8_decode_kernel(const Decode q) {
    const int t = threadIdx.x % TR;
    const uint32_t across = blockIdx.x % q.parts;
    const int64_t first = static_cast<int64_t>(across) * (TR * P * kPiece<DT>);
    for (int64_t r = static_cast<int64_t>(blockIdx.x / q.parts) * kRowsABlock<TR> + threadIdx.x / TR; r < q.rows;
         r += static_cast<int64_t>(gridDim.x / q.parts) * kRowsABlock<TR>) {
        const float s = q.scale[r];
        const char* codes = q.codes + r * q.codes_row;
        char* y = q.y + r * q.y_row;
        Codes<DT> c[P];
        #pragma unroll
        for (int i = 0; i < P; ++i) c[i].load(codes, first + (i * TR + t) * kPiece<DT>, q.dim);
        #pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t d = first + (i * TR + t) * kPiece<DT>;
            float o[kPiece<DT>];
            c[i].values(s, o);
            Piece<DT> p;
            p.round(o);
            if (d < q.dim) p.store(y, d, q.dim);
        }
    }
}

// --------------------------------------------------------- gated activation
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kGelu = 1.59576912160573071176f;      // 2 sqrt(2 / pi)
constexpr float kCubic = 0.044715f;

// act(x) = x p and act'(x).  exp2 and rcp are the instructions' (1 ulp each),
// far inside the half step of 16 bits that follows.  Both give 0 for results
// below 2^-126, where x p is a normal bf16 for another 2^7; with kLow p is
// 2^-z there, as far as fp32 has it, and the same bits everywhere else.  It
// costs 3 % where it runs for all, so rows that have no such gate go without:
// far_gate().  Of 8192 x 16384 silu's gated forward takes 171 us either way on
// values of a normal distribution and 162 and 169 on rows that all have far
// gates; alone 97 and 105, gelu's alone 100 and 115.
// Beyond 16 gelu's p is 0 or 1 in fp32, so its argument stops there: no power
// of a large x overflows.  A NaN x gives NaN.
template <int KIND, bool kLow>
struct Act {
    float x, p, square;
    __device__ __forceinline__ explicit Act(float v) : x(v) {
        float z = -kLog2e * v;
        if constexpr (KIND == ZERO_GLU_GELU) {
            const float c = __builtin_amdgcn_fmed3f(v, -16.0f, 16.0f);
            square = c * c;
            z = c * __builtin_fmaf(square, -kLog2e * kGelu * kCubic, -kLog2e * kGelu);
        }
        p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z));
        if constexpr (kLow) p = z > 125.0f ? __builtin_amdgcn_exp2f(64.0f - z) * 0x1p-64f : p;
    }
    __device__ __forceinline__ float value() const { return x * p; }
    __device__ __forceinline__ float slope() const {
        if constexpr (KIND == ZERO_GLU_SILU) return p * __builtin_fmaf(x, 1.0f - p, 1.0f);
        else return __builtin_fmaf(x * p * (1.0f - p), __builtin_fmaf(square, 3.0f * kCubic * kGelu, kGelu), p);
    }
};

// Below this z may be more than 125: silu's is 124.1 there, gelu's 117.9.
template <int KIND>
constexpr float kFarGate = KIND == ZERO_GLU_SILU ? -86.0f : -9.75f;
// May a gate of this wave's, whose magnitudes are at most `most`, be that low?
// NaN may stand for any.  fp16 has no result that small.
template <int DT, int KIND>
__device__ __forceinline__ bool far_gate(float most) {
    return DT == ZERO_BF16 && __builtin_amdgcn_ballot_w64(!(most < -kFarGate<KIND>)) != 0;
}

struct Glu {
    int64_t tokens, width;
    // bytes from row to row
    int64_t gate_row, up_row, h_row, dh_row, dgate_row, dup_row, gate8_row, up8_row, h8_row;
    const char *gate, *up;
    char *gate8, *up8, *h, *h8;
    float *gate_scale, *up_scale, *h_scale;
    const char* dh;
    char *dgate, *dup;
    uint32_t parts;           // the backward: blocks of one row
};

template <int DT, int KIND, bool kGated, int TR, int P, bool kHeld>
__global__ __launch_bounds__(kThreads<TR>) void glu8_forward_kernel(const Glu q) {
    constexpr int U = kGated ? P : 1;
    const int t = threadIdx.x % TR;
    const int64_t end = (q.width + 15) / 16 * 16;
    int turn = 0;
    int64_t r = static_cast<int64_t>(blockIdx.x) * kRowsABlock<TR> + threadIdx.x / TR;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsABlock<TR>;
    Piece<DT> g[P], u[U], h[P];
    auto load = [&](Piece<DT> (&to_g)[P], Piece<DT> (&to_u)[U], int64_t row, int64_t base) __attribute__((always_inline)) -> void {
        #pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t d = base + (i * TR + t) * kPiece<DT>;
            to_g[i].template load<kHeld>(q.gate + row * q.gate_row, d, q.width);
            if constexpr (kGated) to_u[i].template load<kHeld>(q.up + row * q.up_row, d, q.width);
        }
    };
    auto act = [&](int i, auto low) __attribute__((always_inline)) -> void {
        float x[8], o[8];
        g[i].values(x);
        #pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = Act<KIND, decltype(low)::value>(x[e]).value();
        if constexpr (kGated) {
            u[i].values(x);
            #pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= x[e];
        }
        h[i].round(o);
    };
    // `top`: of the gates' magnitudes
    auto far = [&](uint32_t top) __attribute__((always_inline)) -> bool {
        return far_gate<DT, KIND>(lo_to_f32<DT>(Piece<DT>::one(top)));
    };
    for (; r < q.tokens; r += step, turn ^= 1) {
        uint32_t top[kGated ? 3 : 2] = {};
        for (int64_t base = 0; base < end; base += TR * P * kPiece<DT>) {
            load(g, u, r, base);
            const uint32_t before = top[1];
            #pragma unroll
            for (int i = 0; i < P; ++i) {
                act(i, std::false_type{});
                top[0] = g[i].top(top[0]);
                top[1] = h[i].top(top[1]);
                if constexpr (kGated) top[2] = u[i].top(top[2]);
            }
            // once more, so that what most rows take has no branch among its loads
            // (with one a piece silu alone takes 108 us of 8192 x 16384, for 97)
            if (far(top[0])) {
                top[1] = before;
                #pragma unroll
                for (int i = 0; i < P; ++i) {
                    // nothing of the first time is kept for this: it would take another block's registers
                    g[i].hide();
                    if constexpr (kGated) u[i].hide();
                    act(i, std::true_type{});
                    top[1] = h[i].top(top[1]);
                }
            }
            if (kHeld) break;
        }
        #pragma unroll
        for (uint32_t& x : top) x = Piece<DT>::one(x);
        if (q.gate8 || q.h8) row_max<TR>(top, turn);
        const Scale kg = scale_of<DT>(top[0]), kh = scale_of<DT>(top[1]);
        Scale ku = kg;
        if constexpr (kGated) ku = scale_of<DT>(top[2]);
        if (t == 0) {
            if (q.gate8) q.gate_scale[r] = kg.s;
            if (q.h8) q.h_scale[r] = kh.s;
            if (kGated && q.gate8) q.up_scale[r] = ku.s;
        }
        [[maybe_unused]] const bool again = !kHeld && far(top[0]);
        for (int64_t base = 0; base < end; base += TR * P * kPiece<DT>) {
            if constexpr (!kHeld) load(g, u, r, base);
            #pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t d = base + (i * TR + t) * kPiece<DT>;
                if constexpr (!kHeld) {
                    if (again) act(i, std::true_type{});
                    else act(i, std::false_type{});
                }
                if (d >= end) continue;
                if (q.gate8) {
                    store_codes(g[i], kg, q.gate8 + r * q.gate8_row, d);
                    if constexpr (kGated) store_codes(u[i], ku, q.up8 + r * q.up8_row, d);
                }
                if (q.h8) store_codes(h[i], kh, q.h8 + r * q.h8_row, d);
                if (q.h) h[i].store(q.h + r * q.h_row, d, q.width);
            }
            if (kHeld) break;
        }
    }
}

// dgate or dup may be dh's own memory: a thread has read its piece before it
// writes there.
template <int DT, int KIND, bool kGated, int TR, int P>
__global__ __launch_bounds__(256) void glu8_backward_kernel(const Glu q) {
    const int t = threadIdx.x % TR;
    const uint32_t across = blockIdx.x % q.parts;
    const int64_t first = static_cast<int64_t>(across) * (TR * P * kPiece<DT>);
    for (int64_t r = static_cast<int64_t>(blockIdx.x / q.parts) * kRowsABlock<TR> + threadIdx.x / TR; r < q.tokens;
         r += static_cast<int64_t>(gridDim.x / q.parts) * kRowsABlock<TR>) {
        const float sg = q.gate_scale[r], su = kGated ? q.up_scale[r] : 1.0f;
        const bool far = far_gate<DT, KIND>(128.0f * __builtin_fabsf(sg));
        const char *gate8 = q.gate8 + r * q.gate8_row, *up8 = kGated ? q.up8 + r * q.up8_row : nullptr;
        const char* dh = q.dh + r * q.dh_row;
        Piece<DT> p[P];
        Codes<DT> cg[P], cu[P];
        #pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t d = first + (i * TR + t) * kPiece<DT>;
            p[i].template load<true>(dh, d, q.width);
            cg[i].load(gate8, d, q.width);
            if constexpr (kGated) cu[i].load(up8, d, q.width);
        }
        #pragma unroll
        for (int i = 0; i < P; ++i) {
            const int64_t d = first + (i * TR + t) * kPiece<DT>;
            float g[8], u[8], x[8], dg[8], du[8];
            p[i].values(x);
            cg[i].values(sg, g);
            if constexpr (kGated) cu[i].values(su, u);
            auto gradients = [&](auto low) __attribute__((always_inline)) -> void {
                #pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const Act<KIND, decltype(low)::value> a(g[e]);
                    dg[e] = x[e] * a.slope();
                    if constexpr (kGated) {
                        dg[e] *= u[e];
                        du[e] = x[e] * a.value();
                    }
                }
            };
            if (far) gradients(std::true_type{});
            else gradients(std::false_type{});
            if (d >= q.width) continue;
            Piece<DT> o;
            o.round(dg);
            o.store(q.dgate + r * q.dgate_row, d, q.width);
            if constexpr (kGated) {
                o.round(du);
                o.store(q.dup + r * q.dup_row, d, q.width);
            }
        }
    }
}

// ------------------------------------------------------------------ launches
int launched(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(ZERO_EDEVICE, "%s: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

constexpr int64_t kMostBlocks = 1 << 20;      // times 1024 threads fit the grid's 32 bits

// Blocks along the rows, of `parts` blocks each.
template <int TR>
unsigned row_blocks(int64_t rows, int64_t parts = 1) {
    const int64_t b = (rows + kRowsABlock<TR> - 1) / kRowsABlock<TR>, most = kMostBlocks / parts;
    return static_cast<unsigned>(b < most ? b : most);
}

// The threads and pieces of a row for the encoders, by its length: the fewest
// that hold it.  Microseconds, and with those of the next longer rows, bf16:
// 100000 x 128 encoded 10.0 and 27, 50000 x 128 gated forward 12.7 and 35; 65536
// x 512 24.5 and 30, 32768 x 512 26.7 and 43; 16384 x 2048 19.1 and 23.9, 8192 x
// 2048 24.7 and 28.0; 16384 x 4096 37.6 and 38.5, 8192 x 4096 42 and 53; 8192 x
// 8192 36.5 and 36.4, 4096 x 8192 44 and 56; 4096 x 16384 37.5 and 55 (as rows
// read twice), 2048 x 16384 45 and 76.  Of 16384 elements 512 threads hold two
// parts, gate and up (8192 rows forward 163 us; 256, with 236 registers each,
// 175), and 256 one (4096 rows of gelu 64.5 us, 512 72).
// Short rows, one load a wave between maximum and codes, reach 3.6 to 4.1 TB/s
// (200000 x 64, 65536 x 512, 16384 x 1024).  Rows past 16384 are read twice: 2000
// x 40000 59.5 us (4.0 TB/s), 4096 x 28672 gated forward 197 (4.2).
template <int DT, int kParts, typename F>
void by_row(int64_t dim, const F& f) {
    using std::integral_constant;
    constexpr int kMore = 8 / kPiece<DT>;
    const int64_t eights = (dim + 15) / 16 * 2;
    if (eights <= 16) f(integral_constant<int, 8>{}, integral_constant<int, 2 * kMore>{}, std::true_type{});
    else if (eights <= 64) f(integral_constant<int, 64>{}, integral_constant<int, kMore>{}, std::true_type{});
    else if (eights <= 256) f(integral_constant<int, 64>{}, integral_constant<int, 4 * kMore>{}, std::true_type{});
    else if (eights <= 512) f(integral_constant<int, 256>{}, integral_constant<int, 2 * kMore>{}, std::true_type{});
    else if (eights <= 1024) f(integral_constant<int, 256>{}, integral_constant<int, 4 * kMore>{}, std::true_type{});
    else if (eights <= 2048) f(integral_constant<int, 256 * kParts>{}, integral_constant<int, 8 / kParts * kMore>{}, std::true_type{});
    else f(integral_constant<int, 1024>{}, integral_constant<int, 4 * kMore>{}, std::false_type{});
}
// And for the readers, whose blocks take part of a row.  Microseconds, bf16,
// with 8 and 64 threads a row: 200000 x 64 read back 9.6 and 37, 100000 x 64 gated
// gradient 12.6 and 52; with 64 and 256: 65536 x 512 20.5 and 44, 32768 x 512 25
// and 61, 16384 x 4096 36.4 and 35.5, 8192 x 4096 plain gradient 38 and 31.7.
// From 513 to about 2048 elements, where 256 threads have less than a piece each
// to do, 64 are the faster, which the rule does not take: 32768 x 600 18.9 and
// 27.3, 16384 x 600 gated gradient 22 and 37, 8192 x 1024 14.3 and 20.6, x 2048
// 25.0 and 27.3.
template <int DT, typename F>
void by_piece(int64_t dim, const F& f) {
    using std::integral_constant;
    constexpr int kMore = 8 / kPiece<DT>;
    const int64_t eights = (dim + 15) / 16 * 2;
    if (eights <= 8) f(integral_constant<int, 8>{}, integral_constant<int, kMore>{});
    else if (eights <= 64) f(integral_constant<int, 64>{}, integral_constant<int, kMore>{});
    else f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
}
template <int DT, int TR, int P>
unsigned row_parts(int64_t dim) {
    constexpr int kWide = TR * P * kPiece<DT>;
    return static_cast<unsigned>((dim + kWide - 1) / kWide);
}

template <int DT>
void encode(const Encode& q, hipStream_t st) {
    by_row<DT, 1>(q.dim, [&](auto tr, auto p, auto held) {
        constexpr int TR = decltype(tr)::value, P = decltype(p)::value;
        hipLaunchKernelGGL((rows8_encode_kernel<DT, TR, P, decltype(held)::value>), dim3(row_blocks<TR>(q.rows)),
                           dim3(kThreads<TR>), 0, st, q);
    });
}

template <int DT>
void decode(Decode q, hipStream_t st) {
    by_piece<DT>(q.dim, [&](auto tr, auto p) {
        constexpr int TR = decltype(tr)::value, P = decltype(p)::value;
        q.parts = row_parts<DT, TR, P>(q.dim);
        hipLaunchKernelGGL((rows8_decode_kernel<DT, TR, P>), dim3(row_blocks<TR>(q.rows, q.parts) * q.parts), dim3(256), 0,
                           st, q);
    });
}

template <int DT, int KIND, bool kGated>
void glu_forward(const Glu& q, hipStream_t st) {
    by_row<DT, kGated ? 2 : 1>(q.width, [&](auto tr, auto p, auto held) {
        constexpr int TR = decltype(tr)::value, P = decltype(p)::value;
        hipLaunchKernelGGL((glu8_forward_kernel<DT, KIND, kGated, TR, P, decltype(held)::value>),
                           dim3(row_blocks<TR>(q.tokens)), dim3(kThreads<TR>), 0, st, q);
    });
}
template <int DT, int KIND, bool kGated>
void glu_backward(Glu q, hipStream_t st) {
    by_piece<DT>(q.width, [&](auto tr, auto p) {
        constexpr int TR = decltype(tr)::value, P = decltype(p)::value;
        q.parts = row_parts<DT, TR, P>(q.width);
        hipLaunchKernelGGL((glu8_backward_kernel<DT, KIND, kGated, TR, P>),
                           dim3(row_blocks<TR>(q.tokens, q.parts) * q.parts), dim3(256), 0, st, q);
    });
}

template <typename F>
void by_kind(const zero_glu8_args* a, bool gated, const F& f) {
    using std::integral_constant;
    auto kinds = [&](auto dt) {
        auto gates = [&](auto kind) {
            if (gated) f(dt, kind, std::true_type{});
            else f(dt, kind, std::false_type{});
        };
        if (a->kind == ZERO_GLU_SILU) gates(integral_constant<int, ZERO_GLU_SILU>{});
        else gates(integral_constant<int, ZERO_GLU_GELU>{});
    };
    if (a->dtype == ZERO_BF16) kinds(integral_constant<int, ZERO_BF16>{});
    else kinds(integral_constant<int, ZERO_FP16>{});
}

Glu glu_of(const zero_glu8_args* a) {
    Glu q;
    q.tokens = a->tokens;
    q.width = a->width;
    q.gate_row = a->gate_stride * 2;
    q.up_row = a->up_stride * 2;
    q.h_row = a->h_stride * 2;
    q.dh_row = a->dh_stride * 2;
    q.dgate_row = a->dgate_stride * 2;
    q.dup_row = a->dup_stride * 2;
    q.gate8_row = a->gate8_stride;
    q.up8_row = a->up8_stride;
    q.h8_row = a->h8_stride;
    q.gate = static_cast<const char*>(a->gate);
    q.up = static_cast<const char*>(a->up);
    q.gate8 = static_cast<char*>(a->gate8);
    q.up8 = static_cast<char*>(a->up8);
    q.h = static_cast<char*>(a->h);
    q.h8 = static_cast<char*>(a->h8);
    q.gate_scale = a->gate_scale;
    q.up_scale = a->up_scale;
    q.h_scale = a->h_scale;
    q.dh = static_cast<const char*>(a->dh);
    q.dgate = static_cast<char*>(a->dgate);
    q.dup = static_cast<char*>(a->dup);
    q.parts = 1;
    return q;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

int zero_rows8_encode(const void* x, int64_t x_stride, int32_t dtype, int64_t rows, int64_t dim, void* codes,
                      int64_t codes_stride, float* scale, void* stream) {
    clear_error();
    const int rc = check_rows8(x, x_stride, dtype, rows, dim, codes, codes_stride, scale);
    if (rc || rows == 0) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Encode q = {static_cast<const char*>(x), x_stride * (dtype == ZERO_FP32 ? 4 : 2), rows, dim,
                      static_cast<char*>(codes), codes_stride, scale};
    if (dtype == ZERO_BF16) encode<ZERO_BF16>(q, st);
    else if (dtype == ZERO_FP16) encode<ZERO_FP16>(q, st);
    else encode<ZERO_FP32>(q, st);
    return launched("row encode kernel launch");
}

int zero_rows8_decode(const void* codes, int64_t codes_stride, const float* scale, int64_t rows, int64_t dim, void* y,
                      int64_t y_stride, int32_t dtype, void* stream) {
    clear_error();
    const int rc = check_rows8(y, y_stride, dtype, rows, dim, codes, codes_stride, scale);
    if (rc || rows == 0 || dim == 0) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const Decode q = {static_cast<const char*>(codes), codes_stride, scale, rows, dim,
                      static_cast<char*>(y), y_stride * (dtype == ZERO_FP32 ? 4 : 2), 1};
    if (dtype == ZERO_BF16) decode<ZERO_BF16>(q, st);
    else if (dtype == ZERO_FP16) decode<ZERO_FP16>(q, st);
    else decode<ZERO_FP32>(q, st);
    return launched("row decode kernel launch");
}

int zero_glu8_forward(const zero_glu8_args* a, void* stream) {
    clear_error();
    const int rc = check_glu8_args(a, false);
    if (rc || a->tokens == 0 || a->width == 0) return rc;
    const Glu q = glu_of(a);
    hipStream_t st = static_cast<hipStream_t>(stream);
    by_kind(a, a->up != nullptr, [&](auto dt, auto kind, auto gated) {
        glu_forward<decltype(dt)::value, decltype(kind)::value, decltype(gated)::value>(q, st);
    });
    return launched("gated activation kernel launch");
}

int zero_glu8_backward(const zero_glu8_args* a, void* stream) {
    clear_error();
    const int rc = check_glu8_args(a, true);
    if (rc || a->tokens == 0 || a->width == 0) return rc;
    const Glu q = glu_of(a);
    hipStream_t st = static_cast<hipStream_t>(stream);
    by_kind(a, a->up8 != nullptr, [&](auto dt, auto kind, auto gated) {
        glu_backward<decltype(dt)::value, decltype(kind)::value, decltype(gated)::value>(q, st);
    });
    return launched("gated activation gradient kernel launch");
}

}  // extern "C"
