// train_tensors.hip -- AdamW over a list of tensors with 32-bit or 8-bit
// states, and the conversion between the two (include/zero/train.h).
//
// All of it streams: per element the update reads the gradient twice (norm,
// update) and the state once, and writes the state, with about 25 flops
// (about 60 with the 8-bit codes), so HBM is the bound and the kernels keep
// every access wide, touch every stream once and launch one thread per quad
// of 4 elements.  A chunk is 1024 elements of one tensor; the table maps it
// to its tensor with two scalar loads, so a list of any sizes runs as one
// launch per pass.
#include <hip/hip_runtime.h>

#include "train_internal.h"
#include "zero_device.h"

namespace zero {
namespace {

// Vectors at an element's alignment: a packed list starts tensors anywhere,
// and gfx950 takes such global accesses as one instruction (a wave's quads
// are still one contiguous run, so only the run's two end lines are shared).
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// The table's pointers are device memory, which the compiler cannot see:
// said here, it uses global instead of flat accesses.
#define ZERO_GLOBAL(T, p) ((__attribute__((address_space(1))) T*)(p))

// Read through the scalar cache; nothing writes it while the kernel runs.
#define ZERO_CONSTANT(T, p) ((const __attribute__((address_space(4))) T*)(p))

template <int DT> struct GradQuad { typedef u32x2 T; typedef u32x2_any U; };
template <> struct GradQuad<ZERO_FP32> { typedef f32x4 T; typedef f32x4_any U; };

template <int DT>
__device__ __forceinline__ void widen_quad(const typename GradQuad<DT>::T v, float o[4]) {
    if constexpr (DT == ZERO_FP32) {
        o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
    } else {
        decode4<DT>(v, o);
    }
}

// Quads of elements [e, e + 4) of n: whole where `full`, else the elements
// there are, the rest 0.  What is loaded stays as it lies until it is used,
// so that a thread's loads are all in flight together.
template <int DT>
__device__ __forceinline__ typename GradQuad<DT>::T load_grad(const void* base, int64_t e, int64_t n, bool full) {
    typename GradQuad<DT>::T o = {};
    if constexpr (DT == ZERO_FP32) {
        const float* p = static_cast<const float*>(base) + e;
        if (full) {
            o = *ZERO_GLOBAL(const f32x4_any, p);
        } else {
            #pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k < n) o[k] = ZERO_GLOBAL(const float, p)[k];
        }
    } else {
        const unsigned short* p = static_cast<const unsigned short*>(base) + e;
        if (full) {
            o = *ZERO_GLOBAL(const u32x2_any, p);
        } else {
            #pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k < n)
                    o[k / 2] |= static_cast<unsigned>(ZERO_GLOBAL(const unsigned short, p)[k]) << (16 * (k % 2));
        }
    }
    return o;
}
__device__ __forceinline__ f32x4 load_f32(const float* base, int64_t e, int64_t n, bool full) {
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if (full) {
        o = __builtin_nontemporal_load(ZERO_GLOBAL(const f32x4_any, base + e));
    } else {
        #pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + k < n) o[k] = ZERO_GLOBAL(const float, base)[e + k];
    }
    return o;
}
__device__ __forceinline__ void store_f32(float* base, int64_t e, int64_t n, bool full, const f32x4 x) {
    if (full) {
        __builtin_nontemporal_store(x, ZERO_GLOBAL(f32x4_any, base + e));
    } else {
        #pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + k < n) ZERO_GLOBAL(float, base)[e + k] = x[k];
    }
}
template <int DT>
__device__ __forceinline__ void store_16(void* base, int64_t e, int64_t n, bool full, const f32x4 x) {
    unsigned short* p = static_cast<unsigned short*>(base) + e;
    if (full) {
        u32x2 o;
        o.x = pack2<DT>(x.x, x.y);
        o.y = pack2<DT>(x.z, x.w);
        __builtin_nontemporal_store(o, ZERO_GLOBAL(u32x2_any, p));
    } else {
        #pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + k < n) ZERO_GLOBAL(unsigned short, p)[k] = pack1<DT>(x[k]);
    }
}

// ------------------------------------------------------------ the 8-bit state
// A code is the top bits of an fp32 number moved so that the block's
// exponent E becomes the exponent field B (15 or 31): the code's 3 fraction
// bits are fp32's top 3, its exponent field fp32's, and fp32's subnormals
// give the format's gradual underflow.  Moving is v_ldexp_f32 (one rounding,
// to nearest even, only where the result is subnormal), rounding is an add
// below bit 20.
constexpr int kFieldM = 15, kFieldV = 31;

__device__ __forceinline__ float code_value(uint32_t code, uint32_t sign, int e, int field) {
    return __builtin_ldexpf(__uint_as_float((code << 20) | sign), e - field);
}
__device__ __forceinline__ float decode_m(uint32_t c, int e) {
    return code_value(c & 127u, (c & 128u) << 24, e, kFieldM);
}
__device__ __forceinline__ float decode_v(uint32_t c, int e) { return code_value(c, 0u, e, kFieldV); }

// Largest of the wave's 64 values (bits of fp32 numbers >= 0; a negative
// one counts as 0), in every lane.
__device__ __forceinline__ int wave_max(int x) {
#define ZERO_DPP_MAX(CTRL, ROWS)                                                       \
    {                                                                                  \
        const int y = __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);       \
        x = x > y ? x : y;                                                             \
    }
    ZERO_DPP_MAX(0x111, 0xf)      // row_shr:1, 2, 4, 8: lane 15 of each row of 16
    ZERO_DPP_MAX(0x112, 0xf)
    ZERO_DPP_MAX(0x114, 0xf)
    ZERO_DPP_MAX(0x118, 0xf)
    ZERO_DPP_MAX(0x142, 0xa)      // row_bcast:15 into rows 1 and 3
    ZERO_DPP_MAX(0x143, 0xc)      // row_bcast:31 into rows 2 and 3
#undef ZERO_DPP_MAX
    return __builtin_amdgcn_readlane(x, 63);
}
// Biased exponent of a block from the bits of its largest magnitude: one
// more above mantissa 1.875, which is the largest a code holds.
__device__ __forceinline__ int block_exponent(int top) {
    const int e = (top + 0xFFFFF) >> 23;
    return e < 1 ? 1 : (e > 254 ? 254 : e);
}

// NEAREST rounds to nearest even; otherwise noise (16 random bits, centred
// in a step of 2^20) decides.
template <bool NEAREST>
__device__ __forceinline__ uint32_t encode(float x, int e, int field, uint32_t noise) {
    const int bits = __float_as_int(__builtin_ldexpf(x, field - e));
    const int add = NEAREST ? ((bits >> 20) & 1) + 0x7FFFF : static_cast<int>((noise << 4) + 8);
    const int c = (bits + add) >> 20;
    const int top = 8 * field + 7;
    return static_cast<uint32_t>(c < 0 ? 0 : (c > top ? top : c));
}
template <bool NEAREST>
__device__ __forceinline__ uint32_t encode_m(float m, int e, uint32_t noise) {
    const uint32_t c = encode<NEAREST>(__builtin_fabsf(m), e, kFieldM, noise);
    return c | (c > 0 && __float_as_int(m) < 0 ? 128u : 0u);
}
template <bool NEAREST>
__device__ __forceinline__ uint32_t encode_v(float v, int e, uint32_t noise) {
    const uint32_t c = encode<NEAREST>(v, e, kFieldV, noise);
    return v > 0.0f && c < 1u ? 1u : c;
}

// The 32-bit finalizer of MurmurHash3 (public domain).
__device__ __forceinline__ uint32_t fmix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x85EBCA6Bu;
    x ^= x >> 13;
    x *= 0xC2B2AE35u;
    return x ^ (x >> 16);
}

// Encodes a wave's block: each lane holds 4 elements of it.  `place` is the
// hash input of the lane's first element.
template <bool NEAREST>
__device__ __forceinline__ void encode_block(const f32x4 m, const f32x4 v, uint32_t place, uint32_t key,
                                             unsigned char* state, unsigned char* scale) {
    int tm = 0, tv = 0;
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int a = __float_as_int(m[k]) & 0x7fffffff, b = __float_as_int(v[k]);
        tm = tm > a ? tm : a;
        tv = tv > b ? tv : b;
    }
    const int em = block_exponent(wave_max(tm)), ev = block_exponent(wave_max(tv));
    uint32_t cm = 0, cv = 0;
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t h = NEAREST ? 0u : fmix32((place + k) * 0x9E3779B1u + key);
        cm |= encode_m<NEAREST>(m[k], em, h & 0xffffu) << (8 * k);
        cv |= encode_v<NEAREST>(v[k], ev, h >> 16) << (8 * k);
    }
    const int lane = threadIdx.x & 63;
    auto* s = ZERO_GLOBAL(uint32_t, state);
    __builtin_nontemporal_store(cm, s + lane);
    __builtin_nontemporal_store(cv, s + 64 + lane);
    if (lane == 0)
        *ZERO_GLOBAL(unsigned short, scale) = static_cast<unsigned short>(em | (ev << 8));
}

// One wave per block; the block past the last element is padded with zeros.
__global__ __launch_bounds__(256) void state8_encode_kernel(const float* __restrict__ m,
                                                            const float* __restrict__ v, int64_t n,
                                                            unsigned char* __restrict__ state,
                                                            unsigned char* __restrict__ scale) {
    const int64_t b = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (b * ZERO_STATE8_BLOCK >= n) return;            // whole waves
    const int64_t e = b * ZERO_STATE8_BLOCK + (threadIdx.x & 63) * 4;
    const bool full = e + 4 <= n;
    const f32x4 mq = load_f32(m, e, n, full), vq = load_f32(v, e, n, full);
    encode_block<true>(mq, vq, 0, 0, state + b * 512, scale + b * 2);
}

// A lane writes 16 bytes to each of the two outputs: a wave takes one block
// in fp32, two in 16 bits (with 8 bytes a lane there, the 13B/8 shard's bf16
// moments take 1.79 ms instead of 1.60, 6.1 TB/s).
template <int DT>
constexpr int kDecodeLane = DT == ZERO_FP32 ? 4 : 8;   // elements
template <int DT>
__global__ __launch_bounds__(256) void state8_decode_kernel(const unsigned char* __restrict__ state,
                                                            const unsigned char* __restrict__ scale,
                                                            int64_t n, void* __restrict__ m,
                                                            void* __restrict__ v) {
    constexpr int kLane = kDecodeLane<DT>;
    typedef uint32_t codes __attribute__((ext_vector_type(kLane / 4)));
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * kLane;
    if (e >= n) return;
    const int64_t b = e / ZERO_STATE8_BLOCK;
    const unsigned char* at = state + b * 512 + e % ZERO_STATE8_BLOCK;
    const codes cm = __builtin_nontemporal_load(reinterpret_cast<const codes*>(at));
    const codes cv = __builtin_nontemporal_load(reinterpret_cast<const codes*>(at + ZERO_STATE8_BLOCK));
    const unsigned es = *reinterpret_cast<const unsigned short*>(scale + b * 2);
    const int em = es & 255, ev = es >> 8;
    f32x4 mq[kLane / 4], vq[kLane / 4];
    #pragma unroll
    for (int k = 0; k < kLane; ++k) {
        mq[k / 4][k % 4] = decode_m((cm[k / 4] >> (8 * (k % 4))) & 255u, em);
        vq[k / 4][k % 4] = decode_v((cv[k / 4] >> (8 * (k % 4))) & 255u, ev);
    }
    if constexpr (DT == ZERO_FP32) {
        const bool full = e + kLane <= n;
        store_f32(static_cast<float*>(m), e, n, full, mq[0]);
        store_f32(static_cast<float*>(v), e, n, full, vq[0]);
    } else if (e + kLane <= n) {
        auto store = [e](void* base, const f32x4 (&x)[kLane / 4]) {
            const u32x4 o = {pack2<DT>(x[0].x, x[0].y), pack2<DT>(x[0].z, x[0].w), pack2<DT>(x[1].x, x[1].y),
                             pack2<DT>(x[1].z, x[1].w)};
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<unsigned short*>(base) + e));
        };
        store(m, mq);
        store(v, vq);
    } else {
        #pragma unroll
        for (int h = 0; h < kLane / 4; ++h) {
            store_16<DT>(m, e + 4 * h, n, false, mq[h]);
            store_16<DT>(v, e + 4 * h, n, false, vq[h]);
        }
    }
}

// ------------------------------------------------------------------ the norm
// At most kFoldBlocks blocks of 1024 threads walk the chunks together, 8
// chunks a block and kNormUnroll such runs in flight, so what is in flight
// stays one compact window; each block leaves one entry of a partials slot.
// A wave takes half a chunk, 8 elements a lane.  All loads of a round are
// issued before any is used: a half chunk that ends inside reads the table
// instead, and its elements are taken one by one afterwards.  Every sum has
// a fixed order.
constexpr int kNormThreads = 1024;
constexpr int kNormRun = 8;                           // chunks of a block at a time
constexpr int kNormUnroll = 8;
constexpr int kHalf = kChunk / 2;
static_assert(kNormThreads * 8 == kNormRun * kChunk, "8 elements a thread");

template <int DT>
__global__ __launch_bounds__(kNormThreads) void tensors_norm_kernel(
    const TensorRec* __restrict__ recs, const uint32_t* __restrict__ map, int64_t n_chunks,
    float inv_scale, const zero_tensors_scalars_t* __restrict__ sc, unsigned char* __restrict__ slot) {
    constexpr int kWords = DT == ZERO_FP32 ? 2 : 1;    // 16-byte loads of 8 elements
    typedef u32x4 words __attribute__((aligned(2)));
    if (sc) inv_scale = sc->inv_scale;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int lane = threadIdx.x & 63;
    const int64_t round = static_cast<int64_t>(gridDim.x) * kNormRun;
    double ss = 0.0;
    int bad = 0;
    auto add = [&](float x) {
        const float g = x * inv_scale;
        bad |= !finite(g);
        ss += static_cast<double>(g) * static_cast<double>(g);
    };
    for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * kNormRun + wave / 2; c0 < n_chunks;
         c0 += round * kNormUnroll) {
        const char* base[kNormUnroll];
        int64_t left[kNormUnroll];                     // elements from this half chunk's first on
        u32x4 x[kNormUnroll][kWords];
        // in three sweeps, so that the scalar loads of a sweep overlap
        uint32_t owner[kNormUnroll];
        #pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const int64_t c = c0 + u * round;
            owner[u] = map[c < n_chunks ? c : n_chunks - 1];
        }
        int64_t numel[kNormUnroll], first[kNormUnroll];
        #pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const TensorRec& r = recs[owner[u]];
            base[u] = static_cast<const char*>(r.grad);
            numel[u] = r.numel;
            first[u] = r.first_chunk;
        }
        #pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const int64_t c = c0 + u * round;
            const int64_t e = (c - first[u]) * kChunk + (wave & 1) * kHalf;
            base[u] += e * (DT == ZERO_FP32 ? 4 : 2);
            left[u] = c < n_chunks ? numel[u] - e : 0;
        }
        #pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            const char* at = left[u] >= kHalf ? base[u] + lane * (16 * kWords) : reinterpret_cast<const char*>(recs);
            #pragma unroll
            for (int w = 0; w < kWords; ++w) x[u][w] = *ZERO_GLOBAL(const words, at + 16 * w);
        }
        #pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            if (left[u] >= kHalf) {
                #pragma unroll
                for (int w = 0; w < kWords; ++w)
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (DT == ZERO_FP32) {
                            add(__uint_as_float(x[u][w][k]));
                        } else {
                            add(lo_to_f32<DT>(x[u][w][k]));
                            add(hi_to_f32<DT>(x[u][w][k]));
                        }
                    }
            } else {
                for (int64_t i = lane; i < left[u]; i += 64) {
                    if constexpr (DT == ZERO_FP32) add(ZERO_GLOBAL(const float, base[u])[i]);
                    else add(lo_to_f32<DT>(ZERO_GLOBAL(const unsigned short, base[u])[i]));
                }
            }
        }
    }
    block_reduce<kNormThreads>(ss, bad);
    if (threadIdx.x == 0) {
        SlotHeader* h = reinterpret_cast<SlotHeader*>(slot);
        Partial* out = reinterpret_cast<Partial*>(h + 1);
        out[blockIdx.x].sumsq = ss;
        out[blockIdx.x].flag = bad;
        out[blockIdx.x].pad = 0;
        if (blockIdx.x == 0) h->n_blocks = static_cast<int32_t>(gridDim.x);
    }
}

// The list's result from its slot, by one block of 256 threads, for all of
// them.
static_assert(kFoldBlocks <= kChunkThreads, "one entry a thread");
__device__ __forceinline__ zero_global_t fold_slot(const unsigned char* __restrict__ slot,
                                                   const zero_tensors_scalars_t& k,
                                                   const zero_tensors_scalars_t* __restrict__ sc) {
    const SlotHeader* h = reinterpret_cast<const SlotHeader*>(slot);
    const Partial* p = reinterpret_cast<const Partial*>(h + 1);
    const int nb = h->n_blocks;
    double ss = 0.0;
    int bad = 0;
    if (static_cast<int>(threadIdx.x) < nb && threadIdx.x < kFoldBlocks) {
        ss = p[threadIdx.x].sumsq;
        bad = p[threadIdx.x].flag;
    }
    block_reduce<kChunkThreads>(ss, bad);
    __shared__ double s_total;
    __shared__ int s_any;
    if (threadIdx.x == 0) {
        s_total = ss;
        s_any = bad;
    }
    __syncthreads();
    ss = s_total;
    bad = s_any;
    double peer = k.peer_sumsq, max_norm = k.max_grad_norm;
    int peer_bad = k.peer_overflow;
    if (sc) {
        const auto* d = ZERO_CONSTANT(zero_tensors_scalars_t, sc);
        peer = d->peer_sumsq;
        max_norm = d->max_grad_norm;
        peer_bad = d->peer_overflow;
    }
    ss += peer;
    bad |= peer_bad;
    zero_global_t o;
    o.sumsq = ss;
    o.norm = sqrt(ss);
    const double c = max_norm / (o.norm + 1e-6);
    o.clipped = (max_norm > 0.0 && c < 1.0) ? 1 : 0;
    o.coef = o.clipped ? static_cast<float>(c) : 1.0f;
    o.overflow = (bad || !__builtin_isfinite(ss)) ? 1 : 0;
    o.reserved = 0;
    return o;
}

__global__ __launch_bounds__(kChunkThreads) void tensors_combine_kernel(
    const unsigned char* __restrict__ slot, zero_tensors_scalars_t k,
    const zero_tensors_scalars_t* __restrict__ sc, zero_global_t* __restrict__ out) {
    const zero_global_t o = fold_slot(slot, k, sc);
    if (threadIdx.x == 0) *out = o;
}

// ---------------------------------------------------------------- the update
// One thread per quad, one wave per block of an 8-bit state.  With FOLD the
// block joins the norm's partials itself (4 KB from L2, behind its loads)
// instead of reading a result that a launch in between made.
template <int GT, int PT, int BITS, bool FOLD>
__global__ __launch_bounds__(kChunkThreads) void tensors_apply_kernel(
    const TensorRec* __restrict__ recs, const uint32_t* __restrict__ map, int64_t last_chunk,
    const zero_global_t* __restrict__ glob, const unsigned char* __restrict__ slot, zero_tensors_scalars_t k,
    const zero_tensors_scalars_t* __restrict__ sc, zero_global_t* __restrict__ result) {
    if constexpr (!FOLD) {
        if (glob->overflow) return;                    // skipped step: touch nothing
    }
    // from the end of the list: what the norm pass read last may still be
    // in the last-level cache
    const int64_t chunk = last_chunk - static_cast<int64_t>(blockIdx.x);
    const TensorRec& r = recs[map[chunk]];
    const auto& kg = k.group[r.group];
    AdamConsts c = {kg.decay, kg.beta1, kg.one_minus_beta1, kg.beta2, kg.one_minus_beta2, kg.step_size,
                    kg.inv_sqrt_bc2, kg.eps};
    float inv_scale = k.inv_scale;
    uint32_t key = k.key;
    if (sc) {                                          // the step's scalars in device memory
        const auto* d = ZERO_CONSTANT(zero_tensors_scalars_t, sc);
        const auto& dg = d->group[r.group];
        c = {dg.decay, dg.beta1, dg.one_minus_beta1, dg.beta2, dg.one_minus_beta2, dg.step_size,
             dg.inv_sqrt_bc2, dg.eps};
        inv_scale = d->inv_scale;
        key = d->key;
    }
    const int64_t in_tensor = (chunk - r.first_chunk) * kChunk;
    const int64_t e = in_tensor + threadIdx.x * kQuad;
    const int64_t n = r.numel;
    const bool full = e + kQuad <= n;
    // a wave with no element; within FOLD it still joins the block's fold
    const bool idle = in_tensor + (threadIdx.x & ~63u) * kQuad >= n;
    if constexpr (!FOLD) {
        if (idle) return;
    }
    typename GradQuad<GT>::T gq = {};
    f32x4 p = {}, m = {}, v = {};
    uint32_t cm = 0, cv = 0, es = 0;
    const int lane = threadIdx.x & 63;
    const int64_t b = in_tensor / ZERO_STATE8_BLOCK + (threadIdx.x >> 6);
    unsigned char* state = static_cast<unsigned char*>(r.m) + b * 512;
    unsigned char* scale = static_cast<unsigned char*>(r.v) + b * 2;
    if (!idle) {
        gq = load_grad<GT>(r.grad, e, n, full);
        p = load_f32(r.master, e, n, full);
        if constexpr (BITS == 32) {
            m = load_f32(static_cast<const float*>(r.m), e, n, full);
            v = load_f32(static_cast<const float*>(r.v), e, n, full);
        } else {
            const auto* s = ZERO_GLOBAL(const uint32_t, state);
            cm = __builtin_nontemporal_load(s + lane);
            cv = __builtin_nontemporal_load(s + 64 + lane);
            es = *ZERO_GLOBAL(const unsigned short, scale);
        }
    }
    float coef;
    if constexpr (FOLD) {
        const zero_global_t o = fold_slot(slot, k, sc);
        if (blockIdx.x == 0 && threadIdx.x == 0) *result = o;
        if (idle || o.overflow) return;
        coef = o.coef;
    } else {
        coef = glob->coef;
    }
    if constexpr (BITS == 8) {
        const int em = es & 255, ev = es >> 8;
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = decode_m((cm >> (8 * j)) & 255u, em);
            v[j] = decode_v((cv >> (8 * j)) & 255u, ev);
        }
    }
    float g[4];
    widen_quad<GT>(gq, g);
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
        float pe = p[j], me = m[j], ve = v[j];
        adamw1((g[j] * inv_scale) * coef, pe, me, ve, c);
        p[j] = pe; m[j] = me; v[j] = ve;
    }
    store_f32(r.master, e, n, full, p);
    if constexpr (BITS == 32) {
        store_f32(static_cast<float*>(r.m), e, n, full, m);
        store_f32(static_cast<float*>(r.v), e, n, full, v);
    } else {
        // padding stays zero: its gradient and codes are
        const uint32_t place = (r.first_block + static_cast<uint32_t>(b)) * ZERO_STATE8_BLOCK + lane * kQuad;
        encode_block<false>(m, v, place, key, state, scale);
    }
    if constexpr (PT != 0) store_16<PT>(r.param, e, n, full, p);
}

// ------------------------------------------------------------------ launches
int launch_error(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(ZERO_EDEVICE, "%s: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

// Chunks of one launch: a grid holds fewer than 2^32 threads.
constexpr int64_t kLaunchChunks = int64_t(1) << 23;
static_assert(kLaunchChunks * kChunkThreads < (int64_t(1) << 32), "threads of one launch");

// Up to here the update's blocks are all on the chip at once, so each joining
// the norm's partials costs about a microsecond once, less than the launch of
// a kernel that joins them (2 us and the gap before it).
constexpr int64_t kFoldChunks = 2048;

struct Table {
    const TensorRec* recs;
    const uint32_t* map;
    int64_t n_chunks;
};
Table table_of(const zero_tensors_args* a) {
    const unsigned char* t = static_cast<const unsigned char*>(a->table);
    return {reinterpret_cast<const TensorRec*>(t),
            reinterpret_cast<const uint32_t*>(t + table_map_offset(a->plan.n_tensors)), a->plan.n_chunks};
}

int launch_norm(const zero_tensors_args* a, const zero_tensors_scalars_t& k, unsigned char* slot, hipStream_t st) {
    const Table t = table_of(a);
    int64_t blocks = (t.n_chunks + kNormRun - 1) / kNormRun;
    blocks = blocks < 1 ? 1 : (blocks > kFoldBlocks ? kFoldBlocks : blocks);
#define ZERO_NORM(DT)                                                                                    \
    hipLaunchKernelGGL((tensors_norm_kernel<DT>), dim3(static_cast<unsigned>(blocks)), dim3(kNormThreads), 0, \
                       st, t.recs, t.map, t.n_chunks, k.inv_scale, a->scalars, slot)
    switch (a->plan.grad_dtype) {
        case ZERO_BF16: ZERO_NORM(ZERO_BF16); break;
        case ZERO_FP16: ZERO_NORM(ZERO_FP16); break;
        default: ZERO_NORM(ZERO_FP32); break;
    }
#undef ZERO_NORM
    return launch_error("list norm kernel launch");
}

// Where the update finds the step's result: already joined in glob, or (glob
// NULL) as the partials of `slot`, which it then joins and writes to result.
struct Found {
    const zero_global_t* glob;
    const unsigned char* slot;
    zero_global_t* result;
};

template <int GT, int PT, int BITS>
void launch_apply_types(const zero_tensors_args* a, const zero_tensors_scalars_t& k, const Found& f, hipStream_t st) {
    const Table t = table_of(a);
    for (int64_t last = t.n_chunks - 1; last >= 0; last -= kLaunchChunks) {
        const dim3 grid(static_cast<unsigned>(last + 1 < kLaunchChunks ? last + 1 : kLaunchChunks));
        if (f.glob)
            hipLaunchKernelGGL((tensors_apply_kernel<GT, PT, BITS, false>), grid, dim3(kChunkThreads), 0, st, t.recs,
                               t.map, last, f.glob, f.slot, k, a->scalars, f.result);
        else
            hipLaunchKernelGGL((tensors_apply_kernel<GT, PT, BITS, true>), grid, dim3(kChunkThreads), 0, st, t.recs,
                               t.map, last, f.glob, f.slot, k, a->scalars, f.result);
    }
}

template <int GT, int PT>
void launch_apply_bits(const zero_tensors_args* a, const zero_tensors_scalars_t& k, const Found& f, hipStream_t st) {
    if (a->plan.state_bits == 8) launch_apply_types<GT, PT, 8>(a, k, f, st);
    else launch_apply_types<GT, PT, 32>(a, k, f, st);
}

template <int GT>
void launch_apply_grad(const zero_tensors_args* a, const zero_tensors_scalars_t& k, const Found& f, hipStream_t st) {
    switch (a->plan.param_dtype) {
        case ZERO_BF16: launch_apply_bits<GT, ZERO_BF16>(a, k, f, st); break;
        case ZERO_FP16: launch_apply_bits<GT, ZERO_FP16>(a, k, f, st); break;
        default: launch_apply_bits<GT, 0>(a, k, f, st); break;
    }
}

int launch_apply(const zero_tensors_args* a, const zero_tensors_scalars_t& k, const Found& f, hipStream_t st) {
    if (a->plan.n_chunks == 0) return ZERO_OK;
    switch (a->plan.grad_dtype) {
        case ZERO_BF16: launch_apply_grad<ZERO_BF16>(a, k, f, st); break;
        case ZERO_FP16: launch_apply_grad<ZERO_FP16>(a, k, f, st); break;
        default: launch_apply_grad<ZERO_FP32>(a, k, f, st); break;
    }
    return launch_error("list update kernel launch");
}

int check_state8(const void* m, const void* v, int64_t n, const void* state8, const void* scale8) {
    if (n < 0) return fail(ZERO_EINVAL, "n %lld < 0", (long long)n);
    if (n == 0) return ZERO_OK;
    if (!m || !v || !state8 || !scale8) return fail(ZERO_EINVAL, "a required pointer is NULL");
    if (!aligned16(m) || !aligned16(v) || !aligned16(state8))
        return fail(ZERO_EALIGN, "m, v or state8 is not 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(scale8) & 1u) return fail(ZERO_EALIGN, "scale8 is not 2-byte aligned");
    return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

int zero_state8_encode(const float* m, const float* v, int64_t n, void* state8, void* scale8, void* stream) {
    clear_error();
    const int rc = check_state8(m, v, n, state8, scale8);
    if (rc || n == 0) return rc;
    unsigned char* s8 = static_cast<unsigned char*>(state8);
    unsigned char* e8 = static_cast<unsigned char*>(scale8);
    for (int64_t at = 0; at < n; at += kLaunchChunks * kChunk) {
        const int64_t len = n - at < kLaunchChunks * kChunk ? n - at : kLaunchChunks * kChunk;
        hipLaunchKernelGGL(state8_encode_kernel, dim3(static_cast<unsigned>((len + kChunk - 1) / kChunk)),
                           dim3(kChunkThreads), 0, static_cast<hipStream_t>(stream), m + at, v + at, len,
                           s8 + 2 * at, e8 + at / 128);
    }
    return launch_error("state encode kernel launch");
}

int zero_state8_decode(const void* state8, const void* scale8, int64_t n, void* m, void* v, int32_t dtype,
                       void* stream) {
    clear_error();
    if (dtype != ZERO_FP16 && dtype != ZERO_BF16 && dtype != ZERO_FP32)
        return fail(ZERO_EINVAL, "dtype %d is not ZERO_FP16, ZERO_BF16 or ZERO_FP32", dtype);
    const int rc = check_state8(m, v, n, state8, scale8);
    if (rc || n == 0) return rc;
    const unsigned char* s8 = static_cast<const unsigned char*>(state8);
    const unsigned char* e8 = static_cast<const unsigned char*>(scale8);
    const int size = dtype == ZERO_FP32 ? 4 : 2;
#define ZERO_DECODE(DT)                                                                                   \
    hipLaunchKernelGGL((state8_decode_kernel<DT>),                                                              \
                       dim3(static_cast<unsigned>((len + 256 * kDecodeLane<DT> - 1) / (256 * kDecodeLane<DT>))),     \
                       dim3(256), 0, static_cast<hipStream_t>(stream), s8 + 2 * at, e8 + at / 128,                   \
                       len, static_cast<char*>(m) + at * size, static_cast<char*>(v) + at * size)
    for (int64_t at = 0; at < n; at += kLaunchChunks * kChunk) {
        const int64_t len = n - at < kLaunchChunks * kChunk ? n - at : kLaunchChunks * kChunk;
        switch (dtype) {
            case ZERO_BF16: ZERO_DECODE(ZERO_BF16); break;
            case ZERO_FP16: ZERO_DECODE(ZERO_FP16); break;
            default: ZERO_DECODE(ZERO_FP32); break;
        }
    }
#undef ZERO_DECODE
    return launch_error("state decode kernel launch");
}

int zero_tensors_norm(const zero_tensors_args* a, int32_t slot, void* partials_dev, void* stream) {
    clear_error();
    zero_tensors_scalars_t k;
    const int rc = tensors_constants(a, false, false, &k);
    if (rc) return rc;
    if (slot < 0) return fail(ZERO_EINVAL, "slot %d < 0", slot);
    if (!partials_dev) return fail(ZERO_EINVAL, "partials_dev is NULL");
    if (!aligned16(partials_dev)) return fail(ZERO_EALIGN, "partials_dev is not 16-byte aligned");
    return launch_norm(a, k, static_cast<unsigned char*>(partials_dev) + static_cast<size_t>(slot) * kSlotBytes,
                       static_cast<hipStream_t>(stream));
}

int zero_tensors_apply(const zero_tensors_args* a, const void* global_dev, void* stream) {
    clear_error();
    zero_tensors_scalars_t k;
    const int rc = tensors_constants(a, false, false, &k);
    if (rc) return rc;
    if (!global_dev) return fail(ZERO_EINVAL, "global_dev is NULL");
    if (!aligned16(global_dev)) return fail(ZERO_EALIGN, "global_dev is not 16-byte aligned");
    return launch_apply(a, k, {static_cast<const zero_global_t*>(global_dev), nullptr, nullptr},
                        static_cast<hipStream_t>(stream));
}

int zero_tensors_step(const zero_tensors_args* a, zero_step_info* info, void* stream) {
    clear_error();
    zero_tensors_scalars_t k;
    int rc = tensors_constants(a, true, true, &k);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    unsigned char* slot = static_cast<unsigned char*>(a->workspace);
    if ((rc = launch_norm(a, k, slot, st))) return rc;
    if (a->plan.n_chunks > 0 && a->plan.n_chunks <= kFoldChunks) {
        if ((rc = launch_apply(a, k, {nullptr, slot, a->result}, st))) return rc;
    } else {
        hipLaunchKernelGGL(tensors_combine_kernel, dim3(1), dim3(kChunkThreads), 0, st, slot, k, a->scalars,
                           a->result);
        if ((rc = launch_error("list combine kernel launch"))) return rc;
        if ((rc = launch_apply(a, k, {a->result, nullptr, nullptr}, st))) return rc;
    }
    if (info) {
        hipError_t e = hipMemcpyAsync(info, a->result, sizeof(zero_global_t), hipMemcpyDeviceToHost, st);
        if (e == hipSuccess) e = hipStreamSynchronize(st);
        if (e != hipSuccess) return fail(ZERO_EDEVICE, "reading the step result: %s", hipGetErrorString(e));
    }
    return ZERO_OK;
}

}  // extern "C"
