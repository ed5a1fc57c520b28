// train_host.cpp -- host-only parts of libzero_train_mi355x.so: the plan of
// a tensor list, the step's constants and argument checks.  No HIP calls.
#include <cmath>
#include <cstring>

#include "train_internal.h"

namespace zero {

static bool finite_positive(double x) { return std::isfinite(x) && x > 0.0; }

static bool off(const void* p, unsigned align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

static int check_plan_types(int32_t state_bits, int32_t grad_dtype, int32_t param_dtype) {
    if (state_bits != 32 && state_bits != 8)
        return fail(ZERO_EINVAL, "state_bits %d is not 32 or 8", state_bits);
    if (grad_dtype != ZERO_FP16 && grad_dtype != ZERO_BF16 && grad_dtype != ZERO_FP32)
        return fail(ZERO_EINVAL, "grad_dtype %d is not ZERO_FP16, ZERO_BF16 or ZERO_FP32", grad_dtype);
    if (param_dtype != 0 && param_dtype != ZERO_FP16 && param_dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "param_dtype %d is not 0, ZERO_FP16 or ZERO_BF16", param_dtype);
    return ZERO_OK;
}

// MurmurHash3's 32-bit finalizer (public domain, by its published steps).
static uint32_t fmix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x85EBCA6Bu;
    x ^= x >> 13;
    x *= 0xC2B2AE35u;
    return x ^ (x >> 16);
}

int tensors_constants(const zero_tensors_args* a, bool peers, bool buffers, zero_tensors_scalars_t* k) {
    if (!a) return fail(ZERO_EINVAL, "args is NULL");
    const zero_tensors_plan_t& p = a->plan;
    int rc;
    if ((rc = check_plan_types(p.state_bits, p.grad_dtype, p.param_dtype))) return rc;
    // the size and the count of chunks bound each other, and a chunk is one
    // tensor's and holds an element; nothing here overflows
    if (p.n_tensors < 0 || p.numel < 0 || p.n_chunks < 0 || p.n_chunks > INT32_MAX ||
        p.numel > static_cast<int64_t>(INT32_MAX) * kChunk || (p.n_tensors == 0 && p.n_chunks > 0) ||
        p.n_chunks > p.numel || p.n_chunks < (p.numel + kChunk - 1) / kChunk ||
        p.n_chunks > p.numel / kChunk + p.n_tensors || p.n_groups < 1 ||
        p.n_groups > ZERO_MAX_GROUPS ||
        p.table_bytes != round_up(table_map_offset(p.n_tensors) + 4u * static_cast<size_t>(p.n_chunks), 16) ||
        p.workspace_bytes != kTensorsWorkspace)
        return fail(ZERO_EINVAL, "plan is not one that zero_tensors_plan fills");
    if (!a->groups) return fail(ZERO_EINVAL, "groups is NULL");
    if (a->n_groups < p.n_groups || a->n_groups > ZERO_MAX_GROUPS)
        return fail(ZERO_EINVAL, "n_groups %d outside [%d, %d]", a->n_groups, p.n_groups, ZERO_MAX_GROUPS);
    if (a->step < 1) return fail(ZERO_EINVAL, "step %lld < 1", (long long)a->step);
    if (!finite_positive(a->loss_scale)) return fail(ZERO_EINVAL, "loss_scale must be finite and > 0");
    if (!finite_positive(a->grad_predivide))
        return fail(ZERO_EINVAL, "grad_predivide must be finite and > 0");
    if (std::isnan(a->max_grad_norm)) return fail(ZERO_EINVAL, "max_grad_norm is NaN");
    std::memset(k, 0, sizeof *k);
    k->inv_scale = static_cast<float>(1.0 / (a->loss_scale * a->grad_predivide));
    const uint32_t high = fmix32(static_cast<uint32_t>(a->seed >> 32));
    k->key = static_cast<uint32_t>(a->seed) ^ high;
    k->max_grad_norm = a->max_grad_norm;
    for (int32_t i = 0; i < a->n_groups; ++i) {
        const zero_adam_group_t& g = a->groups[i];
        if (!std::isfinite(g.lr) || g.lr < 0.0) return fail(ZERO_EINVAL, "groups[%d].lr must be finite and >= 0", i);
        if (!(g.beta1 >= 0.0 && g.beta1 < 1.0)) return fail(ZERO_EINVAL, "groups[%d].beta1 outside [0, 1)", i);
        if (!(g.beta2 >= 0.0 && g.beta2 < 1.0)) return fail(ZERO_EINVAL, "groups[%d].beta2 outside [0, 1)", i);
        if (!finite_positive(g.eps)) return fail(ZERO_EINVAL, "groups[%d].eps must be finite and > 0", i);
        if (!std::isfinite(g.weight_decay)) return fail(ZERO_EINVAL, "groups[%d].weight_decay must be finite", i);
        const AdamConsts c = adam_consts(g.lr, g.beta1, g.beta2, g.eps, g.weight_decay, a->step);
        auto& o = k->group[i];
        o.decay = c.decay;
        o.beta1 = c.b1;
        o.one_minus_beta1 = c.c1;
        o.beta2 = c.b2;
        o.one_minus_beta2 = c.c2;
        o.step_size = c.step_size;
        o.inv_sqrt_bc2 = c.inv_sqrt_bc2;
        o.eps = c.eps;
    }
    if (!aligned16(a->scalars)) return fail(ZERO_EALIGN, "scalars is not 16-byte aligned");
    if (p.n_chunks > 0 && !a->table) return fail(ZERO_EINVAL, "table is NULL");
    if (!aligned16(a->table)) return fail(ZERO_EALIGN, "table is not 16-byte aligned");
    if (peers) {
        if (!(a->peer_sumsq >= 0.0)) return fail(ZERO_EINVAL, "peer_sumsq must be >= 0 (got NaN or negative)");
        k->peer_sumsq = a->peer_sumsq;
        k->peer_overflow = a->peer_overflow ? 1 : 0;
    }
    if (!buffers) return ZERO_OK;
    if (!a->workspace || !a->result) return fail(ZERO_EINVAL, "workspace or result is NULL");
    if (!aligned16(a->workspace) || !aligned16(a->result))
        return fail(ZERO_EALIGN, "workspace or result is not 16-byte aligned");
    if (a->workspace_bytes < p.workspace_bytes)
        return fail(ZERO_ESIZE, "workspace_bytes %zu < %llu needed", a->workspace_bytes,
                    (unsigned long long)p.workspace_bytes);
    return ZERO_OK;
}

int check_xent_args(const zero_xent_args* a, bool backward) {
    if (!a) return fail(ZERO_EINVAL, "args is NULL");
    if (a->tokens < 0 || a->dim < 0 || a->vocab < 0) return fail(ZERO_EINVAL, "a size is negative");
    const size_t need = zero_xent_workspace_bytes(a->tokens, a->dim, a->vocab);
    if (!need)
        return fail(ZERO_EINVAL, "tokens %lld, dim %lld, vocab %lld are out of range", (long long)a->tokens,
                    (long long)a->dim, (long long)a->vocab);
    if (a->dtype != ZERO_FP16 && a->dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "dtype %d is not ZERO_FP16 or ZERO_BF16", a->dtype);
    if (a->reserved != 0) return fail(ZERO_EINVAL, "reserved must be 0");
    if (!a->result) return fail(ZERO_EINVAL, "result is NULL");
    if (!aligned16(a->result)) return fail(ZERO_EALIGN, "result is not 16-byte aligned");
    // the kernels' row offsets: a row count times a stride stays in 63 bits
    const int64_t top = int64_t(1) << 31;
    if (a->x_stride < a->dim || a->w_stride < a->dim || a->x_stride > top || a->w_stride > top)
        return fail(ZERO_EINVAL, "x_stride or w_stride outside [dim, 2^31]");
    if (backward) {
        if (!std::isfinite(a->grad_scale)) return fail(ZERO_EINVAL, "grad_scale must be finite");
        if (a->dx_stride < a->dim || a->dw_stride < a->dim || a->dx_stride > top || a->dw_stride > top)
            return fail(ZERO_EINVAL, "dx_stride or dw_stride outside [dim, 2^31]");
        // dw is written even where there is no token
        if ((a->vocab > 0 && a->dim > 0 && !a->dw) || (a->tokens > 0 && a->dim > 0 && !a->dx))
            return fail(ZERO_EINVAL, "dx or dw is NULL");
        if (off(a->dx, 2) || off(a->dw, 2)) return fail(ZERO_EALIGN, "dx or dw is not 2-byte aligned");
    }
    if (a->tokens > 0) {
        if (!a->target || !a->lse || (!backward && !a->loss)) return fail(ZERO_EINVAL, "a token buffer is NULL");
        if (a->dim > 0 && (!a->x || !a->w)) return fail(ZERO_EINVAL, "x or w is NULL");
    }
    if (off(a->x, 2) || off(a->w, 2)) return fail(ZERO_EALIGN, "x or w is not 2-byte aligned");
    if (off(a->target, 8)) return fail(ZERO_EALIGN, "target is not 8-byte aligned");
    if (off(a->lse, 4) || off(a->loss, 4)) return fail(ZERO_EALIGN, "loss or lse is not 4-byte aligned");
    if (!a->workspace) return fail(ZERO_EINVAL, "workspace is NULL");
    if (off(a->workspace, 256)) return fail(ZERO_EALIGN, "workspace is not 256-byte aligned");
    if (a->workspace_bytes < need)
        return fail(ZERO_ESIZE, "workspace_bytes %zu < %zu needed", a->workspace_bytes, need);
    return ZERO_OK;
}

}  // namespace zero

using namespace zero;

extern "C" {

static_assert(sizeof(zero_tensors_scalars_t) == 288, "list scalars are 288 bytes");
static_assert(sizeof(zero_xent_result_t) == 32, "the loss result is 32 bytes");

int zero_tensors_plan(const zero_tensor_t* tensors, int32_t n_tensors, int32_t state_bits,
                      int32_t grad_dtype, int32_t param_dtype, void* table, size_t table_cap,
                      zero_tensors_plan_t* plan) {
    clear_error();
    if (!plan) return fail(ZERO_EINVAL, "plan is NULL");
    if (n_tensors < 0) return fail(ZERO_EINVAL, "n_tensors %d < 0", n_tensors);
    if (n_tensors > 0 && !tensors) return fail(ZERO_EINVAL, "tensors is NULL");
    int rc;
    if ((rc = check_plan_types(state_bits, grad_dtype, param_dtype))) return rc;
    const unsigned galign = grad_dtype == ZERO_FP32 ? 4 : 2;
    zero_tensors_plan_t p;
    std::memset(&p, 0, sizeof p);
    p.n_groups = 1;
    for (int32_t t = 0; t < n_tensors; ++t) {
        const zero_tensor_t& q = tensors[t];
        if (q.numel < 0) return fail(ZERO_EINVAL, "tensor %d has numel %lld < 0", t, (long long)q.numel);
        if (q.group < 0 || q.group >= ZERO_MAX_GROUPS)
            return fail(ZERO_EINVAL, "tensor %d has group %d outside [0, %d)", t, q.group, ZERO_MAX_GROUPS);
        if (q.reserved != 0) return fail(ZERO_EINVAL, "tensor %d: reserved must be 0", t);
        if (q.group >= p.n_groups) p.n_groups = q.group + 1;
        if (q.numel == 0) continue;
        if (!q.grad || !q.master || !q.exp_avg || !q.exp_avg_sq)
            return fail(ZERO_EINVAL, "tensor %d has a NULL grad, master or state", t);
        if ((q.param != nullptr) != (param_dtype != 0))
            return fail(ZERO_EINVAL, "tensor %d: param is given with param_dtype, and only then", t);
        if (off(q.grad, galign) || off(q.master, 4) || off(q.param, 2) ||
            off(q.exp_avg, state_bits == 8 ? 16 : 4) || off(q.exp_avg_sq, state_bits == 8 ? 2 : 4))
            return fail(ZERO_EALIGN, "tensor %d has a pointer off its element's alignment", t);
        const int64_t chunks = q.numel / kChunk + (q.numel % kChunk != 0);
        if (chunks > INT32_MAX - p.n_chunks)
            return fail(ZERO_EINVAL, "the list has more than %d chunks of %d elements", INT32_MAX, kChunk);
        p.numel += q.numel;
        p.n_chunks += chunks;
    }
    p.n_tensors = n_tensors;
    p.state_bits = state_bits;
    p.grad_dtype = grad_dtype;
    p.param_dtype = param_dtype;
    p.table_bytes = round_up(table_map_offset(n_tensors) + 4u * static_cast<size_t>(p.n_chunks), 16);
    p.workspace_bytes = kTensorsWorkspace;
    if (table) {
        if (table_cap < p.table_bytes)
            return fail(ZERO_ESIZE, "table_cap %zu < %llu needed", table_cap, (unsigned long long)p.table_bytes);
        unsigned char* out = static_cast<unsigned char*>(table);
        std::memset(out, 0, p.table_bytes);
        unsigned char* map = out + table_map_offset(n_tensors);
        int64_t chunk = 0;
        uint32_t block = 0;
        for (int32_t t = 0; t < n_tensors; ++t) {
            const zero_tensor_t& q = tensors[t];
            const TensorRec r = {q.grad, q.master, q.exp_avg, q.exp_avg_sq, q.param, q.numel, chunk, block, q.group};
            std::memcpy(out + sizeof r * static_cast<size_t>(t), &r, sizeof r);
            const int64_t end = chunk + q.numel / kChunk + (q.numel % kChunk != 0);
            for (; chunk < end; ++chunk) std::memcpy(map + 4u * static_cast<size_t>(chunk), &t, 4);
            block += static_cast<uint32_t>(q.numel / ZERO_STATE8_BLOCK + (q.numel % ZERO_STATE8_BLOCK != 0));
        }
    }
    *plan = p;
    return ZERO_OK;
}

int zero_tensors_scalars(const zero_tensors_args* a, zero_tensors_scalars_t* out) {
    clear_error();
    if (!out) return fail(ZERO_EINVAL, "out is NULL");
    zero_tensors_scalars_t k;
    const int rc = tensors_constants(a, true, false, &k);
    if (rc) return rc;
    *out = k;
    return ZERO_OK;
}

}  // extern "C"
