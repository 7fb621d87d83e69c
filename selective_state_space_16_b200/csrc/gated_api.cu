// gated_api.cu -- the C ABI of the gated linear recurrence (ssm_gated.h): argument checks,
// workspace layout, dispatch over the element type.
#include <cmath>
#include <limits>

#include "gated_host.h"
#include "host_common.h"

namespace {

using namespace ssmh;
using ssm::GatedParams;
using ssm::GatedTensor;

// dlam, dr_bias and di_bias of a channel: sums over the batch rows, in their order.  A programmatic dependent of the
// backward, launched while it ends.  (One batch row written by the backward itself: 2 us less for 384 rows of
// 32768 steps, but its registers cost 8 x 1536 x 2048 steps 4 us.)
__global__ void __launch_bounds__(128) gated_bwd_params_kernel(const float* part, const float* lam, float* dlam, float* drb,
                                                               float* dib, int batch, int dim) {
    ssm::pdl_wait_primary();
    const int d = blockIdx.x * 128 + threadIdx.x;
    if (d >= dim) return;
    const long long rows = static_cast<long long>(batch) * dim;
    float s[3] = {0.f, 0.f, 0.f};
    for (int b = 0; b < batch; ++b)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += part[k * rows + static_cast<long long>(b) * dim + d];
    if (dlam) {  // T is dL / d log v; d log v / dlam = sigmoid / softplus -> 1 for lam -> -inf
        const float l = lam[d], e = expf(l);
        dlam[d] = s[0] * (l < -15.f ? 1.f : l > 20.f ? 1.f / l : e / (1.f + e) / log1pf(e));
    }
    if (drb) drb[d] = s[1];
    if (dib) dib[d] = s[2];
}

bool valid_sizes(int batch, int dim, int64_t seqlen) { return batch >= 0 && dim >= 0 && seqlen >= 0; }

constexpr long long kMaxSteps = (1LL << 31) - (1 << 16);  // (steps are 32-bit in the kernels, a few tiles past the last)
constexpr int kMaxStepBatch = 65535;  // (far past a batch of a decode step)

bool supported_sizes(int batch, int dim, int64_t seqlen) {
    return static_cast<long long>(batch) * dim < (1LL << 31) && seqlen < kMaxSteps;
}

// Floats of a row of checkpoints: one for each group of steps, of which the first can begin up to
// kGroup - 1 steps before the row (an aligned window), rounded up to 16 bytes.
long long checkpoint_row(int64_t seqlen) {
    return static_cast<long long>(round_up((static_cast<size_t>(seqlen) + 2 * (ssm::kGroup - 1)) / ssm::kGroup, 4));
}

template <typename T>
GatedTensor tensor(const T& t, int batch, int dim) {
    const bool up = t.batch_stride >= 0 && t.dim_stride >= 0;
    return {t.data, t.batch_stride, t.dim_stride, (batch - 1LL) * t.batch_stride + (dim - 1LL) * t.dim_stride, up ? 15ull : 0ull};
}

bool element_aligned(const void* p, int io) {
    return (reinterpret_cast<uintptr_t>(p) & (io == SSM_BF16 ? 1u : 3u)) == 0;
}
bool float_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks what forward and backward read alike and fills the kernels' parameters.
ssm_status_t common_params(const ssm_gated_args_t* a, GatedParams* p) {
    if (!a || !valid_sizes(a->batch, a->dim, a->seqlen)) return SSM_ERR_INVALID_ARG;
    if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16) return SSM_ERR_INVALID_ARG;
    if (!(a->c > 0.f) || !std::isfinite(a->c)) return SSM_ERR_INVALID_ARG;
    if (!supported_sizes(a->batch, a->dim, a->seqlen)) return SSM_ERR_UNSUPPORTED;
    const bool rows = a->batch > 0 && a->dim > 0;
    if (rows && !a->lam) return SSM_ERR_INVALID_ARG;
    if (rows && a->seqlen > 0 && (!a->x.data || !a->r.data || !a->i.data)) return SSM_ERR_INVALID_ARG;
    for (const void* q : {a->x.data, a->r.data, a->i.data, a->z.data})
        if (!element_aligned(q, a->io_dtype)) return SSM_ERR_INVALID_ARG;
    for (const void* q : {static_cast<const void*>(a->lam), static_cast<const void*>(a->r_bias), static_cast<const void*>(a->i_bias),
                          static_cast<const void*>(a->initial_state), static_cast<const void*>(a->lengths)})
        if (!float_aligned(q)) return SSM_ERR_INVALID_ARG;
    *p = GatedParams{};
    p->x = tensor(a->x, a->batch, a->dim);
    p->r = tensor(a->r, a->batch, a->dim);
    p->i = tensor(a->i, a->batch, a->dim);
    p->z = tensor(a->z, a->batch, a->dim);
    p->lam = a->lam;
    p->r_bias = a->r_bias;
    p->i_bias = a->i_bias;
    p->h0 = a->initial_state;
    p->lengths = a->lengths;
    p->reset = a->reset;
    p->batch = a->batch;
    p->dim = a->dim;
    p->L = static_cast<int>(a->seqlen);
    p->ckpt_row = checkpoint_row(a->seqlen);
    p->c = a->c;
    return SSM_OK;
}

// Whether no two rows of an output overlap (channels inside batch rows, or the other way round).
bool rows_apart(const GatedTensor& t, int batch, int dim, int64_t L) {
    const auto nested = [L](long long n_out, long long s_out, long long n_in, long long s_in) {
        const long long inner = n_in > 1 ? (s_in >= L ? (n_in - 1) * s_in + L : -1) : L;
        return inner >= 0 && (n_out <= 1 || s_out >= inner);
    };
    return nested(batch, t.bs, dim, t.ds) || nested(dim, t.ds, batch, t.bs);
}

bool is_input(const ssm_gated_args_t* a, const void* q) {
    if (!q) return false;
    for (const void* in : {a->x.data, a->r.data, a->i.data, a->z.data, static_cast<const void*>(a->lam), static_cast<const void*>(a->r_bias),
                           static_cast<const void*>(a->i_bias), static_cast<const void*>(a->initial_state),
                           static_cast<const void*>(a->lengths), static_cast<const void*>(a->reset)})
        if (q == in) return true;
    return false;
}

ssm_status_t launch_fwd(int io, const GatedParams& p, int sms, cudaStream_t s) {
    return io == SSM_BF16 ? launch_gated_fwd<__nv_bfloat16>(p, sms, s) : launch_gated_fwd<float>(p, sms, s);
}

}  // namespace

extern "C" {

size_t ssm_gated_checkpoint_size(int batch, int dim, int64_t seqlen) {
    if (!valid_sizes(batch, dim, seqlen) || !supported_sizes(batch, dim, seqlen)) return 0;
    return sizeof(ssm::CkptHeader) + static_cast<size_t>(batch) * dim * checkpoint_row(seqlen) * sizeof(float);
}

ssm_status_t ssm_gated_scan_fwd(const ssm_gated_args_t* args, const ssm_gated_out_t* out, float* last_state, void* checkpoints,
                                size_t checkpoint_bytes, ssm_stream_t stream) {
    GatedParams p;
    ssm_status_t st = common_params(args, &p);
    if (st != SSM_OK) return st;
    if (!out) return SSM_ERR_INVALID_ARG;
    const ssm_gated_out_t& y = *out;
    const bool rows = p.batch > 0 && p.dim > 0;
    if (rows && p.L > 0 && !y.data) return SSM_ERR_INVALID_ARG;
    if (is_input(args, y.data) || !element_aligned(y.data, args->io_dtype)) return SSM_ERR_INVALID_ARG;
    if (last_state != args->initial_state && is_input(args, last_state)) return SSM_ERR_INVALID_ARG;
    if (!float_aligned(last_state) || !aligned16(checkpoints)) return SSM_ERR_INVALID_ARG;
    p.y = tensor(y, p.batch, p.dim);
    if (rows && p.L > 0 && !rows_apart(p.y, p.batch, p.dim, p.L)) return SSM_ERR_INVALID_ARG;
    if (!rows) return SSM_OK;
    if (checkpoints && checkpoint_bytes < ssm_gated_checkpoint_size(p.batch, p.dim, p.L)) return SSM_ERR_WORKSPACE;
    int sms = 0;
    st = check_device(&sms);
    if (st != SSM_OK) return st;
    if (p.L == 0) {  // no steps (and, with torch, no addresses): the state passes through
        const size_t bytes = static_cast<size_t>(p.batch) * p.dim * sizeof(float);
        cudaError_t e = cudaSuccess;
        if (last_state && p.h0 != last_state)
            e = p.h0 ? cudaMemcpyAsync(last_state, p.h0, bytes, cudaMemcpyDeviceToDevice, reinterpret_cast<cudaStream_t>(stream))
                     : cudaMemsetAsync(last_state, 0, bytes, reinterpret_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? SSM_OK : SSM_ERR_LAUNCH;
    }
    p.last = last_state;
    p.ckpt = static_cast<float*>(checkpoints);
    return launch_fwd(args->io_dtype, p, sms, reinterpret_cast<cudaStream_t>(stream));
}

size_t ssm_gated_bwd_workspace_size(int batch, int dim, int64_t seqlen, int have_checkpoints) {
    if (!valid_sizes(batch, dim, seqlen) || !supported_sizes(batch, dim, seqlen)) return 0;
    const size_t sums = round_up(static_cast<size_t>(batch) * dim * 3 * sizeof(float), 256);
    return sums + (have_checkpoints ? 0 : round_up(ssm_gated_checkpoint_size(batch, dim, seqlen), 256));
}

ssm_status_t ssm_gated_scan_bwd(const ssm_gated_args_t* args, const ssm_gated_grads_t* grads, const void* checkpoints,
                                size_t checkpoint_bytes, void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    GatedParams p;
    ssm_status_t st = common_params(args, &p);
    if (st != SSM_OK) return st;
    if (!grads) return SSM_ERR_INVALID_ARG;
    const ssm_gated_grads_t& g = *grads;
    const bool rows = p.batch > 0 && p.dim > 0;
    if (rows && p.L > 0 && (!g.dy.data || !g.dx.data || !g.dr.data || !g.di.data || (args->z.data && !g.dz.data)))
        return SSM_ERR_INVALID_ARG;
    for (const void* q : {g.dx.data, g.dr.data, g.di.data, g.dz.data})
        if (!element_aligned(q, args->io_dtype)) return SSM_ERR_INVALID_ARG;
    for (const void* q : {g.dx.data, g.dr.data, g.di.data, g.dz.data, static_cast<void*>(g.dlam), static_cast<void*>(g.dr_bias),
                          static_cast<void*>(g.di_bias)})
        if (is_input(args, q) || (q && (q == g.dy.data || q == g.dlast_state))) return SSM_ERR_INVALID_ARG;
    if (is_input(args, g.dinitial_state) || (g.dinitial_state && g.dinitial_state == g.dy.data)) return SSM_ERR_INVALID_ARG;
    if (!element_aligned(g.dy.data, args->io_dtype) || !aligned16(checkpoints)) return SSM_ERR_INVALID_ARG;
    for (const void* q : {static_cast<const void*>(g.dlast_state), static_cast<const void*>(g.dlam), static_cast<const void*>(g.dr_bias),
                          static_cast<const void*>(g.di_bias), static_cast<const void*>(g.dinitial_state)})
        if (!float_aligned(q)) return SSM_ERR_INVALID_ARG;
    p.dy = tensor(g.dy, p.batch, p.dim);
    p.dx = tensor(g.dx, p.batch, p.dim);
    p.dr = tensor(g.dr, p.batch, p.dim);
    p.di = tensor(g.di, p.batch, p.dim);
    p.dz = tensor(g.dz, p.batch, p.dim);
    if (rows && p.L > 0)
        for (const GatedTensor* t : {&p.dx, &p.dr, &p.di, p.z.p ? &p.dz : &p.dx})
            if (!rows_apart(*t, p.batch, p.dim, p.L)) return SSM_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool sums = g.dlam || g.dr_bias || g.di_bias;
    if (p.dim == 0) return SSM_OK;
    if (p.batch == 0 || p.L == 0) {  // no steps: the sums are zero, the state's gradient passes through
        st = check_device(nullptr);
        if (st != SSM_OK) return st;
        cudaError_t e = cudaSuccess;
        for (float* q : {g.dlam, g.dr_bias, g.di_bias})
            if (q && e == cudaSuccess) e = cudaMemsetAsync(q, 0, static_cast<size_t>(p.dim) * sizeof(float), s);
        const size_t bytes = static_cast<size_t>(p.batch) * p.dim * sizeof(float);
        if (g.dinitial_state && bytes && g.dinitial_state != g.dlast_state && e == cudaSuccess)
            e = g.dlast_state ? cudaMemcpyAsync(g.dinitial_state, g.dlast_state, bytes, cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(g.dinitial_state, 0, bytes, s);
        return e == cudaSuccess ? SSM_OK : SSM_ERR_LAUNCH;
    }
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < ssm_gated_bwd_workspace_size(p.batch, p.dim, p.L, checkpoints != nullptr) ||
        (checkpoints && checkpoint_bytes < ssm_gated_checkpoint_size(p.batch, p.dim, p.L)))
        return SSM_ERR_WORKSPACE;
    int sms = 0;
    st = check_device(&sms);
    if (st != SSM_OK) return st;
    p.dlast = g.dlast_state;
    p.part = sums ? static_cast<float*>(workspace) : nullptr;
    p.ckpt = static_cast<float*>(const_cast<void*>(checkpoints));
    if (!checkpoints) {
        p.ckpt = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                          round_up(static_cast<size_t>(p.batch) * p.dim * 3 * sizeof(float), 256));
        GatedParams f = p;  // a forward that stores nothing but the checkpoints
        f.z.p = nullptr;
        st = launch_fwd(args->io_dtype, f, sms, s);
        if (st != SSM_OK) return st;
    }
    p.dh0 = g.dinitial_state;
    st = args->io_dtype == SSM_BF16 ? launch_gated_bwd<__nv_bfloat16>(p, sms, s) : launch_gated_bwd<float>(p, sms, s);
    if (st != SSM_OK || !sums) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((p.dim + 127) / 128));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gated_bwd_params_kernel, static_cast<const float*>(p.part), p.lam, g.dlam,
                                             g.dr_bias, g.di_bias, p.batch, p.dim);
    return e == cudaSuccess ? launch_status() : SSM_ERR_LAUNCH;
}

ssm_status_t ssm_gated_state_update(const ssm_gated_step_t* args, ssm_stream_t stream) {
    if (!args) return SSM_ERR_INVALID_ARG;
    const ssm_gated_step_t& a = *args;
    if (a.batch < 0 || a.dim < 0 || a.n_slots < 0) return SSM_ERR_INVALID_ARG;
    if (a.io_dtype != SSM_F32 && a.io_dtype != SSM_BF16) return SSM_ERR_INVALID_ARG;
    if (!(a.c > 0.f) || !std::isfinite(a.c)) return SSM_ERR_INVALID_ARG;
    if (a.batch == 0 || a.dim == 0) return SSM_OK;
    if (!a.x || !a.r || !a.i || !a.y || !a.lam || (a.n_slots > 0 && !a.state)) return SSM_ERR_INVALID_ARG;
    if (a.state_stride < a.dim && a.n_slots > 1) return SSM_ERR_INVALID_ARG;
    if (a.batch > 1 && (a.y_stride < a.dim)) return SSM_ERR_INVALID_ARG;
    if (a.y == a.x || a.y == a.r || a.y == a.i || a.y == a.z) return SSM_ERR_INVALID_ARG;
    for (const void* q : {a.x, a.r, a.i, a.z, static_cast<const void*>(a.y)})
        if (!element_aligned(q, a.io_dtype)) return SSM_ERR_INVALID_ARG;
    for (const void* q : {static_cast<const void*>(a.state), static_cast<const void*>(a.slots), static_cast<const void*>(a.lam),
                          static_cast<const void*>(a.r_bias), static_cast<const void*>(a.i_bias)})
        if (!float_aligned(q)) return SSM_ERR_INVALID_ARG;
    if (a.batch > kMaxStepBatch || a.dim >= kMaxSteps) return SSM_ERR_UNSUPPORTED;
    int sms = 0;
    const ssm_status_t st = check_device(&sms);
    if (st != SSM_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return a.io_dtype == SSM_BF16 ? launch_gated_step<__nv_bfloat16>(a, sms, s) : launch_gated_step<float>(a, sms, s);
}

}  // extern "C"
