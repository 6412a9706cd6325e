// la_ssm.cu -- selective state space scan: C ABI, argument checks, work plan and dispatch.
#include <initializer_list>

#include "la_ssm.cuh"

namespace la {
namespace {

constexpr int kUnit = 16;   // tokens that segments are whole numbers of (the scan's tile)

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct SsmPlan {
    int seg_len, nseg;
    size_t off_d, off_bc, off_A, off_e, bytes;   // segments' states first
    int blocks, parts;
};

// The segments of a sequence: the count whose kernels end first, in microseconds fitted to GB300 with 16 states a channel in
// bfloat16.  The scan's blocks of a segment each (1024 states) share the SMs evenly, 42 ns a token and block; less than about 1.75
// blocks leave an SM waiting.  The gradient's (8 to 16 times as much work) run in waves of two blocks an SM, 1.2 us a token.  More
// than one segment costs the sums of all but one, 29 ns a token and block, and a launch.  Other state counts (2048 states a block of the
// scan for 64; 2048 to 8192 of the gradient) and float32 are planned with the same figures, and sequences with lengths as if all
// were full.
void cut(int N, bool bwd, long long blocks, long long sum_blocks, int slots, int *seg_len, int *nseg) {
    double best = -1.0;
    const int most = N < 64 * 64 ? (N + 63) / 64 : 64;
    auto per_sm = [&](long long b) {
        const double k = (double)((b + kPlanSms - 1) / kPlanSms);
        return k > 1.75 ? k : 1.75;
    };
    for (int want = 1; want <= most; ++want) {
        const int len = ((N + want - 1) / want + kUnit - 1) / kUnit * kUnit, n = (N + len - 1) / len;
        double cost = bwd ? (double)((blocks * n + slots - 1) / slots) * (10.0 + 1.2 * len) : 0.042 * len * per_sm(blocks * n);
        if (n > 1) cost += 0.029 * len * per_sm(sum_blocks * (n - 1)) + 4.5 + 0.25 * n;
        if (best < 0 || cost < best) {
            best = cost;
            *seg_len = len;
            *nseg = n;
        }
    }
}

SsmPlan make_plan(int nB, int N, int E, int S, int G, bool bwd) {
    SsmPlan pl{};
    const int Eg = E / G;
    auto blocks = [&](int ch) { return (Eg + ch - 1) / ch; };
    const long long heads = (long long)nB * G, scan = heads * blocks(ssm_scan_channels(S));
    pl.blocks = blocks(bwd ? ssm_grad_channels(S) : ssm_scan_channels(S));
    cut(N, bwd, heads * pl.blocks, scan, (S == 64 ? 1 : 2) * kPlanSms, &pl.seg_len, &pl.nseg);
    pl.parts = nB * pl.nseg;
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t off = at;
        at += up(floats * 4);
        return off;
    };
    if (pl.nseg > 1) {
        take((size_t)pl.parts * E * S);
        pl.off_d = take((size_t)pl.parts * E);
    }
    if (bwd) {
        pl.off_bc = take((size_t)G * pl.blocks * nB * N * 2 * S);
        pl.off_A = take((size_t)pl.parts * E * S);
        pl.off_e = take((size_t)pl.parts * 2 * E);
    }
    pl.bytes = at;
    return pl;
}

la_status check(int nB, int N, int E, int S, int G, la_dtype dt) {
    if (nB <= 0 || N <= 0 || E <= 0 || S <= 0 || G <= 0 || E % G || (dt != LA_F32 && dt != LA_BF16)) return LA_ERR_ARG;
    if ((S != 8 && S != 16 && S != 32 && S != 64) || (E / G) % 8) return LA_ERR_UNSUPPORTED;
    // element and block counts within the kernels' 64-bit offsets and 32-bit grids
    if (N > (1 << 30) || (long long)nB * N > (1ll << 36) || E > (1 << 24) || (long long)nB * E > (1ll << 30)) return LA_ERR_ARG;
    if ((long long)nB * N / 256 * ((long long)G * S / 2) >= (1ll << 31) - (1 << 24)) return LA_ERR_ARG;
    if ((long long)nB * (E / 8) * 64 >= (1ll << 31)) return LA_ERR_ARG;
    if ((double)nB * N * E * S > (double)(1ll << 56)) return LA_ERR_ARG;   // (bytes of states and parts)
    return LA_OK;
}

// Strides of a [B, N, E] input (groups 0), or of a [B, N, G, S] one: multiples of 16 bytes.
la_status strides_of(const la_strides *st, int nB, int N, int G, int width, la_dtype dt, Strides *out) {
    const long long row = (long long)(G > 0 ? G : 1) * width;
    *out = Strides{(long long)N * row, G > 0 ? width : 0, row};
    if (!st) return LA_OK;
    if (st->b < 0 || st->n < 0 || (G > 0 && st->h < 0)) return LA_ERR_ARG;
    if (nB > 1) out->b = st->b;
    if (N > 1) out->n = st->n;
    if (G > 1) out->h = st->h;
    const int unit = dt == LA_BF16 ? 8 : 4;
    return out->b % unit || out->n % unit || out->h % unit ? LA_ERR_ALIGN : LA_OK;
}

// What the three entry points check alike.
la_status check_args(const la_ssm_args *a, Strides (&st)[5]) {
    if (!a) return LA_ERR_ARG;
    la_status e = check(a->batch, a->N, a->E, a->S, a->G, a->dtype);
    if (e != LA_OK) return e;
    if (!a->x || !a->dt || !a->B || !a->C || !a->A) return LA_ERR_ARG;
    for (const void *p : {a->x, a->dt, a->B, a->C, a->z, (const void *)a->A, (const void *)a->initial_state})
        if (p && !aligned(p, 16)) return LA_ERR_ALIGN;
    for (const void *p : {(const void *)a->skip, (const void *)a->dt_bias, (const void *)a->lengths})
        if (p && !aligned(p, 4)) return LA_ERR_ALIGN;
    const la_strides *given[5] = {a->x_strides, a->dt_strides, a->z ? a->z_strides : nullptr, a->B_strides, a->C_strides};
    for (int i = 0; i < 5; ++i) {
        e = strides_of(given[i], a->batch, a->N, i < 3 ? 0 : a->G, i < 3 ? a->E : a->S, a->dtype, &st[i]);
        if (e != LA_OK) return e;
    }
    return LA_OK;
}

SsmParams params_of(const la_ssm_args *a, const Strides (&st)[5], const SsmPlan &pl, void *ws) {
    SsmParams p{};
    p.x = a->x; p.dt = a->dt; p.z = a->z; p.B = a->B; p.C = a->C;
    p.sx = st[0]; p.sdt = st[1]; p.sz = st[2]; p.sB = st[3]; p.sC = st[4];
    p.A = a->A; p.skip = a->skip; p.dt_bias = a->dt_bias; p.init = a->initial_state; p.lengths = a->lengths;
    p.nB = a->batch; p.N = a->N; p.E = a->E; p.S = a->S; p.G = a->G; p.Eg = a->E / a->G; p.softplus = a->softplus != 0;
    p.seg_len = pl.seg_len; p.nseg = pl.nseg;
    if (pl.nseg > 1) {
        p.seg_state = static_cast<float *>(ws);
        p.seg_d = reinterpret_cast<float *>(static_cast<char *>(ws) + pl.off_d);
    }
    return p;
}

size_t states_bytes_of(int nB, int N, int E, int S) { return (size_t)nB * ((N + kSsmTile - 1) / kSsmTile) * E * S * 4; }

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

size_t la_ssm_workspace_size(int batch, int N, int E, int S, int G, la_dtype dtype, int is_bwd) {
    if (check(batch, N, E, S, G, dtype) != LA_OK) return 0;
    const size_t fwd = make_plan(batch, N, E, S, G, false).bytes;
    if (!is_bwd) return fwd;
    const size_t bwd = make_plan(batch, N, E, S, G, true).bytes;
    return fwd > bwd ? fwd : bwd;
}

size_t la_ssm_states_size(int batch, int N, int E, int S) {
    if (check(batch, N, E, S, 1, LA_F32) != LA_OK) return 0;
    return states_bytes_of(batch, N, E, S);
}

la_status la_ssm_fwd(const la_ssm_args *a, void *out, float *final_state, void *states, size_t states_bytes,
                     void *workspace, size_t ws_bytes, void *stream) {
    Strides st[5];
    la_status e = check_args(a, st);
    if (e != LA_OK) return e;
    if (!out && !states) return LA_ERR_ARG;
    for (const void *p : {(const void *)out, (const void *)final_state, (const void *)states})
        if (p && !aligned(p, 16)) return LA_ERR_ALIGN;
    if (states && states_bytes < states_bytes_of(a->batch, a->N, a->E, a->S)) return LA_ERR_WORKSPACE;
    const SsmPlan pl = make_plan(a->batch, a->N, a->E, a->S, a->G, false);
    if (pl.bytes > 0) {
        if (!workspace || ws_bytes < pl.bytes) return LA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return LA_ERR_ALIGN;
    }
    SsmParams p = params_of(a, st, pl, workspace);
    p.out = out;
    p.fin = final_state;
    p.kept = static_cast<float *>(states);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t c = pl.nseg > 1 ? ssm_segments(p, a->dtype, false, s) : cudaSuccess;
    if (c == cudaSuccess) c = ssm_scan(p, a->dtype, s);
    return c == cudaSuccess ? LA_OK : cuda_fail(c);
}

la_status la_ssm_bwd(const la_ssm_args *a, const void *grad_out, const la_strides *g_strides, const float *grad_final_state,
                     const void *states, size_t states_bytes, const la_ssm_grads *g, void *workspace, size_t ws_bytes,
                     void *stream) {
    Strides st[5], sg;
    la_status e = check_args(a, st);
    if (e != LA_OK) return e;
    if (!grad_out || !states || !g || !g->dx || !g->ddt || !g->dB || !g->dC || !g->dA) return LA_ERR_ARG;
    if ((a->z == nullptr) != (g->dz == nullptr) || (g->dskip && !a->skip) || (g->ddt_bias && !a->dt_bias)) return LA_ERR_ARG;
    if (g->grad_initial_state && (g->grad_initial_state == a->initial_state || g->grad_initial_state == grad_final_state))
        return LA_ERR_ARG;
    for (const void *p : {grad_out, (const void *)grad_final_state, states, (const void *)g->dx, (const void *)g->ddt,
                          (const void *)g->dB, (const void *)g->dC, (const void *)g->dz, (const void *)g->dA,
                          (const void *)g->grad_initial_state})
        if (p && !aligned(p, 16)) return LA_ERR_ALIGN;
    for (const void *p : {(const void *)g->dskip, (const void *)g->ddt_bias})
        if (p && !aligned(p, 4)) return LA_ERR_ALIGN;
    e = strides_of(g_strides, a->batch, a->N, 0, a->E, a->dtype, &sg);
    if (e != LA_OK) return e;
    if (states_bytes < states_bytes_of(a->batch, a->N, a->E, a->S)) return LA_ERR_WORKSPACE;
    const SsmPlan pl = make_plan(a->batch, a->N, a->E, a->S, a->G, true);
    if (!workspace || ws_bytes < pl.bytes) return LA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LA_ERR_ALIGN;
    SsmParams p = params_of(a, st, pl, workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float *>(static_cast<char *>(workspace) + off); };
    p.g = grad_out;
    p.sg = sg;
    p.dfinal = grad_final_state;
    p.kept = const_cast<float *>(static_cast<const float *>(states));
    p.dx = g->dx; p.ddt = g->ddt; p.dz = g->dz; p.dinit = g->grad_initial_state;
    p.part_bc = at(pl.off_bc); p.part_A = at(pl.off_A); p.part_e = at(pl.off_e);
    SsmReduceParams r{};
    r.part_bc = p.part_bc; r.part_A = p.part_A; r.part_e = p.part_e; r.lengths = a->lengths;
    r.dB = g->dB; r.dC = g->dC; r.dA = g->dA; r.dskip = g->dskip; r.dbias = g->ddt_bias;
    r.nB = a->batch; r.N = a->N; r.E = a->E; r.S = a->S; r.G = a->G; r.blocks = pl.blocks; r.parts = pl.parts;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t c = pl.nseg > 1 ? ssm_segments(p, a->dtype, true, s) : cudaSuccess;
    if (c == cudaSuccess) c = ssm_grad(p, a->dtype, s);
    if (c == cudaSuccess) c = ssm_reduce(r, a->dtype, s);
    return c == cudaSuccess ? LA_OK : cuda_fail(c);
}

la_status la_ssm_step(const la_ssm_args *a, void *out, const float *state, float *state_out, const int *slots, int pool,
                      void *stream) {
    Strides st[5];
    la_status e = check_args(a, st);
    if (e != LA_OK) return e;
    if (a->N != 1 || a->initial_state || a->lengths || !out || !state || !state_out || pool <= 0 || (!slots && pool < a->batch))
        return LA_ERR_ARG;
    for (const void *p : {(const void *)out, (const void *)state, (const void *)state_out})
        if (!aligned(p, 16)) return LA_ERR_ALIGN;
    if (slots && !aligned(slots, 4)) return LA_ERR_ALIGN;
    SsmStepParams p{};
    p.x = a->x; p.dt = a->dt; p.z = a->z; p.B = a->B; p.C = a->C;
    p.sx = st[0]; p.sdt = st[1]; p.sz = st[2]; p.sB = st[3]; p.sC = st[4];
    p.A = a->A; p.skip = a->skip; p.dt_bias = a->dt_bias; p.state = state; p.state_out = state_out; p.slots = slots;
    p.out = out; p.pool = pool; p.nB = a->batch; p.E = a->E; p.S = a->S; p.G = a->G; p.Eg = a->E / a->G;
    p.softplus = a->softplus != 0;
    cudaError_t c = ssm_step(p, a->dtype, static_cast<cudaStream_t>(stream));
    return c == cudaSuccess ? LA_OK : cuda_fail(c);
}

}  // extern "C"
