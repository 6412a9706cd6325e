// la_decay.cu -- C ABI of the decayed linear attention: argument checks, the work plan and
// dispatch (see la_decay.cuh for the passes that the kernels run).
#include <cmath>

#include "la_decay.cuh"

namespace la {
namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool width_ok(int D) { return D == 32 || D == 64 || D == 128; }

la_status check(int B, int Hq, int Hkv, int N, int D, int Dv, int dtype, float scale) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || D <= 0 || Dv <= 0 || Hq % Hkv != 0) return LA_ERR_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_ARG;
    // (a subnormal one has no row factors of two and, as the gradients divide by it, no finite reciprocal)
    if (!std::isnormal(scale)) return LA_ERR_ARG;
    // rows of a tensor are counted in 64 bits, heads and blocks in 31
    if ((unsigned long long)B * Hq >= (1u << 26) || (((unsigned long long)B * Hq * N) >> 50)) return LA_ERR_ARG;
    if (!width_ok(D) || !width_ok(Dv)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

struct DecayPlan {
    la_path path;
    int seg_len, nseg;
    long long state_units;                      // sequences that the state kernel sums
    size_t state_bytes, part_bytes, ws_bytes;   // one array of segment states, one of their parts; all of them
};

bool tc_runs(int D, int Dv, la_dtype dt) { return dt == LA_BF16 && D != 32 && Dv != 32; }

// The parts of a segment that the state kernel sums in blocks of their own: as many as one wave takes.
struct Parts {
    int n, len;
};
Parts parts_of(int chunks, int per) { return Parts{(chunks + per - 1) / per, per * kDecayTcChunk}; }
Parts sum_parts(long long units, int nsum, int chunks) {
    const long long fit = kPlanSms / (units * nsum);
    const int want = fit < 1 ? 1 : fit < chunks ? (int)fit : chunks;
    return parts_of(chunks, (chunks + want - 1) / want);
}
// The same where the sum over `heads` is an output: a block takes its parts one after the other, so the count whose longest
// block ends first: a part costs one product more, or two where it is joined (its state is written and read), and the
// join five.
Parts exact_parts(long long units, int nsum, int chunks, int heads) {
    Parts best = sum_parts(units, nsum, chunks);
    if (nsum > 1 && best.n > 1) return best;   // (joined anyway)
    long long cost = -1;
    for (int n = 1; n <= 16 && n <= chunks; ++n) {
        const Parts p = parts_of(chunks, (chunks + n - 1) / n);
        const long long rounds = (units * nsum * p.n + kPlanSms - 1) / kPlanSms;
        const bool joined = nsum > 1 || p.n > 1;
        const long long c = rounds * ((joined ? 2 : 1) + (long long)(p.len / kDecayTcChunk) * heads) + (joined ? 5 : 0);
        if (cost < 0 || c < cost) {
            cost = c;
            best = p;
        }
    }
    return best;
}

// The segments of a sequence: the count whose schedule ends first.  A schedule is waves of blocks that run at once,
// a block costing its start and its chunks (a chunk more where two blocks share an SM), and at least what the memory
// traffic takes; more than one segment costs the kernels that sum and join them.  Times in microseconds, fitted to
// GB300: on the tensor cores (one block an SM) 27 chunks of four heads of 128 x 128 take 270 us, 32 of 64 x 64 78 us, sums
// of 8 chunks 128 x 128 20 us; on the CUDA cores 64 chunks of 64 x 64 362 us with one block an SM and 610 us with two.
struct Cost {
    int per_sm;                      // blocks an SM holds
    double start, chunk, pair;       // of a block: its start, a chunk, a chunk's factor beside another block
    double waves(long long blocks, int chunks) const {
        const long long full = blocks / (per_sm * kPlanSms), rest = blocks % (per_sm * kPlanSms);
        return full * (start + chunks * chunk * pair) + (rest ? start + chunks * chunk * (rest > kPlanSms ? pair : 1.0) : 0.0);
    }
    // One block an SM: `nl` blocks of `cl` chunks, then `ns` of `cs` on the SMs that are free first.
    double two(long long nl, int cl, long long ns, int cs) const {
        const double tl = start + cl * chunk, ts = start + cs * chunk;
        const long long full = nl / kPlanSms, busy = nl % kPlanSms;
        const double t0 = full * tl, end = t0 + (busy ? tl : 0.0);
        long long k = ns / kPlanSms;
        auto done = [&](double t) {
            return (kPlanSms - busy) * (long long)((t - t0) / ts + 1e-9) +
                   (t > end ? busy * (long long)((t - end) / ts + 1e-9) : 0);
        };
        while (done(t0 + k * ts) < ns) ++k;
        const double t = t0 + k * ts;
        return t > end ? t : end;
    }
};

DecayPlan make_plan(int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dt, bool bwd) {
    DecayPlan pl{};
    const int reps = Hq / Hkv;
    const long long heads = (long long)B * Hkv;
    long long units, state_units;                  // blocks of a segment: of the passes, of the sums
    int chunk;
    Cost pass, sum;
    double bytes = 0.0, s_bytes = 0.0;             // of a chunk over all blocks
    double join, join_seg;                         // the sums' join, and of it each segment
    const double rate = 5.8e6;                     // bytes a microsecond
    if (tc_runs(D, Dv, dt)) {
        pl.path = LA_PATH_TCGEN05;
        chunk = kDecayTcChunk;
        units = heads * (bwd ? 3 : 1);
        pass = Cost{1, 6.0, reps * (D + Dv == 256 ? 2.4 : D + Dv == 192 ? 2.2 : 2.0), 1.0};
        // q, k, v and out; the gradients: three passes of as much (their common inputs from L2 in part)
        bytes = chunk * 2.0 * heads * ((reps + 1.0) * (D + Dv)) * (bwd ? 2.5 : 1.0);
        state_units = heads * (bwd ? 2 : 1);
        sum = Cost{1, 7.0, (bwd ? (reps + 1.0) / 2.0 : 1.0) * (D + Dv == 256 ? 1.4 : D + Dv == 192 ? 1.1 : 0.8), 1.0};
        s_bytes = chunk * 2.0 * heads * (D + Dv) * (bwd ? reps + 1.0 : 1.0);
        join = 5.0;
        join_seg = 0.2;
    } else {
        pl.path = LA_PATH_SIMT;
        chunk = 32;
        const int wide = D > Dv ? D : Dv, DZ = bwd ? wide : Dv;
        units = heads * (DZ / decay_simt_slice(DZ)) * (bwd ? 3 : 1);
        pass = Cost{2, 3.0, reps * (0.5 + 0.085 * wide), 1.7};
        state_units = heads * (Dv / decay_simt_slice(Dv)) * (bwd ? 2 : 1);
        sum = Cost{2, 4.0, (bwd ? reps : 1) * (0.4 + 0.026 * D), 1.7};
        join = 0.0;
        join_seg = 0.5;   // (each block of a pass sums the segments before its own)
    }
    const int nchunks = (N + chunk - 1) / chunk;
    double best = -1.0;
    int best_cps = nchunks;
    auto consider = [&](int cps) {
        const int nseg = (nchunks + cps - 1) / cps, tail = nchunks - (nseg - 1) * cps;
        const double mem = nchunks * bytes / rate;
        double cost = pl.path == LA_PATH_SIMT ? pass.waves(units * nseg, cps) : pass.two(units * (nseg - 1), cps, units, tail);
        if (cost < mem) cost = mem;
        if (nseg > 1) {
            const Parts parts = pl.path == LA_PATH_SIMT ? Parts{1, 0} : sum_parts(state_units, nseg - 1, cps);
            const double smem = (double)(nseg - 1) * cps * s_bytes / rate;
            const double sc = sum.waves(state_units * (nseg - 1) * parts.n, (cps + parts.n - 1) / parts.n);
            cost += (sc < smem ? smem : sc) + join + join_seg * nseg;
        }
        if (best < 0 || cost < best) {
            best = cost;
            best_cps = cps;
        }
    };
    // (past a few waves more segments only cost)
    const long long most = 4 * pass.per_sm * kPlanSms / units + 2;
    for (int want = 1; want <= nchunks && want <= most; ++want) {
        const int cps = (nchunks + want - 1) / want;
        consider(cps);
        // one to three long segments and a short one: the short blocks run where the long ones leave SMs idle (the
        // gradients of 2 x 16 heads, N 8192, D 128: 167 us in one segment, 175 in three, 161 in 44 and 20 chunks)
        const int longer = want > 1 ? (nchunks + want - 2) / (want - 1) : 0;
        if (pl.path == LA_PATH_TCGEN05 && want > 1 && want <= 4)
            for (int i = 1; i < 16; ++i) consider(cps + (longer - cps) * i / 16);
    }
    pl.seg_len = best_cps * chunk;
    pl.nseg = (N + pl.seg_len - 1) / pl.seg_len;
    const int out_heads = bwd ? reps : 1;
    if (pl.nseg == 1) {
        // a state that goes out, where its sum is in several parts
        pl.state_units = heads;
        const int n = pl.path == LA_PATH_TCGEN05 ? exact_parts(heads, 1, nchunks, out_heads).n : 1;
        if (n > 1) pl.ws_bytes = pl.part_bytes = (size_t)heads * n * D * Dv * 4;
        return pl;
    }
    pl.state_bytes = ((size_t)heads * pl.nseg * D * Dv * 4 + 255) / 256 * 256;
    if (pl.path == LA_PATH_SIMT) {
        pl.ws_bytes = pl.state_bytes * (bwd ? 2 : 1);
        return pl;
    }
    // room for the parts of all segments (with a final state) and of all but the last
    pl.state_units = state_units;
    const int n0 = (pl.nseg - 1) * sum_parts(state_units, pl.nseg - 1, best_cps).n,
              n1 = pl.nseg * exact_parts(state_units, pl.nseg, best_cps, out_heads).n;
    pl.part_bytes = ((size_t)heads * (n0 > n1 ? n0 : n1) * D * Dv * 4 + 255) / 256 * 256;
    // forward: S; backward: S^T, A and A^T
    pl.ws_bytes = pl.state_bytes * (bwd ? 3 : 1) + pl.part_bytes * (bwd ? 2 : 1);
    return pl;
}

// Strides of a [B, H, N, W] input (st NULL: contiguous); false for a negative one.  A dimension of one
// has no step.
bool input_strides(const la_strides *st, int B, int H, int N, int W, Strides *out) {
    *out = contiguous_strides(H, N, W);
    if (!st) return true;
    if (st->b < 0 || st->h < 0 || st->n < 0) return false;
    if (B > 1) out->b = st->b;
    if (H > 1) out->h = st->h;
    if (N > 1) out->n = st->n;
    return true;
}

struct Given {
    const void *q, *k, *v, *g;
    const la_strides *sq, *sk, *sv, *sg;
    void *out, *dq, *dk, *dv;
    const float *log_decay, *s_in, *ds_in;
    float *s_out, *ds_out;
    const int *lengths;
};

la_status run(bool bwd, const Given &a, int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dt, float scale, void *ws,
              size_t ws_bytes, void *stream) {
    la_status st = check(B, Hq, Hkv, N, D, Dv, dt, scale);
    if (st != LA_OK) return st;
    if (!a.q || !a.k || !a.v || !a.log_decay) return LA_ERR_ARG;
    if (bwd ? (!a.g || !a.dq || !a.dk || !a.dv) : !a.out) return LA_ERR_ARG;
    // (the passes of the gradients read both states while one of them writes grad_initial_state)
    if (a.ds_out && (a.ds_out == a.s_in || a.ds_out == a.ds_in)) return LA_ERR_ARG;
    const void *ptrs[] = {a.q, a.k, a.v, a.g, a.out, a.dq, a.dk, a.dv, a.s_in, a.ds_in, a.s_out, a.ds_out};
    for (const void *p : ptrs)
        if (p && !aligned(p, 16)) return LA_ERR_ALIGN;
    if (!aligned(a.log_decay, 4) || (a.lengths && !aligned(a.lengths, 4))) return LA_ERR_ALIGN;
    Strides sq, sk, sv, sg;
    if (!input_strides(a.sq, B, Hq, N, D, &sq) || !input_strides(a.sk, B, Hkv, N, D, &sk) ||
        !input_strides(a.sv, B, Hkv, N, Dv, &sv) || !input_strides(a.sg, B, Hq, N, Dv, &sg))
        return LA_ERR_ARG;
    const DecayPlan pl = make_plan(B, Hq, Hkv, N, D, Dv, dt, bwd);
    const bool tc = pl.path == LA_PATH_TCGEN05, state_out = a.s_out || a.ds_out;
    const bool sums = tc && (pl.nseg > 1 || state_out);   // the state kernel runs
    if (pl.ws_bytes > 0 && (pl.nseg > 1 || state_out)) {
        if (!ws || ws_bytes < pl.ws_bytes) return LA_ERR_WORKSPACE;
        if (!aligned(ws, 256)) return LA_ERR_ALIGN;
    }
    if (tc)   // TMA: every stride a multiple of 16 bytes (8 bf16)
        for (const Strides &x : {sq, sk, sv, sg})
            if (x.b % 8 || x.h % 8 || x.n % 8) return LA_ERR_ALIGN;
    DecayParams p{};
    p.log_decay = a.log_decay;
    p.lengths = a.lengths;
    p.B = B; p.Hkv = Hkv; p.n_rep = Hq / Hkv; p.N = N; p.D = D; p.Dv = Dv;
    p.scale = scale;
    p.seg_len = pl.seg_len; p.nseg = pl.nseg;
    auto mem = [&](size_t off) { return reinterpret_cast<float *>(static_cast<char *>(ws) + off); };
    auto at = [&](size_t off) { return pl.nseg > 1 ? mem(off) : nullptr; };
    float *slots0 = at(0), *slots1 = at(pl.state_bytes), *slots2 = tc ? at(2 * pl.state_bytes) : slots1;
    DecayStateParams sp{};
    sp.log_decay = a.log_decay;
    sp.lengths = a.lengths;
    sp.B = B; sp.Hkv = Hkv; sp.N = N; sp.D = D; sp.Dv = Dv; sp.seg_len = pl.seg_len; sp.nseg = pl.nseg;
    // S = sum k v^T (both directions of a training step start from it)
    sp.y[0] = a.k; sp.z[0] = a.v; sp.sy[0] = sk; sp.sz[0] = sv; sp.init[0] = a.s_in; sp.init_mul[0] = 1.f;
    sp.heads[0] = 1; sp.rev[0] = 0; sp.slots[0] = slots0; sp.exact[0] = a.s_out != nullptr;
    sp.n = 1;
    sp.fin[0] = a.s_out; sp.fin[1] = a.ds_out; sp.fin_mul[0] = 1.f; sp.fin_mul[1] = scale;
    sp.nsum = state_out ? pl.nseg : pl.nseg - 1;
    if (sums) {
        const int chunks = pl.seg_len / kDecayTcChunk;
        const Parts parts = state_out ? exact_parts(pl.state_units, sp.nsum, chunks, bwd ? p.n_rep : 1)
                                      : sum_parts(pl.state_units, sp.nsum, chunks);
        sp.nsub = parts.n;
        sp.sub_len = parts.len;
    }
    sp.part[0] = at(pl.state_bytes * (bwd ? 3 : 1));
    sp.part[1] = at(pl.state_bytes * 3 + pl.part_bytes);
    if (!bwd) {
        sp.start[0] = slots0;
        DecayPass &f = p.pass[0];
        f.x = a.q; f.y = a.k; f.z = a.v; f.sx = sq; f.sy = sk; f.sz = sv; f.out = a.out;
        f.slots = slots0; f.init = a.s_in; f.fin = tc ? nullptr : a.s_out; f.init_mul = f.fin_mul = 1.f;
        p.npass = 1;
    } else {
        // A = sum q g^T from the last token back
        sp.y[1] = a.q; sp.z[1] = a.g; sp.sy[1] = sq; sp.sz[1] = sg; sp.init[1] = a.ds_in; sp.init_mul[1] = 1.f / scale;
        sp.heads[1] = p.n_rep; sp.rev[1] = 1; sp.slots[1] = slots1; sp.exact[1] = a.ds_out != nullptr;
        sp.n = 2;
        sp.first_off[1] = 1;
        sp.start_tr[0] = slots0; sp.start[1] = slots1; sp.start_tr[1] = slots2;
        DecayPass &q = p.pass[0], &k = p.pass[1], &v = p.pass[2];
        q.x = a.g; q.y = a.v; q.z = a.k; q.sx = sg; q.sy = sv; q.sz = sk; q.out = a.dq;
        q.slots = slots0; q.init = a.s_in; q.tr = 1; q.init_mul = q.fin_mul = 1.f;
        k.x = a.v; k.y = a.g; k.z = a.q; k.sx = sv; k.sy = sg; k.sz = sq; k.out = a.dk;
        k.slots = slots2; k.init = a.ds_in; k.tr = 1;
        v.x = a.k; v.y = a.q; v.z = a.g; v.sx = sk; v.sy = sq; v.sz = sg; v.out = a.dv;
        v.slots = slots1; v.init = a.ds_in; v.fin = tc ? nullptr : a.ds_out;
        for (DecayPass *ps : {&k, &v}) {
            ps->many_yz = 1;
            ps->rev = 1;
            ps->first_off = 1;
            ps->init_mul = 1.f / scale;
            ps->fin_mul = scale;
        }
        p.npass = 3;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (tc) {
        e = error_word(&p.err);
        sp.err = p.err;
        if (e == cudaSuccess && pl.nseg > 1) e = decay_tc_states(sp, s);
        if (e == cudaSuccess && pl.nseg > 1) e = decay_tc_join(sp, s);
        if (e == cudaSuccess) e = decay_tc_passes(p, s);
        if (sums && pl.nseg == 1) {
            // the sum of the array that goes out; after the pass, which reads the starting state that this may replace
            sp.start[0] = sp.start[1] = sp.start_tr[0] = sp.start_tr[1] = nullptr;
            sp.first = bwd;
            sp.n = 1;
            sp.direct = sp.nsub == 1;
            if (!sp.direct) sp.part[bwd] = mem(0);
            if (e == cudaSuccess) e = decay_tc_states(sp, s);
            if (e == cudaSuccess && !sp.direct) e = decay_tc_join(sp, s);
        }
        return e == cudaSuccess ? LA_OK : cuda_fail(e);
    }
    if (pl.nseg > 1) e = decay_simt_states(sp, dt, s);
    // (the gradients' passes have two shapes of state, D x Dv and its transpose)
    if (e == cudaSuccess && (p.npass == 1 || D == Dv)) {
        e = decay_simt_passes(p, 0, p.npass, dt, s);
    } else if (e == cudaSuccess) {
        e = decay_simt_passes(p, 0, 2, dt, s);
        if (e == cudaSuccess) e = decay_simt_passes(p, 2, 1, dt, s);
    }
    return e == cudaSuccess ? LA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

size_t la_decay_workspace_size(int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype, int is_bwd) {
    if (check(B, Hq, Hkv, N, D, Dv, dtype, 1.f) != LA_OK) return 0;
    // (a training step's one workspace serves its forward too, which may be cut into more segments)
    const size_t fwd = make_plan(B, Hq, Hkv, N, D, Dv, dtype, false).ws_bytes;
    if (!is_bwd) return fwd;
    const size_t bwd = make_plan(B, Hq, Hkv, N, D, Dv, dtype, true).ws_bytes;
    return fwd > bwd ? fwd : bwd;
}

la_path la_decay_kernel_path(int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype, int is_bwd) {
    if (check(B, Hq, Hkv, N, D, Dv, dtype, 1.f) != LA_OK) return LA_PATH_SIMT;
    return make_plan(B, Hq, Hkv, N, D, Dv, dtype, is_bwd).path;
}

la_status la_decay_fwd(const void *q, const void *k, const void *v, void *out, const float *log_decay,
                       const float *initial_state, float *final_state, const int *lengths, int B, int Hq, int Hkv,
                       int N, int D, int Dv, la_dtype dtype, float scale, const la_strides *q_strides,
                       const la_strides *k_strides, const la_strides *v_strides, void *workspace, size_t ws_bytes,
                       void *stream) {
    Given a{};
    a.q = q; a.k = k; a.v = v; a.out = out; a.log_decay = log_decay; a.s_in = initial_state; a.s_out = final_state;
    a.lengths = lengths; a.sq = q_strides; a.sk = k_strides; a.sv = v_strides;
    return run(false, a, B, Hq, Hkv, N, D, Dv, dtype, scale, workspace, ws_bytes, stream);
}

la_status la_decay_bwd(const void *q, const void *k, const void *v, const void *grad_out, void *dq, void *dk, void *dv,
                       const float *log_decay, const float *initial_state, const float *grad_final_state,
                       float *grad_initial_state, int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype,
                       float scale, const la_strides *q_strides, const la_strides *k_strides,
                       const la_strides *v_strides, const la_strides *g_strides, void *workspace, size_t ws_bytes,
                       void *stream) {
    Given a{};
    a.q = q; a.k = k; a.v = v; a.g = grad_out; a.dq = dq; a.dk = dk; a.dv = dv; a.log_decay = log_decay;
    a.s_in = initial_state; a.ds_in = grad_final_state; a.ds_out = grad_initial_state;
    a.sq = q_strides; a.sk = k_strides; a.sv = v_strides; a.sg = g_strides;
    return run(true, a, B, Hq, Hkv, N, D, Dv, dtype, scale, workspace, ws_bytes, stream);
}

la_status la_decay_step(const void *q, const void *k, const void *v, void *out, const float *state, float *state_out,
                        const float *log_decay, const int *slots, int pool, int B, int Hq, int Hkv, int D, int Dv,
                        la_dtype dtype, float scale, const la_strides *q_strides, const la_strides *k_strides,
                        const la_strides *v_strides, void *stream) {
    la_status st = check(B, Hq, Hkv, 1, D, Dv, dtype, scale);
    if (st != LA_OK) return st;
    if (!q || !k || !v || !out || !state || !state_out || !log_decay || pool <= 0) return LA_ERR_ARG;
    if (!slots && pool < B) return LA_ERR_ARG;
    const void *ptrs[] = {q, k, v, out, state, state_out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return LA_ERR_ALIGN;
    if (!aligned(log_decay, 4) || (slots && !aligned(slots, 4))) return LA_ERR_ALIGN;
    DecayStepParams p{};
    if (!input_strides(q_strides, B, Hq, 1, D, &p.sq) || !input_strides(k_strides, B, Hkv, 1, D, &p.sk) ||
        !input_strides(v_strides, B, Hkv, 1, Dv, &p.sv))
        return LA_ERR_ARG;
    p.q = q; p.k = k; p.v = v; p.out = out; p.state = state; p.state_out = state_out; p.log_decay = log_decay;
    p.slots = slots; p.pool = pool; p.B = B; p.Hkv = Hkv; p.n_rep = Hq / Hkv; p.D = D; p.Dv = Dv; p.scale = scale;
    cudaError_t e = decay_step(p, dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : cuda_fail(e);
}

}  // extern "C"
