// la_ssm_grad.cu -- gradient of the selective state space scan.
//
// With a_t = exp(d_t A), u_t = d_t x_t, dy_t the gradient of y (grad_out times the gate) and G_t that of h_t,
//
//   G_t = C_t dy_t + P_t,   P_(t-1) = a_t G_t,   q_t = P_(t-1) h_(t-1)
//   dB_t = sum_e G u,  dC_t = sum_e dy h,  du = sum_s G B,  dA = sum_t q d,  dd = sum_s q A + x du
//   dx = d du + skip dy,  ddt = dd sigmoid(v),  dz = grad_out y (z sigmoid(z))',  dskip = sum dy x
//
// 12 float operations and an ex2 a state and token.  h is found again from the state that the scan kept for every eight
// tokens; then the eight tokens are walked back, h and the decays still in registers.  Layout as in the scan, but 4 states a
// lane (h and decays of eight tokens and the sums below are 128 registers): a lane prepares its own tokens, those of the next
// unit while it works on this one; sums over states come by exchanged halves.
//
// The sums over channels (dB, dC) would cost more than all the rest if each token's were exchanged.  So a warp takes K
// channel groups one after the other for the same eight tokens and adds up in 64 registers; only then do its lanes exchange
// halves, the warps' sums meet in shared memory, and the block's are written as one part.  P, dA and A of the groups
// wait in shared memory meanwhile.  A unit is a warp's channels of one group and eight tokens; its rows come and go by the
// warp's own copies, so that there is a barrier only for each eight tokens.
//
// 4 x 4096 x 4096 x 16, bfloat16: 1054 us (float operations alone: 320); 246 registers, two blocks an SM, issue slots 54 %,
// shared memory 66 %.  64 states: one block an SM, 28 (float32: 32) bytes spilled.  168 registers and three blocks spill; 8
// states a lane with four tokens at a time find h again twice as often: 1404.  Neither 5 % fewer instructions (packed sums,
// simpler counters) nor 3 % less shared memory change the time: eight warps an SM do not hide the chains through h, P and the
// shuffles.  The tokens' d, d x and dy handed out through shared memory instead of shuffles: 1098, and 1118 with the decays
// found again to free their registers (three blocks: 1494).
#include "la_ssm.cuh"

namespace la {
namespace {

constexpr int kRing = 8;      // units of a warp in shared memory (a power of 2): one leaves, one is worked on, one is prepared,
constexpr int kAhead = 3;     // and copies run this many units ahead

constexpr int warps_of(int S) { return S == 64 ? 8 : 4; }
constexpr int groups_of(int S) { return S == 8 ? 4 : 8; }   // channel groups of a warp

template <typename T, int S>
struct Shape {
    static constexpr int LPC = S / 4, CPW = 32 / LPC, NW = warps_of(S), THREADS = NW * 32, OWN = LPC < 8 ? 8 / LPC : 1;
    static constexpr int CHK = NW * CPW, K = groups_of(S), CH = CHK * K;
    // a warp's rows of 8 tokens come and go by copies of CB bytes
    static constexpr int ROW = CPW * (int)sizeof(T), CB = ROW < 16 ? ROW : 16, PER = ROW / CB;
    static constexpr int XBYTES = 8 * ROW, UNIT = 4 * XBYTES;              // x, dt, z, g
    static constexpr int IN = (4 * 8 * PER + 31) / 32, OUT = (3 * 8 * PER + 31) / 32;   // copies of a lane
    static constexpr int V = 16 / (int)sizeof(T), BV = S / V, NB = 8 * BV;
    static constexpr int WIDE = 8 * 2 * S;                                 // floats: B and C of a tile; a warp's dB and dC
    static constexpr int KEEP = K * THREADS;                               // P, dA, A; sums for skip and dt_bias, bias and skip
    static constexpr int OFF_WIDE = NW * kRing * UNIT, OFF_P = OFF_WIDE + 2 * WIDE * 4, OFF_DA = OFF_P + KEEP * 16,
                         OFF_A = OFF_DA + KEEP * 16, OFF_E = OFF_A + KEEP * 16, OFF_RED = OFF_E + KEEP * 16,
                         SMEM = OFF_RED + 2 * NW * WIDE * 4;
    static_assert(SMEM <= 227 * 1024 && 2 * NB <= THREADS && WIDE % THREADS == 0, "a block's shared memory and its copies of B and C");
};

template <int BYTES>
__device__ __forceinline__ void copy_in(void *dst, const void *src, bool there) {
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(there ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "r"(there ? BYTES : 0) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_out(void *dst, const void *src) {
    if (BYTES == 16) *static_cast<uint4 *>(dst) = *static_cast<const uint4 *>(src);
    else if (BYTES == 8) *static_cast<uint2 *>(dst) = *static_cast<const uint2 *>(src);
    else *static_cast<unsigned *>(dst) = *static_cast<const unsigned *>(src);
}

template <typename T, int S>
__global__ void __launch_bounds__(Shape<T, S>::THREADS, S == 64 ? 1 : 2) k_ssm_grad(SsmParams p) {
    using H = Shape<T, S>;
    constexpr int LPC = H::LPC, CPW = H::CPW, OWN = H::OWN, OP = OWN > 1 ? OWN / 2 : 1, CHK = H::CHK, TH = H::THREADS, CB = H::CB;
    constexpr int EC = CB / (int)sizeof(T);                                  // channels of a copy
    extern __shared__ __align__(16) unsigned char smem[];
    float *wide = reinterpret_cast<float *>(smem + H::OFF_WIDE);
    float *red = reinterpret_cast<float *>(smem + H::OFF_RED);
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane / CPW, chan = lane % CPW;
    unsigned char *const ring = smem + warp * kRing * H::UNIT;
    float4 *const keep_P = reinterpret_cast<float4 *>(smem + H::OFF_P) + tid, *const keep_dA = reinterpret_cast<float4 *>(smem + H::OFF_DA) + tid,
                  *const keep_A = reinterpret_cast<float4 *>(smem + H::OFF_A) + tid;
    float2 *const keep_c = reinterpret_cast<float2 *>(smem + H::OFF_E) + tid, *const keep_s = keep_c + H::KEEP;   // bias, skip; sums
    const int blocks = (p.Eg + H::CH - 1) / H::CH;
    unsigned idx = blockIdx.x;
    const int cb = idx % blocks;
    idx /= blocks;
    const int grp = idx % p.G;
    idx /= p.G;
    const int seg = idx % p.nseg, b = idx / p.nseg;
    const int c0 = cb * H::CH, left = min(H::CH, p.Eg - c0), nk = (left + CHK - 1) / CHK;
    const int e0 = grp * p.Eg + c0, w0 = warp * CPW;                         // the warp's first channel of each group
    const int t0 = seg * p.seg_len, t1 = min(t0 + p.seg_len, p.N);
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int te = min(t1, len), n = max(te - t0, 0), nt = (n + 7) / 8, units = nt * nk;
    const bool gated = p.z != nullptr, sp = p.softplus;

    // A lane's copies: one place of every unit (tensor, row, piece of the row).  Unit u is group u % nk of tile nt - 1 - u / nk;
    // pointers move on by a group, and after the last group to the first of the tile before.  A copy is there for the
    // groups below `in_k`, in the last tile only where its row is within the length.
    const T *from[H::IN];
    long long wrap[H::IN];
    int in_k[H::IN];
    T *to[H::OUT];
    int out_k[H::OUT];
    const int last_rows = n - (nt - 1) * 8;                                  // tokens of the last tile
    auto groups = [&](int c) { return c < left ? (left - c - 1) / CHK + 1 : 0; };   // groups whose channel w0 + c is there
#pragma unroll
    for (int q = 0; q < H::IN; ++q) {
        const int v = lane + q * 32, m = v / (8 * H::PER), row = v / H::PER % 8, c = w0 + v % H::PER * EC;
        const void *base = m == 0 ? p.x : m == 1 ? p.dt : m == 2 ? p.z : p.g;
        const Strides st = m == 0 ? p.sx : m == 1 ? p.sdt : m == 2 ? p.sz : p.sg;
        wrap[q] = -8 * st.n - (long long)(nk - 1) * CHK;
        from[q] = static_cast<const T *>(base ? base : p.x) + b * st.b + (t0 + (nt - 1) * 8 + (long long)row) * st.n + e0 + c;
        in_k[q] = m > 3 || !base ? 0 : groups(c) + (row < last_rows ? 0 : 256);   // 256: not in the last tile
    }
#pragma unroll
    for (int q = 0; q < H::OUT; ++q) {
        const int v = lane + q * 32, m = v / (8 * H::PER), row = v / H::PER % 8, c = w0 + v % H::PER * EC;
        void *base = m == 0 ? p.dx : m == 1 ? p.ddt : p.dz;
        to[q] = static_cast<T *>(base ? base : p.dx) + ((long long)b * p.N + t0 + (nt - 1) * 8 + row) * p.E + e0 + c;
        out_k[q] = m > 2 || !base ? 0 : groups(c) + (row < last_rows ? 0 : 256);
    }
    int load_k = 0, load_u = 0, load_at = 0;
    auto load = [&]() {
        if (load_u < units) {
            const bool wraps = load_k + 1 == nk;
#pragma unroll
            for (int q = 0; q < H::IN; ++q) {
                const bool in = load_k < (in_k[q] & 255) && (in_k[q] < 256 || load_u >= nk);
                if (4 * 8 * H::PER % 32 == 0 || lane + q * 32 < 4 * 8 * H::PER)
                    copy_in<CB>(ring + load_at + (lane + q * 32) * CB, in ? from[q] : static_cast<const T *>(p.x), in);
                from[q] += wraps ? wrap[q] : CHK;
            }
            load_k = wraps ? 0 : load_k + 1;
            ++load_u;
            load_at = (load_at + H::UNIT) % (kRing * H::UNIT);
        }
        copy_commit();
    };
    // the rows of dx, ddt and dz that a unit leaves in the places of x, dt and z
    int leave_k = 0, leave_u = 0, leave_at = 0;
    const long long out_wrap = -8ll * p.E - (long long)(nk - 1) * CHK;
    auto leave = [&]() {
        const bool wraps = leave_k + 1 == nk;
#pragma unroll
        for (int q = 0; q < H::OUT; ++q) {
            if (leave_k < (out_k[q] & 255) && (out_k[q] < 256 || leave_u >= nk))
                copy_out<CB>(to[q], ring + leave_at + (lane + q * 32) * CB);
            to[q] += wraps ? out_wrap : CHK;
        }
        leave_k = wraps ? 0 : leave_k + 1;
        ++leave_u;
        leave_at = (leave_at + H::UNIT) % (kRing * H::UNIT);
    };
    // B and C of a tile: a copy a thread, through registers a tile ahead
    const int bv = tid % H::NB;
    const bool bthere = tid < 2 * H::NB;
    const T *bfrom = static_cast<const T *>(tid < H::NB ? p.B : p.C);
    const long long bstep = tid < H::NB ? p.sB.n : p.sC.n;
    bfrom += b * (tid < H::NB ? p.sB.b : p.sC.b) + grp * (tid < H::NB ? p.sB.h : p.sC.h) + bv % H::BV * H::V +
             (t0 + (nt - 1) * 8 + bv / H::BV) * bstep;
    alignas(16) T raw[H::V];
    auto ask = [&](int i) {   // rows past the length: zeros
        const bool in = bthere && i < nt && (i > 0 || bv / H::BV < last_rows);
        *reinterpret_cast<uint4 *>(raw) = in ? *reinterpret_cast<const uint4 *>(bfrom) : make_uint4(0, 0, 0, 0);
        bfrom -= 8 * bstep;
    };
    float *const wide_to = wide + bv / H::BV * (2 * S) + tid / H::NB * S + bv % H::BV * H::V;
    auto widen = [&](int i) {
        if (bthere) widen16(wide_to + (i & 1) * H::WIDE, raw);
    };
    // a tile's part of dB and dC
    float *part = p.part_bc + (((size_t)(grp * blocks + cb) * p.nB + b) * p.N + t0 + (long long)(nt - 1) * 8) * (2 * S) + tid;
    auto leave_bc = [&](int i) {
        const float *a = red + (i & 1) * H::NW * H::WIDE + tid;
#pragma unroll
        for (int v = 0; v < H::WIDE; v += TH) {
            float sum = a[v];
#pragma unroll
            for (int w = 1; w < H::NW; ++w) sum += a[w * H::WIDE + v];
            if (i > 0 || (v + tid) / (2 * S) < last_rows) part[v] = sum;
        }
        part -= 8 * 2 * S;
    };

#pragma unroll
    for (int i = 0; i < kAhead; ++i) load();
    ask(0);
    // P of the segment's end: the final state's gradient through the later segments, all groups side by side (their loads
    // are what this takes)
    {
        float4 A[H::K], P[H::K];
        size_t e[H::K];
        bool there[H::K];
#pragma unroll
        for (int k = 0; k < H::K; ++k) {
            const int c = k * CHK + w0 + chan;
            there[k] = c < left;
            e[k] = e0 + (there[k] ? c : 0);
            A[k] = *reinterpret_cast<const float4 *>(p.A + e[k] * S + 4 * r);
            P[k] = p.dfinal && there[k] ? *reinterpret_cast<const float4 *>(p.dfinal + ((size_t)b * p.E + e[k]) * S + 4 * r)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 3
        for (int j = p.nseg - 1; j > seg; --j) {
            const size_t w = ((size_t)b * p.nseg + j) * p.E;
#pragma unroll
            for (int k = 0; k < H::K; ++k) {
                const float d = there[k] ? p.seg_d[w + e[k]] * kLog2e : 0.f;
                const float4 R = there[k] ? *reinterpret_cast<const float4 *>(p.seg_state + (w + e[k]) * S + 4 * r) : make_float4(0.f, 0.f, 0.f, 0.f);
                P[k] = make_float4(join(d, A[k].x, P[k].x, R.x), join(d, A[k].y, P[k].y, R.y), join(d, A[k].z, P[k].z, R.z),
                                   join(d, A[k].w, P[k].w, R.w));
            }
        }
#pragma unroll
        for (int k = 0; k < H::K; ++k) {
            keep_P[k * TH] = P[k];
            keep_dA[k * TH] = make_float4(0.f, 0.f, 0.f, 0.f);
            // A place without a channel has the bias of another and a dt of 0, a step that no token takes: with that one's A its
            // decay could have no value, and infinity times 0 in its sums would reach dB and dC through the other lanes.  With an A
            // of 0 every decay is 1.
            keep_A[k * TH] = there[k] ? make_float4(A[k].x * kLog2e, A[k].y * kLog2e, A[k].z * kLog2e, A[k].w * kLog2e)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            keep_c[k * TH] = make_float2(p.dt_bias ? p.dt_bias[e[k]] : 0.f, p.skip ? p.skip[e[k]] : 0.f);
            keep_s[k * TH] = make_float2(0.f, 0.f);
        }
    }
    widen(0);
    ask(1);
    // h at the start of a unit's tokens, read a unit ahead
    const float4 *kept = reinterpret_cast<const float4 *>(p.kept) +
                         (((size_t)b * ((p.N + kSsmTile - 1) / kSsmTile) + t0 / 8 + nt - 1) * LPC + r) * p.E + e0 + w0 + chan;
    const long long kept_wrap = -(long long)LPC * p.E - (long long)(nk - 1) * CHK;
    const int kept_k = groups(w0 + chan);
    int next_k = 0;
    auto take = [&]() {
        const float4 h = next_k < kept_k ? *kept : make_float4(0.f, 0.f, 0.f, 0.f);
        const bool wraps = next_k + 1 == nk;
        kept += wraps ? kept_wrap : CHK;
        next_k = wraps ? 0 : next_k + 1;
        return h;
    };

    // The lane's own tokens of a unit, in pairs (of one: it and itself).
    struct Own {
        F2 x[OP], d[OP], u[OP], dy[OP], slope[OP], gz[OP];
        float skip;
    };
    const int own = LPC == 16 ? r % 8 : r * OWN;
    const unsigned own_at = own * H::ROW + chan * (int)sizeof(T);
    auto prepare = [&](const unsigned char *st, int k, int t, Own &w) {      // t: of the first own token, from t0 on
        const float2 es = keep_c[k * TH];
        w.skip = es.y;
#pragma unroll
        for (int o = 0; o < OP; ++o) {
            const unsigned char *at = st + own_at + 2 * o * H::ROW;
            auto get = [&](int m) {
                const unsigned char *q = at + m * H::XBYTES;
                return F2{to_f32(*reinterpret_cast<const T *>(q)), to_f32(*reinterpret_cast<const T *>(q + (OWN > 1 ? H::ROW : 0)))};
            };
            w.x[o] = get(0);
            const F2 v = add2(get(1), f2(es.x)), g = get(3);
            F2 ev;
            const F2 plus = softplus(v, ev), s1 = add2(ev, f2(1.f)), q = F2{rcp(s1.x), rcp(s1.y)};
            const F2 sl = mul2(q, F2{v.x >= 0.f ? 1.f : ev.x, v.y >= 0.f ? 1.f : ev.y});
            // (past the length: h stays as it is)
            const bool in0 = t + 2 * o < n, in1 = t + 2 * o + 1 < n;
            w.d[o] = F2{in0 ? (sp ? plus.x : v.x) : 0.f, in1 ? (sp ? plus.y : v.y) : 0.f};
            w.slope[o] = F2{in0 ? (sp ? sl.x : 1.f) : 0.f, in1 ? (sp ? sl.y : 1.f) : 0.f};
            w.u[o] = mul2(w.d[o], w.x[o]);
            // (z sigmoid(z))' = s (1 + z (1 - s)) = s + z s (1 - s)
            const F2 z = get(2), sz = sigmoid(z), zs = mul2(z, sz);
            w.dy[o] = mul2(g, F2{gated ? zs.x : 1.f, gated ? zs.y : 1.f});
            w.gz[o] = mul2(g, fma2(zs, F2{1.f - sz.x, 1.f - sz.y}, sz));
        }
    };
    auto all = [&](const F2 (&v)[OP], int j) {   // token j's value, from the lane that owns it
        const int o = j % OWN;
        return f2(__shfl_sync(0xffffffffu, o % 2 ? v[o / 2].y : v[o / 2].x, j / OWN * CPW + chan));
    };
    Own now;
    float4 h_next = nt > 0 ? take() : make_float4(0.f, 0.f, 0.f, 0.f);
    copy_wait<kAhead - 1>();
    __syncwarp();
    prepare(ring, 0, (nt - 1) * 8 + own, now);
    int at = 0;
    for (int i = 0; i < nt; ++i) {
        __syncthreads();   // the tile's B and C are whole, and the warps' dB and dC of the one before
        if (i > 0) leave_bc(i - 1);
        widen(i + 1);
        ask(i + 2);
        const float *bc = wide + (i & 1) * H::WIDE + 4 * r;
        const int first = (nt - 1 - i) * 8;
        F2 accB[8][2], accC[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int m = 0; m < 2; ++m) accB[j][m] = accC[j][m] = f2(0.f);
#pragma unroll 1
        for (int k = 0; k < nk; ++k) {
            copy_wait<kAhead - 2>();
            __syncwarp();   // the next unit's rows have come; the last one's outputs are whole
            if (i + k > 0) leave();
            load();
            unsigned char *const st = ring + at + own_at;
            at = (at + H::UNIT) % (kRing * H::UNIT);
            const float4 h4 = h_next;
            if (i + 1 < nt || k + 1 < nk) h_next = take();
            const float4 A4 = keep_A[k * TH], P4 = keep_P[k * TH], dA4 = keep_dA[k * TH];
            const F2 A[2] = {F2{A4.x, A4.y}, F2{A4.z, A4.w}};
            const F2 d0 = all(now.d, 0), tilt = tilt_of(d0.x * fminf(fminf(fabsf(A4.x), fabsf(A4.y)), fminf(fabsf(A4.z), fabsf(A4.w))));
            Own then;
            prepare(ring + at, k + 1 < nk ? k + 1 : 0, first - (k + 1 < nk ? 0 : 8) + own, then);
            // forward: h after each token
            F2 hs[8][2];
            {
                F2 h[2] = {F2{h4.x, h4.y}, F2{h4.z, h4.w}};
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const F2 dj = j == 0 ? d0 : all(now.d, j), uj = all(now.u, j), gj = all(now.dy, j);
                    const float4 B4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S), C4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S + S);
                    const F2 Bj[2] = {F2{B4.x, B4.y}, F2{B4.z, B4.w}}, Cj[2] = {F2{C4.x, C4.y}, F2{C4.z, C4.w}};
                    F2 acc;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        h[m] = fma2(decay2(dj, A[m], tilt), h[m], mul2(uj, Bj[m]));
                        hs[j][m] = h[m];
                        accC[j][m] = fma2(gj, h[m], accC[j][m]);
                        acc = m == 0 ? mul2(Cj[m], h[m]) : fma2(Cj[m], h[m], acc);
                    }
                    y[j] = acc.x + acc.y;
                }
                part_sums<LPC, 8>(y, lane);
#pragma unroll
                for (int o = 0; o < OP; ++o) {   // (without a gate: into the place of z, which nothing reads)
                    const F2 dz = mul2(now.gz[o], fma2(f2(now.skip), now.x[o], F2{y[2 * o], OWN > 1 ? y[2 * o + 1] : y[2 * o]}));
                    unsigned char *q = st + 2 * o * H::ROW + 2 * H::XBYTES;
                    if (LPC < 16 || r < 8) *reinterpret_cast<T *>(q) = from_f32<T>(dz.x);
                    if (OWN > 1) *reinterpret_cast<T *>(q + H::ROW) = from_f32<T>(dz.y);
                }
            }
            // and back (the decays are written as found again; the compiler keeps those of the way there: one ex2 a state runs)
            float du[8], dq[8];
            F2 P[2] = {F2{P4.x, P4.y}, F2{P4.z, P4.w}}, dA[2];   // (dA of the eight tokens first: short sums)
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                const F2 dj = all(now.d, j), uj = all(now.u, j), gj = all(now.dy, j);
                const float4 B4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S), C4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S + S);
                const F2 Bj[2] = {F2{B4.x, B4.y}, F2{B4.z, B4.w}}, Cj[2] = {F2{C4.x, C4.y}, F2{C4.z, C4.w}};
                F2 sb, sq;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const F2 before = j > 0 ? hs[j > 0 ? j - 1 : 0][m] : m == 0 ? F2{h4.x, h4.y} : F2{h4.z, h4.w};
                    const F2 G = fma2(Cj[m], gj, P[m]);
                    sb = m == 0 ? mul2(G, Bj[m]) : fma2(G, Bj[m], sb);
                    accB[j][m] = fma2(G, uj, accB[j][m]);
                    P[m] = mul2(decay2(dj, A[m], tilt), G);
                    const F2 q = mul2(P[m], before);
                    sq = m == 0 ? mul2(q, A[m]) : fma2(q, A[m], sq);
                    dA[m] = j == 7 ? mul2(q, dj) : fma2(q, dj, dA[m]);
                }
                du[j] = sb.x + sb.y;
                dq[j] = sq.x + sq.y;
            }
            keep_P[k * TH] = make_float4(P[0].x, P[0].y, P[1].x, P[1].y);
            keep_dA[k * TH] = make_float4(dA4.x + dA[0].x, dA4.y + dA[0].y, dA4.z + dA[1].x, dA4.w + dA[1].y);
            part_sums<LPC, 8>(du, lane);
            part_sums<LPC, 8>(dq, lane);
            float2 es = keep_s[k * TH];
#pragma unroll
            for (int o = 0; o < OP; ++o) {
                const F2 s1 = F2{du[2 * o], OWN > 1 ? du[2 * o + 1] : du[2 * o]}, s2 = F2{dq[2 * o], OWN > 1 ? dq[2 * o + 1] : dq[2 * o]};
                const F2 dx = fma2(now.d[o], s1, mul2(f2(now.skip), now.dy[o]));
                // (past the length: d, x, dy and the slope are zeros, the sums over states are not)
                const F2 ddt = mul2(fma2(now.x[o], s1, mul2(f2(kLn2), s2)), now.slope[o]), ey = mul2(now.dy[o], now.x[o]);
                es.x += OWN > 1 ? ey.x + ey.y : ey.x;
                es.y += OWN > 1 ? ddt.x + ddt.y : ddt.x;
                unsigned char *q = st + 2 * o * H::ROW;
                if (LPC < 16 || r < 8) {
                    *reinterpret_cast<T *>(q) = from_f32<T>(dx.x);
                    *reinterpret_cast<T *>(q + H::XBYTES) = from_f32<T>(ddt.x);
                }
                if (OWN > 1) {
                    *reinterpret_cast<T *>(q + H::ROW) = from_f32<T>(dx.y);
                    *reinterpret_cast<T *>(q + H::ROW + H::XBYTES) = from_f32<T>(ddt.y);
                }
            }
            keep_s[k * TH] = es;
            now = then;
        }
        // dB and dC of the tile over the warp's channels: lanes of the same states exchange halves of the 64 sums (value
        // j * 8 + n: token j; n < 4: dB, else dC, of the lane's 4 states), until each is with one lane
        float v[64];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                v[j * 8 + 2 * m] = accB[j][m].x;
                v[j * 8 + 2 * m + 1] = accB[j][m].y;
                v[j * 8 + 4 + 2 * m] = accC[j][m].x;
                v[j * 8 + 4 + 2 * m + 1] = accC[j][m].y;
            }
        int base = 0, half = 64;
#pragma unroll
        for (int m = CPW / 2; m >= 1; m >>= 1) {
            half >>= 1;
            const bool up = lane & m;
            base += up ? half : 0;
#pragma unroll
            for (int q = 0; q < 32; ++q)
                if (q < half) {
                    const float send = up ? v[q] : v[q + half], hold = up ? v[q + half] : v[q];
                    v[q] = hold + __shfl_xor_sync(0xffffffffu, send, m);
                }
        }
        constexpr int LEFT = 64 / CPW;   // values a lane is left with
        float *sums = red + ((i & 1) * H::NW + warp) * H::WIDE + 4 * r;
#pragma unroll
        for (int q = 0; q < LEFT; q += 4) {
            const int w = base + q;
            *reinterpret_cast<float4 *>(sums + (w / 8) * 2 * S + (w % 8 / 4) * S) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
        }
    }
    __syncthreads();
    if (nt > 0) {
        leave_bc(nt - 1);
        leave();
    }
    // rows past the length
    {
        constexpr int XV = H::CH / H::V;
        T *const out3[3] = {static_cast<T *>(p.dx), static_cast<T *>(p.ddt), static_cast<T *>(p.dz)};
#pragma unroll
        for (int m = 0; m < 3; ++m) {
            if (m == 2 && !gated) continue;
            T *out = out3[m] + ((long long)b * p.N + t0) * p.E + e0;
            for (long long v = (long long)n * XV + tid; v < (long long)(t1 - t0) * XV; v += TH) {
                const int c = (int)(v % XV) * H::V;
                if (c < left) *reinterpret_cast<uint4 *>(out + (v / XV) * p.E + c) = make_uint4(0, 0, 0, 0);
            }
        }
    }
#pragma unroll 1
    for (int k = 0; k < nk; ++k) {
        const int c = k * CHK + w0 + chan;
        const bool there = c < left;
        const size_t e = e0 + (there ? c : 0), w = (size_t)b * p.nseg + seg;
        float2 es = keep_s[k * TH];
#pragma unroll
        for (int m = 1; m < (LPC == 16 ? 8 : LPC); m <<= 1) {
            es.x += __shfl_xor_sync(0xffffffffu, es.x, m * CPW);
            es.y += __shfl_xor_sync(0xffffffffu, es.y, m * CPW);
        }
        if (!there) continue;
        *reinterpret_cast<float4 *>(p.part_A + (w * p.E + e) * S + 4 * r) = keep_dA[k * TH];
        if (r == 0) {
            p.part_e[(w * 2) * p.E + e] = es.x;
            p.part_e[(w * 2 + 1) * p.E + e] = es.y;
        }
        if (p.dinit && seg == 0) *reinterpret_cast<float4 *>(p.dinit + ((size_t)b * p.E + e) * S + 4 * r) = keep_P[k * TH];
    }
}

// The parts added up in a fixed order: dB and dC over the blocks of a group (a thread four states of a token),
// dA over batch and segments (a thread four states of a channel), skip's and dt_bias' gradients (a thread a channel).
template <typename T>
__global__ void __launch_bounds__(256) k_ssm_reduce(SsmReduceParams p, unsigned bc_blocks, unsigned a_blocks) {
    pdl_wait();
    if (blockIdx.x < bc_blocks) {
        const int q = p.S / 2;                                               // float4s of a token's row (dB, dC)
        const long long i = (long long)blockIdx.x * 256 + threadIdx.x, row = i / q;
        if (row >= (long long)p.G * p.nB * p.N) return;
        const int w = (int)(i % q);
        const int g = (int)(row % p.G);
        const long long bt = row / p.G;                                      // (row order of the outputs: batch, token, group)
        const int b = (int)(bt / p.N), t = (int)(bt % p.N);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < (p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N))
#pragma unroll 8
            for (int c = 0; c < p.blocks; ++c) {
                const float4 v = *reinterpret_cast<const float4 *>(
                    p.part_bc + ((size_t)(g * p.blocks + c) * p.nB * p.N + bt) * (2 * p.S) + 4 * w);
                s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
            }
        T *to = static_cast<T *>(w < q / 2 ? p.dB : p.dC) + row * p.S + 4 * (w % (q / 2));
        to[0] = from_f32<T>(s.x);
        to[1] = from_f32<T>(s.y);
        to[2] = from_f32<T>(s.z);
        to[3] = from_f32<T>(s.w);
        return;
    }
    if (blockIdx.x < bc_blocks + a_blocks) {
        const size_t i = (size_t)(blockIdx.x - bc_blocks) * 256 + threadIdx.x, n = (size_t)p.E * p.S / 4;
        if (i >= n) return;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int w = 0; w < p.parts; ++w) {
            const float4 v = reinterpret_cast<const float4 *>(p.part_A)[w * n + i];
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
        reinterpret_cast<float4 *>(p.dA)[i] = s;
        return;
    }
    const int i = (blockIdx.x - bc_blocks - a_blocks) * 256 + threadIdx.x;
    if (i >= 2 * p.E) return;
    float *to = i < p.E ? p.dskip : p.dbias;
    if (!to) return;
    float s = 0.f;
#pragma unroll 8
    for (int w = 0; w < p.parts; ++w) s += p.part_e[(size_t)w * 2 * p.E + i];
    to[i % p.E] = s;
}

template <typename T, int S>
cudaError_t launch(const SsmParams &p, cudaStream_t s) {
    using H = Shape<T, S>;
    TraceScope tr("ssm_grad", s);
    auto kern = k_ssm_grad<T, S>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, H::SMEM);
    if (e != cudaSuccess) return e;
    const long long blocks = (long long)((p.Eg + H::CH - 1) / H::CH) * p.G * p.nB * p.nseg;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(H::THREADS), H::SMEM, s, p);
}

}  // namespace

int ssm_grad_channels(int S) { return warps_of(S) * (32 / (S / 4)) * groups_of(S); }

cudaError_t ssm_grad(const SsmParams &p, la_dtype dt, cudaStream_t s) {
    if (dt == LA_BF16) {
        if (p.S == 8) return launch<__nv_bfloat16, 8>(p, s);
        if (p.S == 16) return launch<__nv_bfloat16, 16>(p, s);
        if (p.S == 32) return launch<__nv_bfloat16, 32>(p, s);
        return launch<__nv_bfloat16, 64>(p, s);
    }
    if (p.S == 8) return launch<float, 8>(p, s);
    if (p.S == 16) return launch<float, 16>(p, s);
    if (p.S == 32) return launch<float, 32>(p, s);
    return launch<float, 64>(p, s);
}

cudaError_t ssm_reduce(const SsmReduceParams &p, la_dtype dt, cudaStream_t s) {
    TraceScope tr("ssm_reduce", s);
    const long long bc = (long long)p.nB * p.N * p.G * (p.S / 2);
    const unsigned nbc = (unsigned)((bc + 255) / 256), na = (unsigned)(((size_t)p.E * p.S / 4 + 255) / 256),
                   ne = (unsigned)((2 * (size_t)p.E + 255) / 256);
    auto kern = dt == LA_BF16 ? k_ssm_reduce<__nv_bfloat16> : k_ssm_reduce<float>;
    return launch_pdl(kern, dim3(nbc + na + ne), dim3(256), 0, s, p, nbc, na);
}

}  // namespace la
